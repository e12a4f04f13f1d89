// Rows quantized to int8 with one float32 scale per row:
//   v = x                (plain)
//   v = silu(x) u        (u given), silu(z) = z / (1 + exp(-z))
//   v times col_scale[e] (col_scale given; e the row's expert; float32 product)
//   scale = max|v| / 127, q = v / scale rounded to nearest even.
// The quotient is rounded as if computed exactly: a first guess from the
// reciprocal of the scale is at most one off, and the remainder v - q scale,
// which float32 holds exactly, decides (ties to even).  A row of zeros (or one
// whose scale underflows to 0) has scale 0 and q 0; a row with a value that is
// not finite has scale NaN and q 0, so that its products are NaN.
//
// NT threads per row (a wave, or a block when rows are few or long), 8
// adjacent columns a thread and chunk.  The first NH chunks stay in registers
// between the maximum and the quantization (their index is a compile-time
// constant: an index that a loop runs past the array would move other
// registers); what lies behind them is computed again.  Bound by memory:
// 98304 x 768 SwiGLU rows in 93 us (378 MB), 8192 x 2048 in 15 us (50 MB).
#include <algorithm>

#include "common.h"
#include "kernels.h"

namespace moe {

// Nearest whole number of v / s, ties to even (inv: 1 / s).
DEV int quant_round(float v, float s, float inv) {
  const float q = rintf(v * inv);
  const float r = fmaf(-q, s, v);          // exact: |r| <= about s
  const int i = (int)q;
  // one step towards v if |r| > s / 2, or |r| = s / 2 and q is odd: for odd q
  // the border is the float below s / 2
  const float h = __uint_as_float(__float_as_uint(0.5f * s) - (uint32_t)(i & 1));
  const int step = fabsf(r) > h ? (__float_as_int(r) >> 31) | 1 : 0;
  return min(max(i + step, -127), 127);
}

// The expert of row p: the number of experts that end at or before it.  All
// lanes of a wave ask for the same row; every load is in flight at once.
DEV int expert_of_row(const int32_t *offsets, int E, int p) {
  const int lane = threadIdx.x & 63;
  int e = 0;
  for (int i = 0; i < E; i += 64) {
    const bool ends = i + lane < E && offsets[i + lane + 1] <= p;
    e += __popcll(__ballot(ends));
  }
  return min(e, E - 1);
}

// 8 adjacent values from column c (those at K and behind are 0)
template <typename T, bool VEC> DEV void load8(const T *p, int c, int K, float *v) {
  if constexpr (VEC) {   // K is a multiple of 8 and the rows are 16-byte aligned
    if (c < K) {
      if constexpr (sizeof(T) == 2) {
        const uint4 t = *reinterpret_cast<const uint4 *>(p + c);
        const uint32_t u[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[2 * i] = __uint_as_float(u[i] << 16);
          v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        }
      } else {
        const float4 a = *reinterpret_cast<const float4 *>(p + c);
        const float4 b = *reinterpret_cast<const float4 *>(p + c + 4);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < K ? Elem<T>::ld(p, c + i) : 0.f;
  }
}

template <typename T, int NT, int NH, bool VEC, bool SWIGLU>
__global__ __launch_bounds__(256) void quant_i8_kernel(QuantArgs A) {
  constexpr int RB = 256 / NT;              // rows per block
  __shared__ uint32_t red[4];
  const int tid = threadIdx.x % NT, p = A.p0 + blockIdx.x * RB + threadIdx.x / NT;
  if (p >= A.p0 + A.M || (A.offsets && p >= A.offsets[A.E])) return;   // (NT = 256: the whole block)
  const T *x = (const T *)A.x + (size_t)p * A.ldx;
  const T *u = (const T *)A.u + (SWIGLU ? (size_t)p * A.ldu : 0);
  const float *cs = nullptr;
  if (A.col_scale)
    cs = A.col_scale + (size_t)(A.offsets ? expert_of_row(A.offsets, A.E, p) : 0) * A.K;
  auto value = [&](int c, float *v) {
    load8<T, VEC>(x, c, A.K, v);
    if constexpr (SWIGLU) {
      // (the hardware's exponential and reciprocal: a few roundings of v)
      float m[8];
      load8<T, VEC>(u, c, A.K, m);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[i] *= __builtin_amdgcn_rcpf(1.0f + __expf(-v[i])) * m[i];
    }
    if (cs) {
      float m[8];
      load8<float, VEC>(cs, c, A.K, m);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= m[i];
    }
  };
  float hold[NH][8];
  uint32_t top = 0;   // the bits of |v| order like |v|, NaN above infinity
#pragma unroll
  for (int j = 0; j < NH; ++j) value((j * NT + tid) * 8, hold[j]);
#pragma unroll
  for (int j = 0; j < NH; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(hold[j][i]) & 0x7fffffffu);
  for (int c = (NH * NT + tid) * 8; c < A.K; c += NT * 8) {
    float v[8];
    value(c, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off));
  if constexpr (NT > 64) {
    if ((tid & 63) == 0) red[tid >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) top = max(top, red[w]);
  }
  const bool finite = top < 0x7f800000u;
  const float s = finite ? __uint_as_float(top) / 127.0f : __uint_as_float(0x7fc00000u);
  const bool some = finite && s > 0.f;
  // a tiny scale and the values are multiplied by the same power of two, so
  // that its reciprocal stays finite
  const float up = s < 0x1p-100f ? 0x1p64f : 1.0f;
  const float su = some ? s * up : 1.0f, inv = 1.0f / su;
  if (tid == 0) A.scale[p] = s;
  int8_t *q = A.q + (size_t)p * A.ldq;
  auto put = [&](int c, const float *v) {
    uint32_t o[2] = {0, 0};
    if (some) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        o[i >> 2] |= ((uint32_t)quant_round(v[i] * up, su, inv) & 0xFFu) << (8 * (i & 3));
    }
    *reinterpret_cast<uint2 *>(q + c) = make_uint2(o[0], o[1]);
  };
#pragma unroll
  for (int j = 0; j < NH; ++j) {
    const int c = (j * NT + tid) * 8;
    if (c < A.ldq) put(c, hold[j]);
  }
  for (int c = (NH * NT + tid) * 8; c < A.ldq; c += NT * 8) {
    float v[8];
    value(c, v);
    put(c, v);
  }
}

// A wave per row up to 4096 columns when the rows fill the chip (eight waves a
// CU from 2048 rows on); a block of four waves per row otherwise.
constexpr int QU_WAVE_ROWS = 2048;

template <typename T, bool VEC, bool SWIGLU>
static void quant_launch(const QuantArgs &A, hipStream_t st) {
#define MOE_Q(NT, NH) \
  quant_i8_kernel<T, NT, NH, VEC, SWIGLU><<<(A.M + 256 / NT - 1) / (256 / NT), 256, 0, st>>>(A)
  const bool wave = A.M >= QU_WAVE_ROWS;
  if (wave && A.K <= 1024) MOE_Q(64, 2);
  else if (wave && A.K <= 2048) MOE_Q(64, 4);
  else if (wave && A.K <= 4096) MOE_Q(64, 8);
  else if (A.K <= 2048) MOE_Q(256, 1);
  else MOE_Q(256, 4);
#undef MOE_Q
}
template <typename T> static void quant_launch(const QuantArgs &A, bool vec, hipStream_t st) {
  if (A.u) {
    if (vec) quant_launch<T, true, true>(A, st);
    else quant_launch<T, false, true>(A, st);
  } else {
    if (vec) quant_launch<T, true, false>(A, st);
    else quant_launch<T, false, false>(A, st);
  }
}

void launch_quant_i8(bool bf16, const QuantArgs &all, hipStream_t st) {
  constexpr int kRows = 1 << 22;   // per launch: a grid's threads are counted in 32 bits
  QuantArgs A = all;
  if (all.M > kRows) {
    for (int p = 0; p < all.M; p += kRows) {
      A.p0 = all.p0 + p;
      A.M = std::min(kRows, all.M - p);
      launch_quant_i8(bf16, A, st);
    }
    return;
  }
  const int ab = bf16 ? 2 : 4;
  const bool vec = A.K % 8 == 0 &&
                   (((uintptr_t)A.x | (uintptr_t)(A.ldx * ab)) & 15) == 0 &&
                   (!A.u || (((uintptr_t)A.u | (uintptr_t)(A.ldu * ab)) & 15) == 0) &&
                   ((uintptr_t)A.col_scale & 15) == 0;
  if (bf16) quant_launch<bf16_t>(A, vec, st);
  else quant_launch<float>(A, vec, st);
}

}  // namespace moe
