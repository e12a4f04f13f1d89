// Rows quantized to int8 with one float32 scale per row:
//   v = x                (plain)
//   v = silu(x) u        (u given), silu(z) = z / (1 + exp(-z))
//   v times col_scale[e] (col_scale given; e the row's expert; float32 product)
//   scale = max|v| / 127, q = v / scale rounded to nearest even.
// The quotient is rounded as if computed exactly.  v times the reciprocal of
// the scale, added to 1.5 2^23, leaves the rounded quotient in the low byte of
// the sum; where the quotient may be too near to a half for that (one value in
// 16000), the chunk is done again, exactly: the guess is then at most one off,
// and the remainder v - q scale, which float32 holds exactly, decides (ties to
// even).  Rows of tiny scales and rows that are not finite go that way
// throughout.  A row of zeros (or one whose scale underflows to 0) has scale 0
// and q 0; a row with a value that is not finite has scale NaN and q 0, so that
// its products are NaN.
//
// NT threads per row (a wave, or a block when rows are few or long), 8
// adjacent columns a thread and chunk.  The first NH chunks stay in registers
// between the maximum and the quantization (their index is a compile-time
// constant: an index that a loop runs past the array would move other
// registers); what lies behind them, or is done again, is computed again.
// Bound by memory where there are many rows: 24576 x 2048 with channel scales in
// 30 us (150 MB), 8192 x 2048 in 13.8 us (50 MB); 46 and 15.3 us with the exact
// remainder for every value.  A few rows take 4.5 us, the latency of one pass.
// SwiGLU rows are bound by the vector units: 98304 x 768 in 110 us (378 MB), of
// which the exponential and the quotient in full float32 take 41 (69 us with the
// hardware's exponential and reciprocal, whose error grows with |x| to 63
// roundings at x = -80 and moved one value in 10^4 over a rounding border).
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

// The largest of the wave's values, in every lane: exchanges inside each row
// of 16 lanes (pairs, quads, halves, rows), then the four row results.
DEV uint32_t wave_max(uint32_t v) {
#define MOE_DPP(C) (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, C, 0xF, 0xF, false)
  v = max(v, MOE_DPP(0xB1));    // quad_perm [1, 0, 3, 2]
  v = max(v, MOE_DPP(0x4E));    // quad_perm [2, 3, 0, 1]
  v = max(v, MOE_DPP(0x141));   // row_half_mirror
  v = max(v, MOE_DPP(0x140));   // row_mirror
#undef MOE_DPP
  auto row = [&](int r) { return (uint32_t)__builtin_amdgcn_readlane((int)v, 16 * r); };
  return max(max(row(0), row(1)), max(row(2), row(3)));
}

// 8 adjacent values from column c, asked for without a condition (the columns
// held inside the row) and turned into floats (0 at K and behind) once they
// are needed.  VEC: K is a multiple of 8 and the rows are 16-byte aligned.
// p: the row, the same in the whole wave (a base and 32-bit offsets).
template <typename T, bool VEC> struct Values8 {
  T raw[8];
  DEV void load(const T *p, int c, int K) {
    const char *b = reinterpret_cast<const char *>(p);
    auto at = [&](int i) { return b + (size_t)((uint32_t)i * (uint32_t)sizeof(T)); };
    if constexpr (VEC) {
      const uint4 *q = reinterpret_cast<const uint4 *>(at(min(c, K - 8)));
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4 *>(raw)[i] = q[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) raw[i] = *reinterpret_cast<const T *>(at(min(c + i, K - 1)));
    }
  }
  DEV void get(int c, int K, float *v) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = VEC || c + i < K ? Elem<T>::ld(raw, i) : 0.f;
    if (VEC && c >= K) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
    }
  }
};

// What a value is: x, x times the channel's scale, or SwiGLU of x and u (which
// takes channel scales too where they are given).
enum QuantMode { Q_PLAIN, Q_SCALED, Q_SWIGLU };

// Waves per SIMD that the registers are held to: as many as the chunks, with
// what they are made from, leave room for.
constexpr int quant_waves(int NT, int NH, bool VEC, QuantMode MODE) {
  return NH == 1 || (VEC && NT == 64 && NH <= 4 && MODE == Q_PLAIN) ? 8 : VEC && NH <= 4 ? 5 : 1;
}

template <typename T, int NT, int NH, bool VEC, QuantMode MODE>
__global__ __launch_bounds__(256, quant_waves(NT, NH, VEC, MODE)) void quant_i8_kernel(QuantArgs A) {
  constexpr int RB = 256 / NT;              // rows per block
  constexpr bool SWIGLU = MODE == Q_SWIGLU;
  const bool scaled = MODE == Q_SCALED || (SWIGLU && A.col_scale);
  __shared__ uint32_t red[4];
  const int tid = threadIdx.x % NT;
  const int p = A.p0 + blockIdx.x * RB + __builtin_amdgcn_readfirstlane(threadIdx.x / NT);
  if (p >= A.p0 + A.M || (A.offsets && p >= A.offsets[A.E])) return;   // (NT = 256: the whole block)
  const T *x = (const T *)A.x + (size_t)p * A.ldx;
  const T *u = SWIGLU ? (const T *)A.u + (size_t)p * A.ldu : nullptr;
  const float *cs = nullptr;
  // the values asked for, and what they become
  struct Chunk {
    Values8<T, VEC> x, u;
  };
  auto ask = [&](Chunk &C, int c) {
    C.x.load(x, c, A.K);
    if constexpr (SWIGLU) C.u.load(u, c, A.K);
  };
  auto value = [&](const Chunk &C, int c, float *v) {
    C.x.get(c, A.K, v);
    if constexpr (SWIGLU) {
      // (exactly this formula in float32: a value next to a border falls where
      // the formula says, and gates far below 0 keep every bit)
      float m[8];
      C.u.get(c, A.K, m);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = v[i] / (1.0f + expf(-v[i])) * m[i];
    }
    if (scaled) {
      Values8<float, VEC> s;
      float m[8];
      s.load(cs, c, A.K);
      s.get(c, A.K, m);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= m[i];
    }
  };
  Chunk C[NH];
  const bool by_expert = scaled && A.offsets;
  // the expert of row p is the number of experts that end at or before it (all
  // lanes of a wave ask for the same row); its first 64 ends are asked for
  // before the row
  const int lane = threadIdx.x & 63;
  const int32_t end0 = by_expert ? A.offsets[min(lane + 1, A.E)] : 0;
#pragma unroll
  for (int j = 0; j < NH; ++j) ask(C[j], (j * NT + tid) * 8);
  if (scaled) {
    int e = 0;
    if (by_expert) {
      e = __popcll(__ballot(lane < A.E && end0 <= p));
      for (int i = 64; i < A.E; i += 64)
        e += __popcll(__ballot(i + lane < A.E && A.offsets[min(i + lane + 1, A.E)] <= p));
      e = min(e, A.E - 1);
    }
    cs = A.col_scale + (size_t)e * A.K;
  }
  float hold[NH][8];
  uint32_t top = 0;   // the bits of |v| order like |v|, NaN above infinity
#pragma unroll
  for (int j = 0; j < NH; ++j) {
    value(C[j], (j * NT + tid) * 8, hold[j]);
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(hold[j][i]) & 0x7fffffffu);
  }
  for (int c = (NH * NT + tid) * 8; c < A.K; c += NT * 8) {
    float v[8];
    ask(C[0], c);
    value(C[0], c, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
  }
  top = wave_max(top);
  if constexpr (NT > 64) {
    if (lane == 0) red[tid >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) top = max(top, red[w]);
  }
  const bool finite = top < 0x7f800000u;
  const float s = finite ? __uint_as_float(top) / 127.0f : __uint_as_float(0x7fc00000u);
  const bool tiny = s < 0x1p-100f;
  if (tid == 0) A.scale[p] = s;
  int8_t *q = A.q + (size_t)p * A.ldq;
  // (the reciprocal is at most 2^-23 of itself off, a quotient so 127 2^-23)
  const float fast = tiny ? 0.f : __builtin_amdgcn_rcpf(s);
  constexpr float kWhole = 12582912.f, kNear = 0.5f - 0x1p-15f;
  uint32_t again = 0;   // chunks that are not settled
#pragma unroll
  for (int j = 0; j < NH; ++j) {
    const int c = (j * NT + tid) * 8;
    uint32_t m[8];
    float far = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float w = fmaf(hold[j][i], fast, kWhole);
      far = fmaxf(far, fabsf(fmaf(hold[j][i], fast, kWhole - w)));
      m[i] = __float_as_uint(w);
    }
    if (far > kNear) again |= 1u << j;
    uint32_t o[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {   // the low bytes of four words
      const uint32_t lo = __builtin_amdgcn_perm(m[4 * h + 1], m[4 * h], 0x0c0c0400u);
      const uint32_t hi = __builtin_amdgcn_perm(m[4 * h + 3], m[4 * h + 2], 0x04000c0cu);
      o[h] = lo | hi;
    }
    if (c < A.ldq) *reinterpret_cast<uint2 *>(q + c) = make_uint2(o[0], o[1]);
  }
  if (!finite || (tiny && s > 0.f)) again = ~0u;
  if (A.ldq <= NH * NT * 8 && !__ballot(again)) return;
  // a tiny scale and the values are multiplied by the same power of two, so
  // that its reciprocal stays finite
  const float up = tiny ? 0x1p64f : 1.0f;
  const bool some = finite && s > 0.f;
  const float su = some ? s * up : 1.0f, inv = 1.0f / su;
#pragma unroll 1
  for (int c = tid * 8, j = 0; c < A.ldq; c += NT * 8, ++j) {
    if (j < NH && !(again >> j & 1)) continue;
    uint32_t o[2] = {0, 0};
    if (some) {
      float v[8];
      ask(C[0], c);
      value(C[0], c, v);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        o[i >> 2] |= ((uint32_t)quant_round(v[i] * up, su, inv) & 0xFFu) << (8 * (i & 3));
    }
    *reinterpret_cast<uint2 *>(q + c) = make_uint2(o[0], o[1]);
  }
}

// A wave per row up to 4096 columns when the rows fill the chip (eight waves a
// CU from 2048 rows on); a block of four waves per row otherwise.
constexpr int QU_WAVE_ROWS = 2048;

template <typename T, bool VEC, QuantMode MODE>
static void quant_launch(const QuantArgs &A, hipStream_t st) {
#define MOE_Q(NT, NH) \
  quant_i8_kernel<T, NT, NH, VEC, MODE><<<(A.M + 256 / NT - 1) / (256 / NT), 256, 0, st>>>(A)
  const bool wave = A.M >= QU_WAVE_ROWS;
  if (wave && A.K <= 1024) MOE_Q(64, 2);
  else if (wave && A.K <= 2048) MOE_Q(64, 4);
  else if (wave && A.K <= 4096) MOE_Q(64, 8);
  else if (A.K <= 2048) MOE_Q(256, 1);
  else MOE_Q(256, 4);
#undef MOE_Q
}
template <typename T, bool VEC> static void quant_launch(const QuantArgs &A, hipStream_t st) {
  if (A.u) quant_launch<T, VEC, Q_SWIGLU>(A, st);
  else if (A.col_scale) quant_launch<T, VEC, Q_SCALED>(A, st);
  else quant_launch<T, VEC, Q_PLAIN>(A, st);
}
template <typename T> static void quant_launch(const QuantArgs &A, bool vec, hipStream_t st) {
  if (vec) quant_launch<T, true>(A, st);
  else quant_launch<T, false>(A, st);
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
