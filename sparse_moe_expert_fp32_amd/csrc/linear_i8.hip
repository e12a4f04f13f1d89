// Product of int8 rows with int8 matrices (one, or one per expert), a float32
// scale per row and per output channel:
//   out[p][n] = a_scale[r] w_scale[e][n] sum_k a[r][k] w[e][n][k],
//   r = row_src ? row_src[p] / row_div : p,  offsets[e] <= p < offsets[e+1].
// The sums are exact in int32 (K <= 65536); the two scales are applied in
// float32 and the result is rounded once to the output type.
#include <algorithm>

#include "common.h"
#include "kernels.h"
#include "mfma.h"

namespace moe {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

// D = A(16x64) B(64x16) + C in int32: lane l holds A row l%16 / B column l%16
// with 16 consecutive K bytes of lane group l/16; D lane l holds column l%16,
// rows 4 (l/16) .. + 3.
DEV i32x4_t mfma_i8(uint4 a, uint4 b, i32x4_t c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, a),
                                               __builtin_bit_cast(i32x4_t, b), c, 0, 0, 0);
}

// One 64-row x 64-channel tile per block of 4 waves, each wave 16 rows.
// blockIdx.y counts the tiles of the experts in order.
template <typename T>
__global__ __launch_bounds__(256) void linear_i8_kernel(LinearI8Args A) {
  __shared__ int tile[2];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, lr = lane & 15, lg = lane >> 4;
  if (tid == 0) {
    int left = blockIdx.y, e = 0;
    tile[0] = -1;
    for (; e < A.E; ++e) {
      const int lo = A.offsets ? min(max(A.offsets[e], 0), A.M) : 0;
      const int hi = A.offsets ? min(A.offsets[e + 1], A.M) : A.M;
      const int n = hi > lo ? (hi - lo + 63) / 64 : 0;
      if (left < n) {
        tile[0] = e;
        tile[1] = lo + 64 * left;
        break;
      }
      left -= n;
    }
  }
  __syncthreads();
  const int e = tile[0], p0 = tile[1];
  if (e < 0) return;
  const int end = A.offsets ? min(A.offsets[e + 1], A.M) : A.M;
  const int n0 = blockIdx.x * 64;
  const int p = p0 + 16 * w + lr, pc = min(p, end - 1);
  const int r = min(max(A.row_src ? A.row_src[pc] / A.row_div : pc, 0), A.a_rows - 1);
  const int8_t *ap = A.a + (size_t)r * A.lda;
  const int8_t *wp[4];
#pragma unroll
  for (int f = 0; f < 4; ++f)
    wp[f] = A.w + ((size_t)e * A.N + min(n0 + 16 * f + lr, A.N - 1)) * A.ldw;
  i32x4_t acc[4] = {};
  for (int k = 16 * lg; k < ((A.K + 63) & ~63); k += 64) {
    const uint4 av = *reinterpret_cast<const uint4 *>(ap + k);
    const int kw = min(k, (int)A.ldw - 16);
#pragma unroll
    for (int f = 0; f < 4; ++f)
      acc[f] = mfma_i8(*reinterpret_cast<const uint4 *>(wp[f] + kw), av, acc[f]);
  }
  if (p >= end) return;
  const float sa = A.a_scale[r];
  T *out = (T *)A.out + (size_t)p * A.ldo;
#pragma unroll
  for (int f = 0; f < 4; ++f)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = n0 + 16 * f + 4 * lg + i;
      if (n < A.N) {
        const float sw = A.w_scale ? A.w_scale[(size_t)e * A.N + n] : 1.0f;
        Elem<T>::st(out, n, (float)acc[f][i] * (sa * sw));
      }
    }
}

void launch_linear_i8(bool bf16, const LinearI8Args &A, hipStream_t st) {
  const int tiles = (A.M + 63) / 64 + (A.offsets ? A.E : 0);
  dim3 grid((A.N + 63) / 64, tiles);
  if (bf16) linear_i8_kernel<bf16_t><<<grid, 256, 0, st>>>(A);
  else linear_i8_kernel<float><<<grid, 256, 0, st>>>(A);
}

}  // namespace moe
