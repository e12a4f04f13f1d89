// Backward of the router: the gates' gradient with respect to the logits, and
// the gradients of the router's input, weight and bias.
//
// gate_bwd, per token t with selected experts e_j, gates g_j (softmax over the
// selected logits) and slot positions p_j:
//   dgamma_j = <dy_t, e_out[p_j]>,
//   dsel_j   = g_j (dgamma_j - sum_i g_i dgamma_i),
//   dlogits[t][e] = dlogits_in[t][e] + sum_{j: e_j = e} dsel_j.
// One wave per token, the k dot products in groups of KM whose loads are in
// flight together; bound by reading e_out once.
//
// router_bwd, with D = dlogits:
//   dx = dx_in + D W^T,  dW[c][e] = sum_t x[t][c] D[t][e],  db[e] = sum_t D[t][e].
#include <algorithm>

#include "common.h"
#include "kernels.h"

namespace moe {

// 16 bytes of T as floats
template <typename T> struct V16;
template <> struct V16<float> {
  static constexpr int N = 4;
  static DEV void ld(const float *p, float *v) {
    const float4 t = *reinterpret_cast<const float4 *>(p);
    v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
  }
};
template <> struct V16<bf16_t> {
  static constexpr int N = 8;
  static DEV void ld(const bf16_t *p, float *v) {
    const uint4 t = *reinterpret_cast<const uint4 *>(p);
    const uint32_t u[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
};

template <typename T, int KM>
__global__ __launch_bounds__(256) void gate_bwd_kernel(
    const T *__restrict__ dy, const T *__restrict__ e_out, const int32_t *__restrict__ topk_idx,
    const float *__restrict__ gates, const int32_t *__restrict__ slot_pos,
    const uint8_t *__restrict__ valid, const float *dl_in, int Tn, int d, int E, int k,
    float *dl_out) {
  constexpr int V = V16<T>::N;
  const int lane = threadIdx.x & 63, t = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= Tn) return;
  const bool on = !valid || valid[t];
  float *out = dl_out + (size_t)t * E;
  if (!on) {
    for (int e = lane; e < E; e += 64) out[e] = 0.f;
    return;
  }
  // lane j < k: slot j of the token (indices kept in range)
  const int S = Tn * k;
  int ej = -1, pj = 0;
  float gj = 0.f;
  if (lane < k) {
    ej = min(max(topk_idx[(size_t)t * k + lane], 0), E - 1);
    pj = min(max(slot_pos[(size_t)t * k + lane], 0), S - 1);
    gj = gates[(size_t)t * k + lane];
  }
  float dgj = 0.f;
  for (int j0 = 0; j0 < k; j0 += KM) {
    const T *src[KM];
    float part[KM];
#pragma unroll
    for (int j = 0; j < KM; ++j) {
      src[j] = e_out + (size_t)__builtin_amdgcn_readlane(pj, min(j0 + j, k - 1)) * d;
      part[j] = 0.f;
    }
    for (int c = lane * V; c < d; c += 64 * V) {
      float a[V], b[KM][V];
      V16<T>::ld(dy + (size_t)t * d + c, a);
#pragma unroll
      for (int j = 0; j < KM; ++j) V16<T>::ld(src[j] + c, b[j]);
#pragma unroll
      for (int j = 0; j < KM; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) part[j] = fmaf(a[i], b[j][i], part[j]);
    }
#pragma unroll
    for (int j = 0; j < KM; ++j) {
      float s = part[j];
#pragma unroll
      for (int off = 32; off >= 1; off >>= 1) s += __shfl_xor(s, off);
      if (lane == j0 + j) dgj = s;
    }
  }
  if (lane >= k) dgj = 0.f;
  float mean = gj * dgj;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) mean += __shfl_xor(mean, off);
  const float dsel = gj * (dgj - mean);
  for (int e = lane; e < ((E + 63) & ~63); e += 64) {
    float v = dl_in && e < E ? dl_in[(size_t)t * E + e] : 0.f;
    for (int j = 0; j < k; ++j) {
      const int je = __builtin_amdgcn_readlane(ej, j);
      const float jd = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(dsel), j));
      if (je == e) v += jd;
    }
    if (e < E) out[e] = v;
  }
}

void launch_gate_bwd(bool bf16, const void *dy, const void *e_out, const int32_t *topk_idx,
                     const float *gates, const int32_t *slot_pos, const uint8_t *valid,
                     const float *dl_in, int T, int d, int E, int k, float *dl_out,
                     hipStream_t st) {
  const int grid = (T + 3) / 4;
#define MOE_GB(TY, KM) gate_bwd_kernel<TY, KM><<<grid, 256, 0, st>>>( \
      (const TY *)dy, (const TY *)e_out, topk_idx, gates, slot_pos, valid, dl_in, T, d, E, k, dl_out)
#define MOE_GBK(TY)          \
  if (k <= 2) MOE_GB(TY, 2); \
  else if (k <= 4) MOE_GB(TY, 4); \
  else if (k <= 6) MOE_GB(TY, 6); \
  else if (k <= 8) MOE_GB(TY, 8); \
  else MOE_GB(TY, 12);
  if (bf16) { MOE_GBK(bf16_t) } else { MOE_GBK(float) }
#undef MOE_GBK
#undef MOE_GB
}

// C[m][n] = add[m][n] + sum_k A(m, k) B(k, n) in float32, 64 x 64 tile per
// 256-thread block, 16-deep LDS stages.  A(m, k) = a[m * am + k * ak], B(k, n)
// = b[k * bk + n * bn].  von: row mask over k (VK) or m of the operand A and,
// for VK, of B.
template <typename TA, typename TC, bool VK>
__global__ __launch_bounds__(256) void gemm_f32_kernel(
    const TA *__restrict__ a, size_t am, size_t ak, const float *__restrict__ b, size_t bk,
    size_t bn, int M, int N, int K, const uint8_t *__restrict__ von, const TC *add,
    TC *out) {
  __shared__ float As[16][65], Bs[16][65];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int m0 = blockIdx.x * 64, n0 = blockIdx.y * 64;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < K; k0 += 16) {
    for (int i = tid; i < 1024; i += 256) {
      // consecutive threads along the operand's contiguous direction
      const int ka = ak == 1 ? i & 15 : i >> 6, ma = ak == 1 ? i >> 4 : i & 63;
      const int kb = bk == 1 ? i & 15 : i >> 6, nb = bk == 1 ? i >> 4 : i & 63;
      const bool oa = k0 + ka < K && m0 + ma < M && (!von || von[VK ? k0 + ka : m0 + ma]);
      const bool ob = k0 + kb < K && n0 + nb < N && (!VK || !von || von[k0 + kb]);
      As[ka][ma] = oa ? Elem<TA>::ld(a, (size_t)(m0 + ma) * am + (size_t)(k0 + ka) * ak) : 0.f;
      Bs[kb][nb] = ob ? b[(size_t)(k0 + kb) * bk + (size_t)(n0 + nb) * bn] : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < 16; ++kk) {
      float av[4], bv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) { av[i] = As[kk][ty * 4 + i]; bv[i] = Bs[kk][tx + 16 * i]; }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty * 4 + i, n = n0 + tx + 16 * j;
      if (m < M && n < N) {
        const size_t o = (size_t)m * N + n;
        Elem<TC>::st(out, o, acc[i][j] + (add ? Elem<TC>::ld(add, o) : 0.f));
      }
    }
}

__global__ __launch_bounds__(1024) void colsum_kernel(const float *__restrict__ a,
                                                      const uint8_t *__restrict__ valid, int T,
                                                      int E, float *__restrict__ out) {
  __shared__ float s[16][64];
  const int c = threadIdx.x & 63, g = threadIdx.x >> 6, e = blockIdx.x * 64 + c;
  float v = 0.f;
  if (e < E)
    for (int t = g; t < T; t += 16)
      if (!valid || valid[t]) v += a[(size_t)t * E + e];
  s[g][c] = v;
  __syncthreads();
  if (g == 0 && e < E) {
    for (int i = 1; i < 16; ++i) v += s[i][c];
    out[e] = v;
  }
}

size_t router_bwd_ws_bytes(int T, int d, int E) {
  (void)T; (void)d; (void)E;
  return 0;
}

void launch_router_bwd(bool bf16, const void *x, const float *w, const uint8_t *valid,
                       const float *dl, const void *dx_in, int T, int d, int E, void *dx,
                       float *dw, float *db, void *ws, hipStream_t st) {
  (void)ws;
  if (dx) {
    dim3 grid((T + 63) / 64, (d + 63) / 64);
    if (bf16)
      gemm_f32_kernel<float, bf16_t, false><<<grid, 256, 0, st>>>(
          dl, (size_t)E, 1, w, 1, (size_t)E, T, d, E, valid, (const bf16_t *)dx_in, (bf16_t *)dx);
    else
      gemm_f32_kernel<float, float, false><<<grid, 256, 0, st>>>(
          dl, (size_t)E, 1, w, 1, (size_t)E, T, d, E, valid, (const float *)dx_in, (float *)dx);
  }
  if (dw) {
    dim3 grid((d + 63) / 64, (E + 63) / 64);
    if (bf16)
      gemm_f32_kernel<bf16_t, float, true><<<grid, 256, 0, st>>>(
          (const bf16_t *)x, 1, (size_t)d, dl, (size_t)E, 1, d, E, T, valid, nullptr, dw);
    else
      gemm_f32_kernel<float, float, true><<<grid, 256, 0, st>>>(
          (const float *)x, 1, (size_t)d, dl, (size_t)E, 1, d, E, T, valid, nullptr, dw);
  }
  if (db) colsum_kernel<<<(E + 63) / 64, 1024, 0, st>>>(dl, valid, T, E, db);
}

}  // namespace moe
