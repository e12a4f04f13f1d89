// Load-balance loss of the routed experts, per-expert counts, and the loss's
// gradient with respect to the router logits.
//
//   counts[e] = routed slots of expert e, n = tokens that take part,
//   p_t = softmax(logits[t]) over all E experts, prob[e] = mean_t p_t[e],
//   loss = E sum_e counts[e] / (n k) prob[e],
//   dlogits[t][e] = p_t[e] (w[e] - sum_i w[i] p_t[i]),
//   w[e] = dloss E counts[e] / (n^2 k)          (counts held fixed).
//
// Both directions are one pass over the logits, one wave per token, with the
// row of a token in registers (E <= 64 NEM, expert e = lane + 64 m).  The
// forward keeps the largest logit and the sum of the exponentials of every
// row for the backward; its column sums run in float32 per wave, then per
// block in wave order, then over the blocks in double (the second kernel), so
// the result does not depend on timing.
#include <algorithm>

#include "common.h"
#include "kernels.h"

namespace moe {

constexpr int BL_WAVES = 4;        // waves per block
constexpr int BL_MAX_BLOCKS = 512; // partials the second kernel adds
constexpr int BL_COLS = 32;        // columns per block of the second kernel

DEV float wave_max(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor(v, off));
  return v;
}
DEV float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  return v;
}

template <int NEM>
__global__ __launch_bounds__(64 * BL_WAVES) void balance_part_kernel(
    const float *__restrict__ logits, const int32_t *__restrict__ topk_idx,
    const uint8_t *__restrict__ valid, int T, int E, int k, float2 *__restrict__ stats,
    float *__restrict__ part_p, int *__restrict__ part_c, int *__restrict__ part_n,
    int *__restrict__ done) {
  __shared__ int hist[64 * NEM];
  __shared__ float red[BL_WAVES][64 * NEM];
  __shared__ int ntok[BL_WAVES];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  for (int e = tid; e < 64 * NEM; e += 64 * BL_WAVES) hist[e] = 0;
  if (blockIdx.x == 0 && tid == 0) *done = 0;   // for the second kernel
  __syncthreads();
  float col[NEM];
#pragma unroll
  for (int m = 0; m < NEM; ++m) col[m] = 0.f;
  int n = 0;
  for (int t = blockIdx.x * BL_WAVES + w; t < T; t += gridDim.x * BL_WAVES) {
    if (valid && !valid[t]) {   // (uniform) what stands in its row is not read
      if (lane == 0) stats[t] = make_float2(0.f, 0.f);
      continue;
    }
    ++n;
    const float *row = logits + (size_t)t * E;
    float l[NEM], mx = -INFINITY;
#pragma unroll
    for (int m = 0; m < NEM; ++m) {
      const int e = lane + 64 * m;
      l[m] = e < E ? row[e] : -INFINITY;
      mx = fmaxf(mx, l[m]);
    }
    if (lane < k) {
      const int e = topk_idx[(size_t)t * k + lane];
      if (e >= 0 && e < E) atomicAdd(&hist[e], 1);   // integers: any order
    }
    mx = wave_max(mx);
    if (mx == -INFINITY) mx = 0.f;   // a row of -inf: every probability 0
    float s = 0.f;
#pragma unroll
    for (int m = 0; m < NEM; ++m) {
      l[m] = expf(l[m] - mx);
      s += l[m];
    }
    s = wave_sum(s);
    const float inv = s == 0.f ? 0.f : 1.0f / s;
#pragma unroll
    for (int m = 0; m < NEM; ++m) col[m] += l[m] * inv;
    if (lane == 0) stats[t] = make_float2(mx, s);
  }
#pragma unroll
  for (int m = 0; m < NEM; ++m) red[w][lane + 64 * m] = col[m];
  if (lane == 0) ntok[w] = n;
  __syncthreads();
  for (int e = tid; e < E; e += 64 * BL_WAVES) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < BL_WAVES; ++i) s += red[i][e];
    part_p[(size_t)blockIdx.x * E + e] = s;
    part_c[(size_t)blockIdx.x * E + e] = hist[e];
  }
  if (tid == 0) {
    int s = 0;
    for (int i = 0; i < BL_WAVES; ++i) s += ntok[i];
    part_n[blockIdx.x] = s;
  }
}

// Adds the partials of nb blocks: each block 32 columns, 32 threads a column
// over the blocks, then a tree in LDS in double.  The block that ends last
// adds the blocks' shares of the loss, in block order.
__global__ __launch_bounds__(1024) void balance_sum_kernel(
    const float *__restrict__ part_p, const int *__restrict__ part_c,
    const int *__restrict__ part_n, int nb, int E, int k, float *__restrict__ loss,
    int32_t *__restrict__ counts, float *__restrict__ prob, double *__restrict__ share,
    int *__restrict__ done) {
  __shared__ double sp[32][BL_COLS];
  __shared__ int sc[32][BL_COLS], sn[1024];
  __shared__ int last;
  const int tid = threadIdx.x, c = tid & 31, g = tid >> 5, e = blockIdx.x * BL_COLS + c;
  double p = 0.0;
  int cnt = 0;
  if (e < E) {
    for (int b = g; b < nb; b += 32) {
      p += (double)part_p[(size_t)b * E + e];
      cnt += part_c[(size_t)b * E + e];
    }
  }
  sp[g][c] = p;
  sc[g][c] = cnt;
  sn[tid] = tid < nb ? part_n[tid] : 0;   // nb <= BL_MAX_BLOCKS <= 1024
  __syncthreads();
  for (int h = 16; h >= 1; h >>= 1) {
    if (g < h) {
      sp[g][c] += sp[g + h][c];
      sc[g][c] += sc[g + h][c];
    }
    const int hn = 32 * h;
    if (tid < hn) sn[tid] += sn[tid + hn];
    __syncthreads();
  }
  if (tid < 32) {
    int n = sn[tid];
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) n += __shfl_xor(n, off);
    double s = 0.0;
    if (e < E) {
      const double mean = n > 0 ? sp[0][c] / n : 0.0;
      prob[e] = (float)mean;
      counts[e] = sc[0][c];
      s = n > 0 ? mean * ((double)sc[0][c] * E / ((double)n * k)) : 0.0;
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor(s, off);
    if (tid == 0) {
      if (blockIdx.x == 0) counts[E] = n;
      share[blockIdx.x] = s;
      __threadfence();
      last = atomicAdd(done, 1) == (int)gridDim.x - 1;
      if (last) {
        __threadfence();
        double all = 0.0;
        for (int b = 0; b < (int)gridDim.x; ++b)
          all += __hip_atomic_load(&share[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        *loss = (float)all;
      }
    }
  }
}

template <int NEM>
__global__ __launch_bounds__(64 * BL_WAVES) void balance_bwd_kernel(
    const float *logits, const float2 *__restrict__ stats,
    const int32_t *__restrict__ counts, const uint8_t *__restrict__ valid,
    const float *__restrict__ dloss, int T, int E, int k, float *dlogits) {   // may be logits
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const double n = (double)counts[E];
  const double f = n > 0 ? (double)dloss[0] * E / (n * n * k) : 0.0;
  float wt[NEM];
#pragma unroll
  for (int m = 0; m < NEM; ++m) {
    const int e = lane + 64 * m;
    wt[m] = e < E ? (float)(f * counts[e]) : 0.f;
  }
  for (int t = blockIdx.x * BL_WAVES + w; t < T; t += gridDim.x * BL_WAVES) {
    const bool on = !valid || valid[t];
    float *out = dlogits + (size_t)t * E;
    if (!on) {
#pragma unroll
      for (int m = 0; m < NEM; ++m)
        if (lane + 64 * m < E) out[lane + 64 * m] = 0.f;
      continue;
    }
    const float *row = logits + (size_t)t * E;
    const float2 st = stats[t];
    const float inv = st.y == 0.f ? 0.f : 1.0f / st.y;
    float p[NEM], s = 0.f;
#pragma unroll
    for (int m = 0; m < NEM; ++m) {
      const int e = lane + 64 * m;
      p[m] = e < E ? expf(row[e] - st.x) * inv : 0.f;
      s = fmaf(p[m], wt[m], s);
    }
    s = wave_sum(s);
#pragma unroll
    for (int m = 0; m < NEM; ++m)
      if (lane + 64 * m < E) out[lane + 64 * m] = p[m] * (wt[m] - s);
  }
}

namespace {
int balance_blocks(int T) {
  return std::max(1, std::min((T + BL_WAVES - 1) / BL_WAVES, BL_MAX_BLOCKS));
}
size_t al(size_t b) { return (b + 255) & ~size_t(255); }
}  // namespace

size_t balance_ws_bytes(int T, int E) {
  const size_t nb = balance_blocks(T);
  return 2 * al(nb * E * 4) + al(nb * 4) + al((size_t)ceil_div_h(E, BL_COLS) * 8) + 256;
}

void launch_balance_fwd(const float *logits, const int32_t *topk_idx, const uint8_t *valid, int T,
                        int E, int k, float *loss, int32_t *counts, float *prob, float *stats,
                        void *ws, hipStream_t st) {
  const int nb = balance_blocks(T);
  char *b = (char *)ws;
  float *part_p = (float *)b;
  b += al((size_t)nb * E * 4);
  int *part_c = (int *)b;
  b += al((size_t)nb * E * 4);
  int *part_n = (int *)b;
  b += al((size_t)nb * 4);
  double *share = (double *)b;
  b += al((size_t)ceil_div_h(E, BL_COLS) * 8);
  int *done = (int *)b;
#define MOE_BP(NEM) balance_part_kernel<NEM><<<nb, 64 * BL_WAVES, 0, st>>>( \
      logits, topk_idx, valid, T, E, k, (float2 *)stats, part_p, part_c, part_n, done)
  if (E <= 64) MOE_BP(1);
  else if (E <= 256) MOE_BP(4);
  else if (E <= 512) MOE_BP(8);
  else MOE_BP(16);
#undef MOE_BP
  balance_sum_kernel<<<ceil_div_h(E, BL_COLS), 1024, 0, st>>>(part_p, part_c, part_n, nb, E, k,
                                                              loss, counts, prob, share, done);
}

void launch_balance_bwd(const float *logits, const float *stats, const int32_t *counts,
                        const uint8_t *valid, const float *dloss, int T, int E, int k,
                        float *dlogits, hipStream_t st) {
  const int nb = std::max(1, std::min((T + BL_WAVES - 1) / BL_WAVES, 2048));
#define MOE_BB(NEM) balance_bwd_kernel<NEM><<<nb, 64 * BL_WAVES, 0, st>>>( \
      logits, (const float2 *)stats, counts, valid, dloss, T, E, k, dlogits)
  if (E <= 64) MOE_BB(1);
  else if (E <= 256) MOE_BB(4);
  else if (E <= 512) MOE_BB(8);
  else MOE_BB(16);
#undef MOE_BB
}

}  // namespace moe
