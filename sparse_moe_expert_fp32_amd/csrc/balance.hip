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
//
// NEM is the least of 1, 4, 8 and 16 that holds the row (65536 x 64 with 1: 17 + 10
// us, with 4: 23 + 17; 65536 x 256 with 4: 25 + 22, with 8: 32 + 26; 65536 x 128
// would take 20 + 14 with 2 in the place of the 24 + 17 with 4).
//
// The backward is bound by its bytes (65536 x 460: 39 us for 242 MB), the forward
// by latency (36 us for 121 MB, 3.4 TB/s: one block per CU, the next token's row
// on its way while one is summed; 55 us without), its second kernel too (7 us);
// at small sizes all by the launches (3 to 5 us a kernel).  The reductions over
// the lanes exchange registers instead of going through LDS.
#include <algorithm>

#include "common.h"
#include "kernels.h"

namespace moe {

constexpr int BL_WAVES = 16;       // waves per block of the forward
constexpr int BL_BWD_WAVES = 4;    // and of the backward
constexpr int BL_MAX_BLOCKS = 256; // partials the second kernel adds (one block per CU)
constexpr int BL_COLS = 32;        // columns per block of the second kernel

// A value reduced over the wave, in every lane: exchanges inside each row of
// 16 lanes (pairs, quads, halves, rows), then the four row results.
template <typename Op> DEV float wave_reduce(float v, Op op) {
#define MOE_DPP(C) __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), C, 0xF, 0xF, false))
  v = op(v, MOE_DPP(0xB1));    // quad_perm [1, 0, 3, 2]
  v = op(v, MOE_DPP(0x4E));    // quad_perm [2, 3, 0, 1]
  v = op(v, MOE_DPP(0x141));   // row_half_mirror
  v = op(v, MOE_DPP(0x140));   // row_mirror
#undef MOE_DPP
  auto row = [&](int r) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 16 * r)); };
  return op(op(row(0), row(1)), op(row(2), row(3)));
}
DEV float wave_max(float v) {
  return wave_reduce(v, [](float a, float b) { return fmaxf(a, b); });
}
DEV float wave_sum(float v) {
  return wave_reduce(v, [](float a, float b) { return a + b; });
}

// One token of the forward: its row's largest logit and sum of exponentials,
// and the row as probabilities.
template <int NEM> struct BalanceRow {
  float l[NEM], mx, s;
  DEV void load(const float *row, int lane, int E) {
#pragma unroll
    for (int m = 0; m < NEM; ++m) l[m] = row[min(lane + 64 * m, E - 1)];
  }
  DEV void softmax(int lane, int E) {
    mx = -INFINITY;
#pragma unroll
    for (int m = 0; m < NEM; ++m) {
      if (lane + 64 * m >= E) l[m] = -INFINITY;
      mx = fmaxf(mx, l[m]);
    }
    mx = wave_max(mx);
    if (mx == -INFINITY) mx = 0.f;   // a row of -inf: every probability 0
    s = 0.f;
#pragma unroll
    for (int m = 0; m < NEM; ++m) {
      l[m] = expf(l[m] - mx);
      s += l[m];
    }
    s = wave_sum(s);
    const float inv = s == 0.f ? 0.f : 1.0f / s;
#pragma unroll
    for (int m = 0; m < NEM; ++m) l[m] *= inv;
  }
};

// Loads run one token ahead of the sums.  ONE: a single block, which ends the
// sums itself (no second kernel).
template <int NEM, bool ONE>
__global__ __launch_bounds__(64 * BL_WAVES) void balance_part_kernel(
    const float *__restrict__ logits, const int32_t *__restrict__ topk_idx,
    const uint8_t *__restrict__ valid, int T, int E, int k, float2 *__restrict__ stats,
    float *__restrict__ part_p, int *__restrict__ part_c, int *__restrict__ part_n,
    int *__restrict__ done, float *__restrict__ loss, int32_t *__restrict__ counts,
    float *__restrict__ prob) {
  __shared__ int hist[64 * NEM];
  __shared__ float red[BL_WAVES][64 * NEM];
  __shared__ int ntok[BL_WAVES];
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  for (int e = tid; e < 64 * NEM; e += 64 * BL_WAVES) hist[e] = 0;
  if (!ONE && blockIdx.x == 0 && tid == 0) *done = 0;   // for the second kernel
  __syncthreads();
  float col[NEM];
#pragma unroll
  for (int m = 0; m < NEM; ++m) col[m] = 0.f;
  int n = 0;
  const int stride = gridDim.x * BL_WAVES;
  int t = blockIdx.x * BL_WAVES + w;
  BalanceRow<NEM> R;
  int pick = -1;
  bool on = false;
  auto ask = [&](int u) {   // token u (clamped: a row that is not used)
    const int v = min(u, T - 1);
    R.load(logits + (size_t)v * E, lane, E);
    pick = topk_idx[(size_t)v * k + min(lane, k - 1)];
    on = !valid || valid[v];
  };
  if (t < T) ask(t);
  for (; t < T; t += stride) {
    BalanceRow<NEM> C = R;
    const int e = pick;
    const bool take = on;
    if (t + stride < T) ask(t + stride);
    if (!take) {   // (uniform) what stands in its row is not used
      if (lane == 0) stats[t] = make_float2(0.f, 0.f);
      continue;
    }
    ++n;
    if (lane < k && e >= 0 && e < E) atomicAdd(&hist[e], 1);   // integers: any order
    C.softmax(lane, E);
#pragma unroll
    for (int m = 0; m < NEM; ++m) col[m] += C.l[m];
    if (lane == 0) stats[t] = make_float2(C.mx, C.s);
  }
#pragma unroll
  for (int m = 0; m < NEM; ++m) red[w][lane + 64 * m] = col[m];
  if (lane == 0) ntok[w] = n;
  __syncthreads();
  n = 0;
#pragma unroll
  for (int i = 0; i < BL_WAVES; ++i) n += ntok[i];
  double share = 0.0;
  for (int e = tid; e < E; e += 64 * BL_WAVES) {
    if constexpr (ONE) {
      double s = 0.0;
#pragma unroll
      for (int i = 0; i < BL_WAVES; ++i) s += (double)red[i][e];
      const double mean = n > 0 ? s / n : 0.0;
      prob[e] = (float)mean;
      counts[e] = hist[e];
      share = n > 0 ? mean * ((double)hist[e] * E / ((double)n * k)) : 0.0;   // (E <= 1024: one e)
    } else {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < BL_WAVES; ++i) s += red[i][e];
      part_p[(size_t)blockIdx.x * E + e] = s;
      part_c[(size_t)blockIdx.x * E + e] = hist[e];
    }
  }
  if constexpr (ONE) {
    __shared__ double shares[BL_WAVES];
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) share += __shfl_xor(share, off);
    if (lane == 0) shares[w] = share;
    __syncthreads();
    if (tid == 0) {
      double all = 0.0;
      for (int i = 0; i < BL_WAVES; ++i) all += shares[i];
      *loss = (float)all;
      counts[E] = n;
    }
  } else if (tid == 0) {
    part_n[blockIdx.x] = n;
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
    // (nb <= 256: at most eight partials a thread, all asked for at once)
    float q[BL_MAX_BLOCKS / 32];
    int h[BL_MAX_BLOCKS / 32];
#pragma unroll
    for (int i = 0; i < BL_MAX_BLOCKS / 32; ++i) {
      const int b = min(g + 32 * i, nb - 1);
      q[i] = part_p[(size_t)b * E + e];
      h[i] = part_c[(size_t)b * E + e];
    }
#pragma unroll
    for (int i = 0; i < BL_MAX_BLOCKS / 32; ++i)
      if (g + 32 * i < nb) {
        p += (double)q[i];
        cnt += h[i];
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
__global__ __launch_bounds__(64 * BL_BWD_WAVES) void balance_bwd_kernel(
    const float *logits, const float2 *__restrict__ stats,
    const int32_t *__restrict__ counts, const uint8_t *__restrict__ valid,
    const float *__restrict__ dloss, int T, int E, int k, float *dlogits) {   // may be logits
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int stride = gridDim.x * BL_BWD_WAVES;
  int t = blockIdx.x * BL_BWD_WAVES + w;
  float l[NEM];
  float2 st;
  bool on;
  auto ask = [&](int u) {
#pragma unroll
    for (int m = 0; m < NEM; ++m) l[m] = logits[(size_t)u * E + min(lane + 64 * m, E - 1)];
    st = stats[u];
    on = !valid || valid[u];
  };
  if (t < T) ask(t);
  const double n = (double)counts[E];
  const double f = n > 0 ? (double)dloss[0] * E / (n * n * k) : 0.0;
  float wt[NEM];
#pragma unroll
  for (int m = 0; m < NEM; ++m) wt[m] = (float)(f * counts[min(lane + 64 * m, E - 1)]);
  for (; t < T; t += stride) {
    float p[NEM], s = 0.f;
    const float mx = st.x, inv = st.y == 0.f ? 0.f : 1.0f / st.y;
    const bool take = on;
#pragma unroll
    for (int m = 0; m < NEM; ++m) p[m] = l[m];
    if (t + stride < T) ask(t + stride);
#pragma unroll
    for (int m = 0; m < NEM; ++m) {
      p[m] = lane + 64 * m < E ? expf(p[m] - mx) * inv : 0.f;
      s = fmaf(p[m], wt[m], s);
    }
    s = wave_sum(s);
    float *out = dlogits + (size_t)t * E;
#pragma unroll
    for (int m = 0; m < NEM; ++m)
      if (lane + 64 * m < E) out[lane + 64 * m] = take ? p[m] * (wt[m] - s) : 0.f;
  }
}

namespace {
// up to 128 tokens one block does all (a second launch costs more than its
// eight tokens a wave)
int balance_blocks(int T) {
  return T <= 8 * BL_WAVES ? 1 : std::min(ceil_div_h(T, BL_WAVES), BL_MAX_BLOCKS);
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
#define MOE_BP(NEM, ONE) balance_part_kernel<NEM, ONE><<<nb, 64 * BL_WAVES, 0, st>>>( \
      logits, topk_idx, valid, T, E, k, (float2 *)stats, part_p, part_c, part_n, done, loss, \
      counts, prob)
#define MOE_BPN(NEM) if (nb == 1) MOE_BP(NEM, true); else MOE_BP(NEM, false);
  if (E <= 64) { MOE_BPN(1) }
  else if (E <= 256) { MOE_BPN(4) }
  else if (E <= 512) { MOE_BPN(8) }
  else { MOE_BPN(16) }
#undef MOE_BPN
#undef MOE_BP
  if (nb > 1)
    balance_sum_kernel<<<ceil_div_h(E, BL_COLS), 1024, 0, st>>>(part_p, part_c, part_n, nb, E, k,
                                                                loss, counts, prob, share, done);
}

void launch_balance_bwd(const float *logits, const float *stats, const int32_t *counts,
                        const uint8_t *valid, const float *dloss, int T, int E, int k,
                        float *dlogits, hipStream_t st) {
  const int nb = std::max(1, std::min(ceil_div_h(T, BL_BWD_WAVES), 2048));
#define MOE_BB(NEM) balance_bwd_kernel<NEM><<<nb, 64 * BL_BWD_WAVES, 0, st>>>( \
      logits, (const float2 *)stats, counts, valid, dloss, T, E, k, dlogits)
  if (E <= 64) MOE_BB(1);
  else if (E <= 256) MOE_BB(4);
  else if (E <= 512) MOE_BB(8);
  else MOE_BB(16);
#undef MOE_BB
}

}  // namespace moe
