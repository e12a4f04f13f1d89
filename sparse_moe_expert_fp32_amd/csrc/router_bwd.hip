// Backward of the router: the gates' gradient with respect to the logits, and
// the gradients of the router's input, weight and bias.
//
// gate_bwd, per token t with selected experts e_j, gates g_j (softmax over the
// selected logits) and slot positions p_j:
//   dgamma_j = <dy_t, e_out[p_j]>,
//   dsel_j   = g_j (dgamma_j - sum_i g_i dgamma_i),
//   dlogits[t][e] = dlogits_in[t][e] + sum_{j: e_j = e} dsel_j.
// One wave per token, the k dot products in groups of KM whose loads are in
// flight together; bound by reading e_out once (8192 tokens, k = 12, d = 2048:
// 99 us for 470 MB; the loads of one piece of all rows are asked for before
// anything waits, and stay as loaded until their turn: more waves fit, 113 -> 99).
//
// router_bwd, with D = dlogits:
//   dx = dx_in + D W^T,  dW[c][e] = sum_t x[t][c] D[t][e],  db[e] = sum_t D[t][e].
// Bound by the products (8192 x 2048 x 460 in three planes: dx 78 us, dW 78 us
// and 7 for its partial sums, 0.6 PFLOP/s each; in float32 on the vector units
// 1.3 ms each.  4096 x 2048 x 460 in float32, six plane products: dx 87, dW 97 and
// 8).  db without dW is a plain column sum, 168 us for 8192 x 460: its few blocks
// walk the tokens one after another.
#include <algorithm>

#include "common.h"
#include "kernels.h"
#include "mfma.h"

namespace moe {

// The sum over the wave, in every lane: exchanges inside each row of 16 lanes
// (pairs, quads, halves, rows), then the four row sums.
DEV float wave_sum(float v) {
#define MOE_DPP(C) __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), C, 0xF, 0xF, false))
  v += MOE_DPP(0xB1);    // quad_perm [1, 0, 3, 2]
  v += MOE_DPP(0x4E);    // quad_perm [2, 3, 0, 1]
  v += MOE_DPP(0x141);   // row_half_mirror
  v += MOE_DPP(0x140);   // row_mirror
#undef MOE_DPP
  auto row = [&](int r) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 16 * r)); };
  return (row(0) + row(1)) + (row(2) + row(3));
}

// 16 bytes of T as floats
template <typename T> struct V16;
template <> struct V16<float> {
  static constexpr int N = 4;
  static DEV void get(uint4 t, float *v) {
    v[0] = __uint_as_float(t.x); v[1] = __uint_as_float(t.y);
    v[2] = __uint_as_float(t.z); v[3] = __uint_as_float(t.w);
  }
};
template <> struct V16<bf16_t> {
  static constexpr int N = 8;
  static DEV void get(uint4 t, float *v) {
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
    const uint8_t *__restrict__ valid, const float *dl_in, int Tn, int S, int d, int E, int k,
    float *dl_out) {
  constexpr int V = V16<T>::N, NE = 8;
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (t >= Tn) return;
  float *out = dl_out + (size_t)t * E;
  if (valid && !valid[t]) {
    for (int e = lane; e < E; e += 64) out[e] = 0.f;
    return;
  }
  // lane j < k: slot j of the token (indices kept in range)
  const int at = min(lane, k - 1);
  const int ej = min(max(topk_idx[(size_t)t * k + at], 0), E - 1);
  const int pj = min(max(slot_pos[(size_t)t * k + at], 0), S - 1);
  const float gj = lane < k ? gates[(size_t)t * k + at] : 0.f;
  // the token's row of dl_in (without one: of the output, not used), 64 NE
  // experts at a time; the first ones are on their way during the dot products
  float old[NE];
  const char *in = reinterpret_cast<const char *>((dl_in ? dl_in : dl_out) + (size_t)t * E);
  auto ask = [&](int e0) {
#pragma unroll
    for (int m = 0; m < NE; ++m)
      old[m] = *reinterpret_cast<const float *>(in + (size_t)(4u * (uint32_t)min(e0 + 64 * m + lane, E - 1)));
  };
  float dgj = 0.f;
  for (int j0 = 0; j0 < k; j0 += KM) {
    const char *src[KM];
    float part[KM];
#pragma unroll
    for (int j = 0; j < KM; ++j) {
      src[j] = reinterpret_cast<const char *>(
          e_out + (size_t)__builtin_amdgcn_readlane(pj, min(j0 + j, k - 1)) * d);
      part[j] = 0.f;
    }
    if (j0 == 0) ask(0);
    const char *row = reinterpret_cast<const char *>(dy + (size_t)t * d);
    const uint32_t bytes = (uint32_t)(d * sizeof(T));   // a multiple of 16
    for (uint32_t c0 = 0; c0 < bytes; c0 += 64 * 16) {
      // (behind the end: the last piece again, not used)
      const uint32_t c = min(c0 + 16 * lane, bytes - 16);
      const bool inside = c0 + 16 * lane < bytes;
      const uint4 ra = *reinterpret_cast<const uint4 *>(row + (size_t)c);
      uint4 rb[KM];
#pragma unroll
      for (int j = 0; j < KM; ++j) rb[j] = *reinterpret_cast<const uint4 *>(src[j] + (size_t)c);
      __builtin_amdgcn_sched_barrier(0);   // (the loads first, and as loaded until their turn)
      if (inside) {
        float a[V], b[V];
        V16<T>::get(ra, a);
#pragma unroll
        for (int j = 0; j < KM; ++j) {
          V16<T>::get(rb[j], b);
#pragma unroll
          for (int i = 0; i < V; ++i) part[j] = fmaf(a[i], b[i], part[j]);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < KM; ++j) {
      const float s = wave_sum(part[j]);
      if (lane == j0 + j) dgj = s;
    }
  }
  if (lane >= k) dgj = 0.f;
  const float mean = wave_sum(gj * dgj);
  const float dsel = gj * (dgj - mean);
  for (int e0 = 0; e0 < E; e0 += 64 * NE) {
    if (e0 > 0) ask(e0);
    if (!dl_in) {
#pragma unroll
      for (int m = 0; m < NE; ++m) old[m] = 0.f;
    }
    for (int j = 0; j < k; ++j) {
      const int je = __builtin_amdgcn_readlane(ej, j) - e0 - lane;
      const float jd = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(dsel), j));
#pragma unroll
      for (int m = 0; m < NE; ++m) old[m] += je == 64 * m ? jd : 0.f;
    }
#pragma unroll
    for (int m = 0; m < NE; ++m)
      if (e0 + 64 * m + lane < E) out[e0 + 64 * m + lane] = old[m];
  }
}

void launch_gate_bwd(bool bf16, const void *dy, const void *e_out, const int32_t *topk_idx,
                     const float *gates, const int32_t *slot_pos, const uint8_t *valid,
                     const float *dl_in, int T, int d, int E, int k, float *dl_out,
                     hipStream_t st) {
  constexpr int kTokens = 1 << 24;   // per launch: a grid's threads are counted in 32 bits
  const int S = T * k;
  for (int t0 = 0; t0 < T; t0 += kTokens) {
    const int n = std::min(kTokens, T - t0), grid = (n + 3) / 4;
    const size_t slot = (size_t)t0 * k, row = (size_t)t0 * E;
#define MOE_GB(TY, KM) gate_bwd_kernel<TY, KM><<<grid, 256, 0, st>>>( \
      (const TY *)dy + (size_t)t0 * d, (const TY *)e_out, topk_idx + slot, gates + slot, \
      slot_pos + slot, valid ? valid + t0 : nullptr, dl_in ? dl_in + row : nullptr, n, S, d, E, k, \
      dl_out + row)
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
}

// ---- the two products in float32 accuracy on the bf16 matrix cores.
//
// A float32 value is the sum of three bf16 values exactly: each plane is what is
// left, rounded to nearest (at most 2^-8 of the value is left behind the first
// plane, 2^-17 behind the second, with either sign), a bf16 value is one.  So
//   C[m][n] = sum_k A(m, k) B(n, k)
// is the sum of the products of such planes.  The planes i, j with i + j < 3 are
// kept for float32 results: what is left out is at most 2^-24 (1 + 2^-10) of a
// product, of either sign.  i + j < 2 with two planes are kept for results that
// are rounded to bf16: 2^-17 for the rounding of each operand's second plane and
// 2^-16 left out, 2^-15 of a product in all.  (Planes cut off instead of rounded
// left out up to 2^-21 and 2^-14, always towards 0.)  Three matrix instructions
// of 16 clocks in the place of the eight of 32 that float32 operands take
// (v_mfma_f32_16x16x4_f32).
//
// 128 x BN tile per block of four waves (2 x 2), two blocks per CU, steps of 32
// along k through two LDS slots; two steps are on their way while one is
// multiplied, and are split into planes as they go into LDS (vector work of one
// block beside the products of the other).  An operand lies with k adjacent
// (KADJ: rows of k) or with k as its row index (a thread then takes eight rows
// of one column; neighbouring threads neighbouring columns).
constexpr int RB_BM = 128, RB_KS = 32;

// An operand in LDS: planes of 64-byte rows.  Chunk c (16 bytes) of row r
// stands at place c ^ ((r >> 1) + (r >> 3 & 1)) & 3: 16 lanes reading one chunk of
// 16 rows, and 8 lanes writing one chunk of 8 rows, touch every bank once.
DEV int rb_swz(int r) { return (r >> 1) + ((r >> 3) & 1); }
DEV uint8_t *rb_place(uint8_t *lds, int r, int c) {
  return lds + r * 64 + ((c ^ rb_swz(r)) & 3) * 16;
}

// W values -> planes of W bf16 (W / 2 words each).  A value that rounds to
// infinity leaves planes whose sums are not finite; those are taken again.
template <int P, int W> DEV void split(const float *f, uint32_t (&o)[P][W / 2]) {
  float r[W];
#pragma unroll
  for (int i = 0; i < W; ++i) r[i] = f[i];
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int i = 0; i < W / 2; ++i) {
      o[p][i] = cvt_pk_bf16(r[2 * i], r[2 * i + 1]);
      if (p + 1 < P) {
        r[2 * i] -= __uint_as_float(o[p][i] << 16);
        r[2 * i + 1] -= __uint_as_float(o[p][i] & 0xFFFF0000u);
      }
    }
}

// One operand of a block: R rows (m or n) from r0 on.  Thread items, IT per
// thread: with k adjacent a row and 4 values of k (8 threads ask for a whole
// 128-byte piece of a row); with k as the row index a row (bf16: a pair of
// rows) and 8 values of k.  load() only asks memory (addresses held inside the
// operand, no condition on a value); what lies outside or is masked becomes 0
// in store(), which asks only where a step is not whole.  Two steps are on
// their way at once (Step).  VEC: k adjacent, rows at multiples of 16 bytes,
// k1 a multiple of 4.
template <typename T, int R, bool KADJ, bool VEC> struct Operand {
  static constexpr bool PAIR = !KADJ && sizeof(T) == 2;
  static constexpr int W = KADJ ? 4 : 8;   // values of an item
  static constexpr int IT = R * RB_KS / W / 256 / (PAIR ? 2 : 1), RI = R / (PAIR ? 2 : 1);
  const T *p;           // [rows][ld] (KADJ) or [k][ld]
  size_t ld;
  int rows, r0, k1;     // values of k at k1 and behind are 0
  const uint8_t *von;   // mask over k (not KADJ) or over the rows (KADJ), or null
  const T *at[IT];      // KADJ: the rows
  bool row_on[IT];      // and whether they take part
  uint32_t off[IT][8];  // not KADJ: byte offsets of the 8 values from row k0 of a step

  struct Step {         // [k0, k0 + 32)
    int k0;
    float v[IT][W];     // (PAIR: the bits of two bf16 columns)
    uint8_t on[IT][W];  // not KADJ: masks
  };

  DEV int row(int i) const {
    return KADJ ? (threadIdx.x >> 3) + 32 * i : (threadIdx.x + 256 * i) % RI * (PAIR ? 2 : 1);
  }
  DEV int chunk(int i) const {   // k / W; not KADJ: the same in a whole wave
    return KADJ ? threadIdx.x & 7 : __builtin_amdgcn_readfirstlane((threadIdx.x + 256 * i) / RI);
  }
  DEV void init() {
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      if constexpr (KADJ) {
        const int r = min(r0 + row(i), rows - 1);
        at[i] = p + (size_t)r * ld;
        row_on[i] = r0 + row(i) < rows && (!von || von[r]);
      } else {
        // (PAIR: rows and ld are even, the pair is one aligned word)
        const uint32_t r = min(r0 + row(i), rows - (PAIR ? 2 : 1));
#pragma unroll
        for (int u = 0; u < 8; ++u)
          off[i][u] = ((8 * chunk(i) + u) * (uint32_t)ld + r) * (uint32_t)sizeof(T);
      }
    }
  }
  DEV void load(Step &S, int k0) const {
    S.k0 = k0;
    if constexpr (!KADJ) {
      if (von) {
#pragma unroll
        for (int i = 0; i < IT; ++i)
#pragma unroll
          for (int u = 0; u < 8; ++u) S.on[i][u] = von[min(k0 + 8 * chunk(i) + u, k1 - 1)];
      }
      const char *base = reinterpret_cast<const char *>(p + (size_t)min(k0, k1 - 1) * ld);
      // the last step may end early: its rows behind the end are the last row
      const uint32_t most = (uint32_t)max(k1 - 1 - k0, 0), rb = (uint32_t)(ld * sizeof(T));
      const bool cut = most < RB_KS - 1;
#pragma unroll
      for (int i = 0; i < IT; ++i)
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          uint32_t o = off[i][u];
          if (cut) {
            const uint32_t q = 8 * chunk(i) + u;
            o -= (q - min(q, most)) * rb;
          }
          S.v[i][u] = *reinterpret_cast<const float *>(base + (size_t)o);
        }
    } else {
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        static_assert(!KADJ || sizeof(T) == 4, "float32 rows");
        const int k = k0 + W * chunk(i);
        if constexpr (VEC) {
          const float4 a = *reinterpret_cast<const float4 *>(at[i] + min(k, k1 - 4));
          S.v[i][0] = a.x; S.v[i][1] = a.y; S.v[i][2] = a.z; S.v[i][3] = a.w;
        } else {
#pragma unroll
          for (int u = 0; u < W; ++u) S.v[i][u] = at[i][min(k + u, k1 - 1)];
        }
      }
    }
  }
  // the value of row r (held inside the operand) at k < k1, as a float
  DEV float value(int r, int k) const {
    r = min(r, rows - 1);
    return Elem<T>::ld(p, KADJ ? (size_t)r * ld + k : (size_t)k * ld + r);
  }
  // whether the mask leaves it
  DEV bool takes_part(int r, int k) const { return !von || von[KADJ ? min(r, rows - 1) : k]; }
  // sum: the items' values added up
  template <int P> DEV void store(Step &S, uint8_t *lds, float *sum = nullptr) const {
    if (S.k0 + RB_KS > k1 || r0 + R > rows || von) {   // not all of the step takes part
#pragma unroll
      for (int i = 0; i < IT; ++i)
#pragma unroll
        for (int u = 0; u < W; ++u) {
          bool ok = S.k0 + W * chunk(i) + u < k1;
          if constexpr (KADJ) ok = ok && row_on[i];
          else ok = ok && r0 + row(i) < rows && (!von || S.on[i][u]);
          S.v[i][u] = ok ? S.v[i][u] : 0.f;
        }
    }
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      if constexpr (PAIR) {
        static_assert(P == 1, "a bf16 value is one plane");
        uint32_t lo[4], hi[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t x = __float_as_uint(S.v[i][2 * j]), y = __float_as_uint(S.v[i][2 * j + 1]);
          lo[j] = __builtin_amdgcn_perm(y, x, 0x05040100u);
          hi[j] = __builtin_amdgcn_perm(y, x, 0x07060302u);
        }
        // (even columns in the first half of the rows, odd ones in the second)
        *reinterpret_cast<uint4 *>(rb_place(lds, row(i) / 2, chunk(i))) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        *reinterpret_cast<uint4 *>(rb_place(lds, row(i) / 2 + R / 2, chunk(i))) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      } else {
        if (sum) {
#pragma unroll
          for (int u = 0; u < W; ++u) sum[i] += S.v[i][u];
        }
        uint32_t o[P][W / 2];
        split<P, W>(S.v[i], o);
#pragma unroll
        for (int q = 0; q < P; ++q) {
          uint8_t *pl = lds + q * R * 64;
          if constexpr (KADJ)
            *reinterpret_cast<uint2 *>(rb_place(pl, row(i), chunk(i) >> 1) + 8 * (chunk(i) & 1)) =
                make_uint2(o[q][0], o[q][1]);
          else
            *reinterpret_cast<uint4 *>(rb_place(pl, row(i), chunk(i))) =
                make_uint4(o[q][0], o[q][1], o[q][2], o[q][3]);
        }
      }
    }
  }
};

struct RouterGemmArgs {
  const void *a; size_t lda; const float *b; size_t ldb;
  int M, N, K, klen;                     // klen: k per blockIdx.y
  const uint8_t *von;
  const void *add;                       // ADD: [M][N] or null
  void *out;                             // [M][N], or partials [z][M][N] f32
  float *colsum;                         // [z][N]: sums of B over k (blocks of the first rows), or null
};

template <typename TA, typename TC, int BN, bool KADJ, bool VEC, int PA, int PB>
__global__ __launch_bounds__(256, 2) void router_gemm_kernel(RouterGemmArgs G) {
  constexpr int PM = PA > PB ? PA : PB, NF = BN / 32;
  constexpr int SLOT = (PA * RB_BM + PB * BN) * 64;
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * SLOT];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, lr = lane & 15, lg = lane >> 4;
  const int wm = w & 1, wn = w >> 1;
  const int nx = (G.N + BN - 1) / BN, by = blockIdx.x / nx;   // column tiles of a row tile in turn
  const int m0 = by * RB_BM, n0 = (blockIdx.x - by * nx) * BN;
  const int kb = blockIdx.y * G.klen, ke = min(G.K, kb + G.klen);
  using OA = Operand<TA, RB_BM, KADJ, VEC>;
  using OB = Operand<float, BN, KADJ, VEC>;
  OA A;
  A.p = (const TA *)G.a; A.ld = G.lda; A.rows = G.M; A.r0 = m0; A.k1 = ke; A.von = G.von;
  OB B;
  B.p = G.b; B.ld = G.ldb; B.rows = G.N; B.r0 = n0; B.k1 = ke; B.von = KADJ ? nullptr : G.von;
  A.init();
  B.init();
  f32x4_t acc[4][NF] = {};
  float cs[OB::IT] = {};
  const int get = lr * 64 + ((lg ^ rb_swz(lr)) & 3) * 16;
  // one step from slot g: its values into LDS, the step after the next one
  // asked for, then the products
  auto step = [&](typename OA::Step &SA, typename OB::Step &SB, int k, int g) {
    uint8_t *slot = lds + g * SLOT, *sb = slot + PA * RB_BM * 64;
    A.template store<PA>(SA, slot);
    B.template store<PB>(SB, sb, KADJ ? nullptr : cs);
    __builtin_amdgcn_sched_barrier(0);
    // (behind the end too, from addresses inside: a load that may not happen
    // would make the compiler wait for every load in flight)
    A.load(SA, k + 2 * RB_KS);
    B.load(SB, k + 2 * RB_KS);
    __builtin_amdgcn_s_waitcnt(0xC07F);   // (LDS only: the loads stay in flight)
    block_barrier();
    uint4 av[PA][4];
#pragma unroll
    for (int p = 0; p < PA; ++p)
#pragma unroll
      for (int m = 0; m < 4; ++m)
        av[p][m] = *reinterpret_cast<const uint4 *>(slot + (p * RB_BM + 64 * wm + 16 * m) * 64 + get);
    // B's fragments are read two ahead of their products (left alone, the
    // scheduler reads each one right before its use and waits)
    uint4 bv[3];
    auto read_b = [&](int s) {
      bv[s % 3] = *reinterpret_cast<const uint4 *>(
          sb + (s / NF * BN + (BN / 2) * wn + 16 * (s % NF)) * 64 + get);
    };
    read_b(0);
    read_b(1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = 0; s < PB * NF; ++s) {
      if (s + 2 < PB * NF) read_b(s + 2);
#pragma unroll
      for (int q = 0; q < PA; ++q)
        if (s / NF + q < PM) {
#pragma unroll
          for (int m = 0; m < 4; ++m)
            acc[m][s % NF] = mfma32(bv[s % 3], av[q][m], acc[m][s % NF]);
        }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  typename OA::Step a0, a1;
  typename OB::Step b0, b1;
  A.load(a0, kb);
  B.load(b0, kb);
  __builtin_amdgcn_sched_barrier(0);   // (in this order, so that the first step waits for itself only)
  A.load(a1, kb + RB_KS);
  B.load(b1, kb + RB_KS);
  __builtin_amdgcn_sched_barrier(0);
  for (int k = kb; k < ke; k += 2 * RB_KS) {
    step(a0, b0, k, 0);
    if (k + RB_KS < ke) step(a1, b1, k + RB_KS, 1);
  }
  // a lane has columns n0 + .. + 4 lg + 0..3 of row lr of each fragment
  TC *out = (TC *)G.out + (size_t)blockIdx.y * G.M * G.N;
  const TC *add = (const TC *)G.add;
  const bool vec = G.N % 4 == 0 && (((uintptr_t)out | (uintptr_t)add) & (4 * sizeof(TC) - 1)) == 0;
  auto row_of = [&](int m) {   // see Operand for pairs
    const int rl = 16 * m + lr;
    return m0 + (OA::PAIR ? 2 * rl + wm : 64 * wm + rl);
  };
  auto col_of = [&](int n) { return n0 + (BN / 2) * wn + 16 * n + 4 * lg; };
  // Planes do not carry what is not finite: an infinity (or a value that rounds to
  // one) leaves NaN in its lower planes and meets zeros in the other operand's, and
  // a first plane's product may pass the largest number.  Sums that are not finite are
  // taken again from the values, in float32, by the waves that have any (a row
  // that does not take part has no terms).  Nothing where all is finite; with a
  // whole row of x NaN, 8192 x 2048 x 460 takes 3.9 ms in the place of 0.25.
  bool odd = false;
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int n = 0; n < NF; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) odd |= !(fabsf(acc[m][n][i]) < INFINITY);
  if (__any(odd)) {
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      float s[NF][4] = {};
#pragma unroll 1
      for (int k = kb; k < ke; ++k) {
        const bool on = A.takes_part(row_of(m), k);
        const float a = A.value(row_of(m), k);
#pragma unroll
        for (int n = 0; n < NF; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float t = fmaf(a, B.value(col_of(n) + i, k), s[n][i]);
            s[n][i] = on ? t : s[n][i];
          }
      }
#pragma unroll
      for (int n = 0; n < NF; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!(fabsf(acc[m][n][i]) < INFINITY)) acc[m][n][i] = s[n][i];
    }
  }
  if (add) {   // every load in flight before the first sum
    TC old[4][NF][4];
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int n = 0; n < NF; ++n) {
        const TC *q = add + (size_t)min(row_of(m), G.M - 1) * G.N;
        if (vec) {   // (N is a multiple of 4: the four columns are there, or the last four)
          const int c = min(col_of(n), G.N - 4);
          if constexpr (sizeof(TC) == 2)
            *reinterpret_cast<uint2 *>(old[m][n]) = *reinterpret_cast<const uint2 *>(q + c);
          else
            *reinterpret_cast<float4 *>(old[m][n]) = *reinterpret_cast<const float4 *>(q + c);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) old[m][n][i] = q[min(col_of(n) + i, G.N - 1)];
        }
      }
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int n = 0; n < NF; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][n][i] += Elem<TC>::ld(old[m][n], i);
  }
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const int r = row_of(m);
    if (r >= G.M) continue;
#pragma unroll
    for (int n = 0; n < NF; ++n) {
      const int c = col_of(n);
      TC *q = out + (size_t)r * G.N + c;
      if (c >= G.N) continue;
      const f32x4_t v = acc[m][n];
      if (vec) {
        if constexpr (sizeof(TC) == 2)
          *reinterpret_cast<uint2 *>(q) = make_uint2(cvt_pk_bf16(v[0], v[1]), cvt_pk_bf16(v[2], v[3]));
        else
          *reinterpret_cast<float4 *>(q) = make_float4(v[0], v[1], v[2], v[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (c + i < G.N) {
            if constexpr (sizeof(TC) == 2) q[i] = (uint16_t)cvt_pk_bf16(v[i], v[i]);
            else q[i] = v[i];
          }
      }
    }
  }
  if constexpr (!KADJ) {
    if (G.colsum && by == 0) {   // the threads of a column, in order
      float *red = reinterpret_cast<float *>(lds);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < OB::IT; ++i) red[B.chunk(i) * BN + B.row(i)] = cs[i];
      __syncthreads();
      if (tid < BN && n0 + tid < G.N) {
        float s = 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q) s += red[q * BN + tid];
        G.colsum[(size_t)blockIdx.y * G.N + n0 + tid] = s;
      }
    }
  }
}

// out[i] = sum_z part[z][i] (z ascending) for the weight gradient (n values)
// and the bias gradient (E values; null without one)
__global__ __launch_bounds__(256) void router_sum_kernel(const float *__restrict__ part,
                                                         const float *__restrict__ cpart, int z,
                                                         size_t n, int E, float *__restrict__ out,
                                                         float *__restrict__ db) {
  const size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i < n) {
    if (n % 4 == 0 && ((uintptr_t)out & 15) == 0) {
      float4 s = *reinterpret_cast<const float4 *>(part + i);
      for (int q = 1; q < z; ++q) {
        const float4 v = *reinterpret_cast<const float4 *>(part + q * n + i);
        s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
      }
      *reinterpret_cast<float4 *>(out + i) = s;
    } else {
      for (size_t j = i; j < n && j < i + 4; ++j) {
        float s = part[j];
        for (int q = 1; q < z; ++q) s += part[q * n + j];
        out[j] = s;
      }
    }
  }
  const int e = blockIdx.x * 256 + threadIdx.x;
  if (db && e < E) {
    float s = cpart[e];
    for (int q = 1; q < z; ++q) s += cpart[(size_t)q * E + e];
    db[e] = s;
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

// The weight gradient's sum over tokens is split so that its tiles fill the
// chip (two blocks per CU), each part at least 256 tokens.
struct RouterSplit { int bn, z, klen; };
static RouterSplit router_split(int T, int d, int E) {
  RouterSplit S;
  S.bn = E <= 64 ? 64 : 128;
  const int tiles = ceil_div_h(d, RB_BM) * ceil_div_h(E, S.bn);
  const int z = std::max(1, std::min(512 / tiles, ceil_div_h(T, 256)));
  S.klen = ceil_div_h(ceil_div_h(T, z), RB_KS) * RB_KS;
  S.z = ceil_div_h(T, S.klen);
  return S;
}

size_t router_bwd_ws_bytes(int T, int d, int E) {
  const RouterSplit S = router_split(T, d, E);
  return S.z > 1 ? (size_t)S.z * ((size_t)d * E + E) * 4 + 16 : 0;
}

template <typename TX> static void router_bwd(const void *x, const float *w, const uint8_t *valid,
                                              const float *dl, const void *dx_in, int T, int d,
                                              int E, void *dx, float *dw, float *db, void *ws,
                                              hipStream_t st) {
  constexpr bool f32 = sizeof(TX) == 4;
  if (dx) {
    RouterGemmArgs G{dl, (size_t)E, w, (size_t)E, T, d, E, ceil_div_h(E, RB_KS) * RB_KS, valid,
                     dx_in, dx, nullptr};
    const unsigned grid = (unsigned)ceil_div_h(d, 128) * ceil_div_h(T, RB_BM);
    constexpr int P = f32 ? 3 : 2;
    if (E % 4 == 0 && (((uintptr_t)dl | (uintptr_t)w) & 15) == 0)
      router_gemm_kernel<float, TX, 128, true, true, P, P><<<grid, 256, 0, st>>>(G);
    else
      router_gemm_kernel<float, TX, 128, true, false, P, P><<<grid, 256, 0, st>>>(G);
  }
  if (dw) {
    const RouterSplit S = router_split(T, d, E);
    const size_t n = (size_t)d * E;
    float *part = S.z > 1 ? (float *)ws : dw;
    float *cpart = S.z > 1 ? (float *)ws + ((S.z * n + 3) & ~size_t(3)) : db;
    RouterGemmArgs G{x, (size_t)d, dl, (size_t)E, d, E, T, S.klen, valid, nullptr, part,
                     db ? cpart : nullptr};
    const dim3 grid(ceil_div_h(E, S.bn) * ceil_div_h(d, RB_BM), S.z);
    constexpr int PX = f32 ? 3 : 1;
    if (S.bn == 64) router_gemm_kernel<TX, float, 64, false, false, PX, 3><<<grid, 256, 0, st>>>(G);
    else router_gemm_kernel<TX, float, 128, false, false, PX, 3><<<grid, 256, 0, st>>>(G);
    if (S.z > 1)
      router_sum_kernel<<<(unsigned)((n + 1023) / 1024 + (E + 255) / 256), 256, 0, st>>>(
          part, cpart, S.z, n, E, dw, db);
  } else if (db) {
    colsum_kernel<<<(E + 63) / 64, 1024, 0, st>>>(dl, valid, T, E, db);
  }
}

void launch_router_bwd(bool bf16, const void *x, const float *w, const uint8_t *valid,
                       const float *dl, const void *dx_in, int T, int d, int E, void *dx,
                       float *dw, float *db, void *ws, hipStream_t st) {
  if (bf16) router_bwd<bf16_t>(x, w, valid, dl, dx_in, T, d, E, dx, dw, db, ws, st);
  else router_bwd<float>(x, w, valid, dl, dx_in, T, d, E, dx, dw, db, ws, st);
}

}  // namespace moe
