// Product of int8 rows with int8 matrices (one, or one per expert), a float32
// scale per row and per output channel:
//   out[p][n] = a_scale[r] w_scale[e][n] sum_k a[r][k] w[e][n][k],
//   r = row_src ? row_src[p] / row_div : p,  offsets[e] <= p < offsets[e+1].
// The sums are exact in int32 (K <= 65536); the two scales are applied in
// float32 and the result is rounded once to the output type.
//
// Two kernels: a small launch asks for its matrices at once (short), any other
// one runs row tiles of 32, 64, 128 or 256 through LDS (tiled).  The number of
// rows of an expert is on the device only, so each block finds its tile from
// the offsets itself: one launch per product, no list to build.
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "kernels.h"
#include "mfma.h"

namespace moe {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

// D = A(16x64) B(64x16) + C in int32: lane l holds A row l%16 / B column l%16
// with 16 consecutive K bytes of lane group l/16; D lane l holds column l%16,
// rows 4 (l/16) .. + 3.  The products run with the matrix w as A and the rows
// as B, so that a lane ends with 4 adjacent output channels of one row.
DEV i32x4_t mfma_i8(uint4 a, uint4 b, i32x4_t c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, a),
                                               __builtin_bit_cast(i32x4_t, b), c, 0, 0, 0);
}

// Inclusive sum over the lanes of a wave (DPP: within rows of 16, then the
// row totals passed on).
DEV int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);   // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);   // row_shr:2
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);   // row_shr:4
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);   // row_shr:8
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);   // row_bcast:15
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);   // row_bcast:31
  return v;
}

// The list of row tiles, ceil(rows / BM) for every expert, as a wave holds it:
// lane l has the experts l, l + 64, .. (E <= 64 NC; offsets held inside
// [0, M], loads coalesced and all in flight at once), and the list runs over
// the lanes.  One scan over the lanes' sums finds the lane of a tile, whose
// experts are then walked.  The whole wave asks for the same tile.
// NC = 1 for up to 64 experts (8 matrices of 1536 x 2048 by 64 rows: 7.4 us, 8.8
// with NC = 16), 16 for more (65 to 128 experts with NC = 2: 1 to 3 % less).
struct RowTile { int e, p0, end; };
template <int BM, int NC> struct TileList {
  int lo[NC], hi[NC], sum, upto, M;
  bool all;   // one matrix for every row

  DEV TileList(const int32_t *offsets, int E, int M_) : M(M_), all(!offsets) {
    if (all) return;
    // (opaque: nothing of this is kept in registers for the next search)
    const int lane = (int)opaque(threadIdx.x & 63);
    sum = 0;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      lo[i] = offsets[(unsigned)min(64 * i + lane, E)];
      hi[i] = offsets[(unsigned)min(64 * i + lane + 1, E)];
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      lo[i] = min(max(lo[i], 0), M);
      hi[i] = min(max(hi[i], lo[i]), M);
      sum += (hi[i] - lo[i] + BM - 1) / BM;   // (0 behind the last expert)
    }
    upto = wave_scan(sum);
  }
  DEV int count() const {
    return all ? (M + BM - 1) / BM : __builtin_amdgcn_readlane(upto, 63);
  }
  // tile t (false: there are fewer)
  DEV bool get(int t, RowTile &R) const {
    if (all) {
      R = RowTile{0, t * BM, M};
      return t * BM < M;
    }
    const int src = __popcll(__ballot(upto <= t));   // lanes whose tiles end before t
    if (src >= 64) return false;
    int left = t - __builtin_amdgcn_readlane(upto - sum, src);
    bool found = false;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int l = __builtin_amdgcn_readlane(lo[i], src);
      const int h = __builtin_amdgcn_readlane(hi[i], src);
      const int n = (h - l + BM - 1) / BM;
      if (!found && left < n) {
        found = true;
        R = RowTile{64 * i + src, l + BM * left, h};
      }
      left -= n;
    }
    return found;
  }
};

// The rows of a that the N rows p[..] of the product read (kept inside a).  The
// lookups are all in flight at once: no load depends on a condition.
template <int N> DEV void source_rows(const LinearI8Args &A, const int (&p)[N], int (&r)[N]) {
  const int32_t *src = A.row_src ? A.row_src : reinterpret_cast<const int32_t *>(A.a_scale);
  int raw[N];
#pragma unroll
  for (int i = 0; i < N; ++i) raw[i] = src[A.row_src ? p[i] : 0];
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < N; ++i)
    r[i] = min(max(A.row_src ? raw[i] / A.row_div : p[i], 0), A.a_rows - 1);
}
DEV int source_row(const LinearI8Args &A, int p) {
  const int q[1] = {p};
  int r[1];
  source_rows(A, q, r);
  return r[0];
}

DEV uint4 ld16(const int8_t *p) { return *reinterpret_cast<const uint4 *>(p); }

template <typename T> DEV void put4(T *p, bool vec, int n, int N, const float *v) {
  if (vec && n + 3 < N) {
    if constexpr (sizeof(T) == 2)
      *reinterpret_cast<uint2 *>(p) = make_uint2(cvt_pk_bf16(v[0], v[1]), cvt_pk_bf16(v[2], v[3]));
    else
      *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (n + i < N) {
      if constexpr (sizeof(T) == 2) p[i] = (uint16_t)cvt_pk_bf16(v[i], v[i]);
      else p[i] = v[i];
    }
  }
}

// ---- the short kernel, for small launches (a few rows by one matrix): bound by
// latency, so every byte of the matrices is asked for at once (8 us for 16 rows
// by 2048 x 2048, most of it the launch).
//
// A block takes a tile of up to 16 rows and `per` fragments of 16 output
// channels.  The rows go into LDS once, in the order in which the matrix
// instructions read them (step s of 64: 1 KB, lane after lane; rows too long
// for that are read from memory each time).  The four waves split the steps
// (wave w takes steps w, w + 4, ..) and read the matrix straight into
// registers, SH_D steps ahead and across fragments (four in the place of eight:
// no difference, K = 256 .. 1024); their sums are added through LDS.
constexpr int SH_BM = 16, SH_WAVES = 4, SH_D = 8;

template <typename T, int NC, bool ALDS>
__global__ __launch_bounds__(64 * SH_WAVES) void linear_i8_short_kernel(LinearI8Args A, int per) {
  constexpr int KS = SH_WAVES, D = SH_D;
  extern __shared__ __attribute__((aligned(16))) int8_t lds_a[];
  __shared__ __attribute__((aligned(16))) int red[KS * 256];
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int steps = (A.K + 63) >> 6, nfr = (A.N + 15) >> 4;
  const int ns = (steps - w + KS - 1) / KS, groups = (ns + D - 1) / D;
  const int f0 = blockIdx.x * per, cnt = min(per, nfr - f0);
  const int ldw = (int)A.ldw;
  const bool vec = (((uintptr_t)A.out & (4 * sizeof(T) - 1)) | (A.ldo & 3)) == 0;

  RowTile R;
  for (int t = blockIdx.y; TileList<SH_BM, NC>(A.offsets, A.E, A.M).get(t, R); t += gridDim.y) {
    const int8_t *we = A.w + (size_t)R.e * A.N * A.ldw;
    // steps D g .. D g + D - 1 of this wave's fragment i (the last one again
    // behind the end: read twice, not used)
    uint4 ring[D];
    auto column = [&](int i) { return we + (size_t)min(16 * (f0 + i) + lr, A.N - 1) * A.ldw; };
    auto at_step = [&](int s) { return min(64 * (w + KS * min(s, ns - 1)) + 16 * lg, ldw - 16); };
    if (ns > 0) {
      const int8_t *c = column(0);
#pragma unroll
      for (int j = 0; j < D; ++j) ring[j] = ld16(c + at_step(j));
    }
    const int row = source_row(A, min(R.p0 + lr, R.end - 1));
    const int8_t *ap = A.a + (size_t)row * A.lda + 16 * lg;
    const float sa = A.a_scale[row];
    if constexpr (ALDS) {
      // (what stands in the places of rows behind the end reaches only those
      // rows' sums, which are not stored)
      for (int s = w; s < steps; s += KS)
        if (R.p0 + lr < R.end)
          *reinterpret_cast<uint4 *>(lds_a + (s * 64 + lane) * 16) = ld16(ap + 64 * s);
      __syncthreads();
    }
    for (int i = 0; i < cnt; ++i) {
      // the channels' scales, asked for before the next steps of the matrix
      const int n = 16 * (f0 + i) + 4 * lg;
      const float *ws = A.w_scale ? A.w_scale + (size_t)R.e * A.N : A.a_scale;
      float sw[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) sw[c] = ws[A.w_scale ? min(n + c, A.N - 1) : 0];
      i32x4_t acc = {};
      auto group = [&](int g, auto prefetch) {
        constexpr bool PF = decltype(prefetch)::value;
        const bool wrap = g + 1 == groups;
        const int8_t *nc = PF ? column(wrap ? i + 1 : i) : nullptr;
        const int ng = wrap ? 0 : g + 1;
#pragma unroll
        for (int j = 0; j < D; ++j) {
          const int s = g * D + j;
          if (s < ns) {
            const int sk = w + KS * s;
            uint4 av;
            if constexpr (ALDS) av = *reinterpret_cast<const uint4 *>(lds_a + (sk * 64 + lane) * 16);
            else av = ld16(ap + 64 * sk);
            acc = mfma_i8(ring[j], av, acc);
          }
          if constexpr (PF) ring[j] = ld16(nc + at_step(ng * D + j));
        }
      };
      for (int g = 0; g < groups; ++g) {
        if (g + 1 < groups || i + 1 < cnt) group(g, std::true_type{});
        else group(g, std::false_type{});
      }
      i32x4_t *rv = reinterpret_cast<i32x4_t *>(red);
      rv[w * 64 + lane] = acc;
      __syncthreads();
      if (w == 0) {
#pragma unroll
        for (int o = 1; o < KS; ++o) acc += rv[o * 64 + lane];
        const int p = R.p0 + lr;
        if (p < R.end && n < A.N) {
          float v[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) v[c] = (float)acc[c] * (sa * (A.w_scale ? sw[c] : 1.0f));
          put4<T>((T *)A.out + (size_t)p * A.ldo + n, vec, n, A.N, v);
        }
      }
      __syncthreads();   // the sums (and the rows) are read before the next ones are written
    }
  }
}

// at most one tile more than M / 16 per expert, and none without a row
static int short_tiles(const LinearI8Args &A) {
  return A.offsets ? std::min(A.M, A.M / SH_BM + A.E) : (A.M + SH_BM - 1) / SH_BM;
}

template <typename T> static void launch_short(const LinearI8Args &A, hipStream_t st) {
  const int steps = (A.K + 63) / 64, nfr = (A.N + 15) / 16, tiles = short_tiles(A);
  const size_t lds = (size_t)SH_BM * steps * 64;
  const bool alds = lds <= 128 * 1024;
  // about four blocks per CU: more of them pay for their set-up, fewer leave
  // the memory system idle
  const int per = (int)std::min<int64_t>(nfr, ((int64_t)nfr * tiles + 1023) / 1024);
  const dim3 grid((nfr + per - 1) / per, std::min(tiles, 32768));
#define MOE_L(NC, AL) \
  linear_i8_short_kernel<T, NC, AL><<<grid, 64 * SH_WAVES, AL ? lds : 0, st>>>(A, per)
  if (!alds) MOE_L(16, false);
  else if (A.E > 64) MOE_L(16, true);
  else MOE_L(1, true);
#undef MOE_L
}

// ---- the tiled kernel: tiles of up to BM rows x 128 channels, four waves per
// block (2 x 2, each half of the rows in interleaved fragments of 16 and 64
// channels), steps of 128 along K, so that a row's share of a step is a whole
// 128-byte line (98304 rows by 460 matrices of 1536 x 2048: 658 us with half
// lines, 604 with whole ones).
//
// A step goes from memory into registers and from there into one LDS slot; the
// rows of the next step and the channels of the next two are on their way
// while a step is multiplied, and nothing in the loop waits for more than it
// needs (every load is unconditional and in the order of its use).  Two blocks
// per CU at 256 rows (three at 128, four below) take turns: the one that
// multiplies has priority, the other one writes LDS and waits (45 -> 41 us for
// 8192 x 2048 x 2048).  256 x 256 tiles of eight waves with two LDS slots and
// one block per CU were no faster (49 us where this then took 48).  MI: 16-row
// fragments a wave has (32 MI rows); a tile runs as the smallest class that
// holds its rows (548 -> 532 us for 98304 uneven rows by 460 matrices of 1536 x
// 2048 where the classes went in steps of 64 rows).
//
// What bounds it: a few rows a matrix, reading the matrices (64 matrices of
// 1408 x 2048 in 27 us, 6.8 TB/s); hundreds of rows, LDS traffic and the two
// barriers of a step (38 us for 8192 x 2048 x 2048, 1.8 POP/s, the matrix cores
// busy 0.35 of the time; 98304 unevenly spread rows by 460 matrices of 1536 x
// 2048 in 521 us, 1.2 POP/s, busy 0.30; of 2048 x 768, six steps a tile, in 365
// us, 0.85 POP/s, busy 0.21).
constexpr int TL_BM = 256, TL_BN = 128, TL_KS = 128;
// bytes of LDS for tiles of up to BM rows: channels, row and channel scales, rows
constexpr int TL_SCALES = TL_BN * TL_KS, TL_A = TL_SCALES + (TL_BM + TL_BN) * 4;
constexpr int tl_lds(int BM) { return TL_A + BM * TL_KS; }

// Rows of 128 bytes in LDS.  Chunk c (16 bytes) of row r stands at place
// c ^ (r >> 1) & 7 for the rows of a, whose fragments read 16 adjacent rows,
// and at c ^ (2 (r >> 3 & 3) + (r >> 1 & 1)) for the channels, whose fragments
// read the rows gt_col(f, 0..15): either way 16 lanes reading one chunk touch
// every bank once.  The places are the same for every fragment of a wave and
// every piece of a thread, so that all addresses are a base and a constant.
DEV int tl_swz_a(int r) { return (r >> 1) & 7; }
DEV int tl_swz_w(int r) { return ((r >> 2) & 6) | ((r >> 1) & 1); }

constexpr int kWaitLds = 0xC07F;   // s_waitcnt lgkmcnt(0), nothing else

template <typename T, int MI, typename Off>
DEV void row_tile(const LinearI8Args &A, const RowTile &R, int n0, uint8_t *lds) {
  const int tid = threadIdx.x, lane = tid & 63, lr = lane & 15, lg = lane >> 4;
  const int w = tid >> 6, wm = w & 1, wn = w >> 1;
  const int tr = tid >> 3, tc = tid & 7;     // row and chunk of this thread's first piece
  const int steps = (A.K + TL_KS - 1) / TL_KS;   // (rows of a hold 0 behind K)
  const int a_put = TL_A + tr * TL_KS + (tc ^ tl_swz_a(tr)) * 16;
  const int w_put = tr * TL_KS + (tc ^ tl_swz_w(tr)) * 16;
  const int ar = 16 * wm + lr, wr = 64 * wn + gt_col(0, lr);
  const int a_get = TL_A + ar * TL_KS + (lg ^ tl_swz_a(ar)) * 16;
  const int w_get = wr * TL_KS + (lg ^ tl_swz_w(wr)) * 16;
  // byte offsets inside the matrix, and inside a (from the tile's first row
  // on, where the rows are not looked up): 32 bits, or 64 (launch_linear)
  const int first = A.row_src ? 0 : R.p0;
  const int8_t *ab = A.a + (size_t)first * A.lda;
  const int8_t *we = A.w + (size_t)R.e * A.N * A.ldw;
  Off ao[MI], wo[4];
  int rows[MI + 1], from[MI + 1];   // this thread's pieces, and the row whose scale it fetches
#pragma unroll
  for (int i = 0; i < MI; ++i) rows[i] = min(R.p0 + tr + 32 * i, R.end - 1);
  rows[MI] = min(R.p0 + tid, R.end - 1);
  source_rows(A, rows, from);
#pragma unroll
  for (int i = 0; i < MI; ++i) ao[i] = (Off)(from[i] - first) * (Off)A.lda + 16 * tc;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    wo[i] = (Off)min(n0 + tr + 32 * i, A.N - 1) * (Off)A.ldw;
  // The rows of the next step and the channels of the next two are on their
  // way (the matrix comes from HBM, whose latency is longer than a step).
  uint4 sa_[MI], w0[4], w1[4];
  auto load_a = [&](int s) {
    const uint32_t k = TL_KS * min(s, steps - 1);
#pragma unroll
    for (int i = 0; i < MI; ++i) sa_[i] = ld16(ab + (size_t)(ao[i] + k));
  };
  auto load_w = [&](uint4 (&v)[4], int s) {
    const uint32_t k = (uint32_t)min(TL_KS * min(s, steps - 1) + 16 * tc, (int)A.ldw - 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = ld16(we + (size_t)(wo[i] + k));
  };
  auto store = [&](const uint4 (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4 *>(lds + w_put + 32 * TL_KS * i) = v[i];
#pragma unroll
    for (int i = 0; i < MI; ++i)
      *reinterpret_cast<uint4 *>(lds + a_put + 32 * TL_KS * i) = sa_[i];
  };
  i32x4_t acc[MI][4] = {};
  // One step.  Row fragment q (half h = q / MI of the step, chunks 4 h + lg)
  // is read two fragments before it is multiplied, the second half's channel
  // fragments as the first half's are used up; the scheduler keeps that order
  // (left alone, it reads each fragment right before its use and waits).
  auto multiply = [&]() {
    uint4 wv[4], av[3];
    auto read_w = [&](int h, int f) {
      wv[f] = *reinterpret_cast<const uint4 *>(lds + (w_get ^ (64 * h)) + TL_KS * gt_col(f, 0));
    };
    auto read_a = [&](int q) {
      av[q % 3] = *reinterpret_cast<const uint4 *>(
          lds + (a_get ^ (64 * (q / MI))) + 32 * TL_KS * (q % MI));
    };
#pragma unroll
    for (int f = 0; f < 4; ++f) read_w(0, f);
    read_a(0);
    read_a(1);
#pragma unroll
    for (int q = 0; q < 2 * MI; ++q) {
      if (q + 2 < 2 * MI) read_a(q + 2);
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        acc[q % MI][f] = mfma_i8(wv[f], av[q % 3], acc[q % MI][f]);
        if (q == MI - 1) {
          __builtin_amdgcn_sched_barrier(0);
          read_w(1, f);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // the tile's scales wait in LDS for its end (the first barrier shows them)
  float *scales = reinterpret_cast<float *>(lds + TL_SCALES);
  const float row_scale = A.a_scale[from[MI]];
  const float col_scale = (A.w_scale ? A.w_scale + (size_t)R.e * A.N : A.a_scale)[
      A.w_scale ? min(n0 + (tid & (TL_BN - 1)), A.N - 1) : 0];
  __builtin_amdgcn_sched_barrier(0);   // (loads in this order: the first step waits for itself only)
  load_w(w0, 0);
  load_a(0);
  __builtin_amdgcn_sched_barrier(0);
  load_w(w1, 1);
  __builtin_amdgcn_sched_barrier(0);
  scales[tid] = row_scale;
  if (tid < TL_BN) scales[TL_BM + tid] = A.w_scale ? col_scale : 1.0f;
  auto step = [&](uint4 (&v)[4], int j) {
    store(v);
    __builtin_amdgcn_sched_barrier(0);   // (the registers are free again)
    load_a(j + 1);
    __builtin_amdgcn_sched_barrier(0);   // (in this order: the rows are waited for first)
    load_w(v, j + 2);
    __builtin_amdgcn_s_waitcnt(kWaitLds);
    block_barrier();
    // (while this block multiplies, the other one of the CU should wait with
    // its products, not the other way round: they then take turns)
    __builtin_amdgcn_s_setprio(1);
    multiply();
    __builtin_amdgcn_s_setprio(0);
    block_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  for (int j = 0; j < steps; j += 2) {
    step(w0, j);
    if (j + 1 < steps) step(w1, j + 1);
  }
  const bool vec = (((uintptr_t)A.out & 15) | ((A.ldo * sizeof(T)) & 15)) == 0;
  f32x4_t sw[4];
#pragma unroll
  for (int f = 0; f < 4; ++f)
    sw[f] = *reinterpret_cast<const f32x4_t *>(scales + TL_BM + 64 * wn + gt_col(f, 4 * lg));
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int pl = 16 * (2 * i + wm) + lr, p = R.p0 + pl;
    if (p >= R.end) continue;
    const float sa = scales[pl];
    T *out = (T *)A.out + (size_t)p * A.ldo;
#pragma unroll
    for (int f = 0; f < 4; f += 2) {   // 8 adjacent channels
      const int n = n0 + 64 * wn + gt_col(f, 4 * lg);
      float v[8];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        v[c] = (float)acc[i][f][c] * (sa * sw[f][c]);
        v[4 + c] = (float)acc[i][f + 1][c] * (sa * sw[f + 1][c]);
      }
      if constexpr (sizeof(T) == 2) {
        if (vec && n + 7 < A.N) {
          *reinterpret_cast<uint4 *>(out + n) =
              make_uint4(cvt_pk_bf16(v[0], v[1]), cvt_pk_bf16(v[2], v[3]),
                         cvt_pk_bf16(v[4], v[5]), cvt_pk_bf16(v[6], v[7]));
          continue;
        }
      }
      put4<T>(out + n, vec, n, A.N, v);
      put4<T>(out + n + 4, vec, n + 4, A.N, v + 4);
    }
  }
}

// Blocks go round the 8 XCDs in turn; each XCD takes a contiguous run of the
// (row tile, channel tile) list, so that tiles that share rows and matrices
// share its L2.  The run is an eighth of the tiles there are, not of the grid.
// (Row tiles dealt out one by one to the XCDs: no difference.)
// (Blocks that take two or four channel tiles of a row tile in turn, the next
// one's channels on their way during the end of the last: what the shorter
// start saves, 418 -> 368 us for 98304 rows by 460 matrices of 2048 x 768, the
// registers held over that end cost again; one tile a block takes 365.)
template <typename T, int NC, int BM, typename Off>
__global__ __launch_bounds__(256, BM <= 64 ? 4 : BM == 128 && sizeof(Off) == 4 ? 3 : 2)
void linear_i8_tiled_kernel(LinearI8Args A) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[tl_lds(BM)];
  const int nt = (A.N + TL_BN - 1) / TL_BN;
  RowTile R;
  int n0;
  {
    const TileList<BM, NC> list(A.offsets, A.E, A.M);
    const int64_t items = (int64_t)list.count() * nt, run = (items + 7) / 8;
    const int64_t at = blockIdx.x >> 3, item = run * (blockIdx.x & 7) + at;
    if (at >= run || item >= items) return;
    const int t = (int)(item / nt);
    n0 = (int)(item - (int64_t)t * nt) * TL_BN;
    if (!list.get(t, R)) return;
  }
  const int rows = R.end - R.p0;
  if constexpr (BM <= 64) {
    row_tile<T, BM / 32, Off>(A, R, n0, lds);
  } else {
    if (rows <= 32) row_tile<T, 1, Off>(A, R, n0, lds);
    else if (rows <= 64) row_tile<T, 2, Off>(A, R, n0, lds);
    else if (rows <= 96) row_tile<T, 3, Off>(A, R, n0, lds);
    else if constexpr (BM == 128) row_tile<T, 4, Off>(A, R, n0, lds);
    else if (rows <= 128) row_tile<T, 4, Off>(A, R, n0, lds);
    else if (rows <= 160) row_tile<T, 5, Off>(A, R, n0, lds);
    else if (rows <= 192) row_tile<T, 6, Off>(A, R, n0, lds);
    else if (rows <= 224) row_tile<T, 7, Off>(A, R, n0, lds);
    else row_tile<T, 8, Off>(A, R, n0, lds);
  }
}

template <typename T, int BM, typename Off = uint32_t>
static void launch_tiled(const LinearI8Args &A, hipStream_t st) {
  const int64_t tiles = A.offsets ? A.M / BM + std::min(A.M, A.E) : (A.M + BM - 1) / BM;
  const int64_t items = tiles * ((A.N + TL_BN - 1) / TL_BN);
  const unsigned grid = (unsigned)((items + 7) / 8 * 8);
  if (A.E <= 64) linear_i8_tiled_kernel<T, 1, BM, Off><<<grid, 256, 0, st>>>(A);
  else linear_i8_tiled_kernel<T, 16, BM, Off><<<grid, 256, 0, st>>>(A);
}

// Which kernel, from the rows a matrix has on average (the host knows no more)
// and the work in tiles of 128 x 128 (times of uneven loads, log-normal with
// sigma 0.8):
//  - short where there are few fragments of 16 channels by 16 rows: 8.2 us
//    against 9.4 for 16 rows by 2048 x 2048, 13.6 against 11.5 for 12 rows of
//    12 experts (1152 fragments);
//  - 32-row tiles up to 8 rows a matrix: 124 us against 137 at 1 row by 460
//    matrices of 768 x 2048, 250 against 251 at 8 rows by 1536 x 2048, 267
//    against 265 at 12;
//  - 128-row tiles from three blocks a CU on, from one where they are full
//    (256 rows a matrix): against 64-row ones 62 us for 64 at 64 rows by 128
//    matrices of 2048 x 1024, 46 for 45 at 128 rows by 64 of 1408 x 2048; 19.5
//    for 21.0 at 256 rows by 8 of 2048 x 2048, 15.6 for 15.4 at 160;
//  - 256-row tiles where they have more than three rounds of work (two blocks
//    per CU) and most are whole: against 128-row ones 177 us for 187 at 768 rows by 64
//    matrices of 1408 x 2048, 131 for 127 at 512; 172 for 178 at 384 rows by 128
//    of 2048 x 1024, 101 for 97 at 160; 275 for 281 at 160 rows by 460 of 2048 x
//    768, 249 for 243 at 128.  With one matrix every tile is whole, and a round of
//    them is enough: 39 us against 44 for 8192 rows by 2048 x 2048, 25.7 against
//    22.9 for 4096.
// Past 2^32 bytes the offsets need 64 bits, and with them two blocks per CU the
// registers: 128-row tiles, 49 us against 44 for 8192 rows looked up by one
// matrix of 2048 x 2048, 157 against 160 for 24576 rows by 64 (the short kernel:
// 257 and 763).
template <typename T> static void launch_linear(const LinearI8Args &A, hipStream_t st) {
  const int avg = A.M / A.E;
  // 32-bit byte offsets inside one matrix, and inside a where rows are looked up
  const bool near = (uint64_t)A.N * A.ldw <= (1ull << 32) &&
                    (!A.row_src || (uint64_t)A.a_rows * A.lda <= (1ull << 32));
  const bool small = (int64_t)ceil_div_h(A.N, 16) * short_tiles(A) < 1024;
  const int64_t work = (int64_t)A.M * A.N / (128 * 128);
  const bool many = A.E == 1 ? (int64_t)ceil_div_h(A.M, TL_BM) * ceil_div_h(A.N, TL_BN) >= 512
                             : avg > 144 && work >= 3500;
  if (small) launch_short<T>(A, st);
  else if (!near) launch_tiled<T, 128, uint64_t>(A, st);
  else if (avg <= 8) launch_tiled<T, 32>(A, st);
  else if (many) launch_tiled<T, 256>(A, st);
  else if (work >= 768 || (avg >= 256 && work >= 256)) launch_tiled<T, 128>(A, st);
  else launch_tiled<T, 64>(A, st);
}

void launch_linear_i8(bool bf16, const LinearI8Args &A, hipStream_t st) {
  if (bf16) launch_linear<bf16_t>(A, st);
  else launch_linear<float>(A, st);
}

}  // namespace moe
