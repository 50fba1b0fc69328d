// HIP kernels of the operators on the whole next-token distribution (gfx950):
// the selected log-probability with entropy and top alternatives
// (linear_logp_top), and the divergence from a teacher's kept tokens
// (linear_distill).  Declared in include/rlk/vocab_ops.h.
//
// Forward:
//   distill_rows       which rows hold a teacher's token at all
//   gather_rows_fill   compacted hidden rows; the outputs of inactive rows
//   bucket_entries     the teacher's tokens of a row tile, sorted by vocabulary tile
//   logit_tiles        MFMA logit tiles -> chunk statistics, and the logits
//                      that the row kernels need (top: of a group of splits,
//                      distill: of the teacher's tokens)
//   top_merge          folds the statistics; the K best of a row
//   distill_merge      folds the statistics; the row's divergence
// Backward (per group of vocabulary splits, ascending):
//   gather_rows_grad   compacted hidden rows and the rows' coefficients
//   soft_dz_tiles      recomputed logits -> dz, bf16
//   distill_scatter    dz at the teacher's tokens
//   part_grad_tiles    grad_h in parts of the vocabulary, grad_W
//   grad_h_sum         the parts together (after the last group)
// Up to 128 rows (few_rows: the batch's rows in place, no compaction) other
// kernels give the same bits:
//   few_tiles          for logit_tiles and soft_dz_tiles
//   few_rows_grad      for gather_rows_grad (and the backward's distill_rows)
//   few_grad_h, few_grad_w   for part_grad_tiles
//
// Times below are of one MI355X (which copies at 4.9 TB/s, and whose library
// multiplies 8192^3 bf16 matrices at 1.53 PFLOP/s), V = 151936.
#pragma once

#include "rlk_kernels.h"

namespace rlk {
namespace vocab {

constexpr int kMaxK = 128;  // alternatives, or teacher's tokens, of a row

// Target of a row that has no dz (rowinfo of the few-row kernels).
constexpr int kNoRow = INT32_MIN;

// A product e^d * d is 0 where e^d is (d may be -inf there): d is cut off
// where e^d rounds to 0 in fp32 (e^-103.98 is half the least denormal).
constexpr float kDeepest = -104.f;

// ---------------------------------------------------------------------------
// Statistics with the first moment: m = max z, s = sum e(z - m),
// u = sum e(z - m) (z - m) <= 0.  The entropy is then log s - u / s, a sum of
// two terms >= 0.  m and s are the bits of ms_combine and chunk_stats.
// ---------------------------------------------------------------------------
struct MSU {
  float m, s, u;
};

__device__ __forceinline__ MSU msu_identity() { return {-INFINITY, 0.f, 0.f}; }

// a = lower vocabulary indices.  Moving a set from its max ma to m multiplies
// s by e(ma - m) and gives u' = e(ma - m) u + s' (ma - m).  Sums of sets without
// a max above -inf are 0 or NaN, as in ms_combine.
__device__ __forceinline__ MSU msu_combine(MSU a, MSU b) {
  const float m = fmaxf(a.m, b.m);
  if (m == -INFINITY) return {m, a.s + b.s, a.u + b.u};
  const float ea = rlk_exp(a.m - m), eb = rlk_exp(b.m - m);
  const float pa = a.s * ea, pb = b.s * eb;
  const float ua = a.u * ea + pa * fmaxf(a.m - m, kDeepest);
  const float ub = b.u * eb + pb * fmaxf(b.m - m, kDeepest);
  return {m, pa + pb, ua + ub};
}

// exp_tree with the first moment beside it (x: sum e, y: sum e d).
template <int N>
__device__ __forceinline__ float2 moment_tree(const float (&v)[kRowVals], int k0, float m) {
  if constexpr (N == 1) {
    const float d = v[k0] - m, e = rlk_exp(d);
    return make_float2(e, e * fmaxf(d, kDeepest));
  } else {
    const float2 l = moment_tree<N / 2>(v, k0, m);
    const float2 r = moment_tree<N / 2>(v, k0 + N / 2, m);
    return make_float2(l.x + r.x, l.y + r.y);
  }
}

__device__ __forceinline__ MSU chunk_stats_moment(const float (&v)[kRowVals]) {
  float mx = -INFINITY;
#pragma unroll
  for (int k = 0; k < kRowVals; ++k) mx = fmaxf(mx, v[k]);
  mx = row_max(mx);
  const float2 t = moment_tree<kRowVals>(v, 0, stats_shift(mx));
  return {mx, row_sum(t.x), row_sum(t.y)};
}

// ---------------------------------------------------------------------------
// Logits of a group of splits.  Tiles, statistics and target logit as in
// fwd_tiles; records at [chunk of the vocabulary][active row].
// kTop: also the first moment, and (z != NULL) every logit of the group: of
//   active row i, chunk j of the group's split sl, at
//   z + i * ldz + 128 (sl cps + j).
// !kTop: logits times `scale` (1 / temperature); the tile's entries (see
//   bucket_entries) pick the scaled logits of the teacher's tokens.
// Bound by the engine's MFMAs.  3482 active rows, H = 4096 (4.33 TFLOP): 2.91 -
// 3.02 ms (1.43 - 1.49 PFLOP/s) with 64 tokens of a teacher; with the first
// moment and every logit stored 3.38 - 3.46 ms, 0.35 of them for the 2.2 GB of
// stores (the accumulators leave no registers to pick the alternatives here).
// Stores that bypass the caches add 0.1 ms.
// At 129 to 512 rows each tile waits for its loads: 256 rows 0.31 ms, 257
// 0.40 (see gemm_rows).
// ---------------------------------------------------------------------------
struct LogitArgs {
  const uint16_t* hA;  // active rows of h, compacted, zero padded to a multiple of 256
  const uint16_t* W;
  const int32_t* n_act;
  int H;
  int cus;      // see tile_of_block
  int G;        // splits of this launch: [gm.s0, gm.s0 + G)
  SplitGeom gm;
  TileGeom tg;
  size_t rec_stride;
  float2* rec;
  // kTop
  const int32_t* yA;  // targets of the active rows
  float* zt;
  float* rec_u;
  float* z;
  int64_t ldz;
  // !kTop
  float scale;
  int K;
  const int32_t* ent_off;  // [row group][32 tps + 1]
  const uint32_t* ent;     // [row group][kBucketRows K]
  float* z_ids;            // [active row][K]
};

// Tile of block `bid` when n tiles run on `cus` compute units one at a time:
// whole tiles for whole rounds; the tiles of a last round that would leave
// half of the units idle are cut into their two 128-column halves (half = 0,
// 1; -1: whole), which take half as long.  At up to 256 rows of V = 151936
// that is 2.5 rounds instead of 3.  Waves of a half's other columns only load.
__device__ __forceinline__ bool tile_of_block(int n, int cus, int bid, int& id, int& half) {
  const int full = n / cus * cus, rest = n - full;
  const bool cut = 2 * rest <= cus;
  const int k = bid < full ? xcd_tile(full, bid) : xcd_tile(cut ? 2 * rest : rest, bid - full);
  if (k < 0) return false;
  const bool h = cut && bid >= full;
  id = __builtin_amdgcn_readfirstlane(bid < full ? k : full + (cut ? k >> 1 : k));
  half = __builtin_amdgcn_readfirstlane(h ? k & 1 : -1);
  return true;
}

// Row block b (kBlk rows) of a tile of logits or dz is block b / kWM of wave
// row b % kWM: the row blocks of a last, short row tile are spread over the
// SIMDs, and the waves leave out the others (gemm_rows).
__device__ __forceinline__ int spread_block(int wm, int mi) { return kWM * mi + wm; }
__device__ __forceinline__ int spread_row(int wm, int mi, int lane) { return kBlk * spread_block(wm, mi) + lane % kBlk; }

// rows_k in that order.  Rows past `last` repeat it: 257 rows of H = 4096 lose
// their second tile's other row blocks' MFMAs and, in L2, its 255 other rows
// (each alone gains 2 % or nothing, both 10: 0.44 -> 0.40 ms; 300 rows of H =
// 2048 by half of V 0.158 -> 0.136).  grad_h's tiles have no registers for it.
__device__ __forceinline__ RowsK rows_k_spread(const uint16_t* base, int last, int ld) {
  RowsK R;
  R.base = reinterpret_cast<const char*>(base);
#pragma unroll
  for (int i = 0; i < kDma; ++i) {
    const int row = dma_k_row(i), b = row / kBlk;
    const int at = min(kBlk * spread_block(b / kMI, b % kMI) + row % kBlk, last);
    R.off[i] = (uint32_t)(2 * ((size_t)at * ld + dma_k_seg(row) * 8));
  }
  return R;
}

// The tile product of a wave of which `rows` rows of the tile are wanted: the
// wave's blocks of them, up to a power of two.  Every element computed is the
// same MFMA chain.
template <class LA, class LB, class Tail>
__device__ __forceinline__ void gemm_rows(const LA& A, const LB& B, int nk, Acc& acc, u32x4* lds, int wm, int rows,
                                          const Tail& tail) {
  const int blocks = (rows + kBlk - 1) / kBlk, mine = max(0, (blocks - wm + kWM - 1) / kWM);
  if (mine == 0) {
    gemm256<false, false, 0>(A, B, nk, acc, lds, tail);
  } else if (mine == 1) {
    gemm256<false, false, 1>(A, B, nk, acc, lds, tail);
  } else if (mine == 2 && kMI > 2) {
    gemm256<false, false, kMI / 2>(A, B, nk, acc, lds, tail);
  } else {
    gemm256<false, false>(A, B, nk, acc, lds, tail);
  }
}

// Teacher's tokens are sorted in groups of kBucketRows rows (bucket_entries).
constexpr int kBucketRows = 32;
static_assert(kBM % kBucketRows == 0 && kBucketRows % kBlk == 0, "a row group is whole row blocks");

// An entry: column and row within the tile, slot of the row.
__device__ __forceinline__ uint32_t entry_of(int col, int row, int k) { return (uint32_t)(col | row << 8 | k << 16); }

template <bool kTop>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(RLK_WAVES / 4, RLK_WAVES / 4))) void logit_tiles(
    LogitArgs a) {
  __shared__ u32x4 lds[kLdsU4];
  const int n_act = __builtin_amdgcn_readfirstlane(*a.n_act);
  const int rtiles = (n_act + kBM - 1) / kBM;
  const int C = a.G * a.tg.tps;
  int id, half;
  if (!tile_of_block(rtiles * C, a.cus, blockIdx.x, id, half)) return;
  int rt, ct;
  grouped_tile(id, rtiles, rt, ct, C, row_group(rtiles));
  rt = __builtin_amdgcn_readfirstlane(rt);  // (tile addresses derive from them)
  ct = __builtin_amdgcn_readfirstlane(ct);
  const int i0 = rt * kBM;
  const int sl = __builtin_amdgcn_readfirstlane(ct / a.tg.tps), j = ct - sl * a.tg.tps;
  const int sbeg = (a.gm.s0 + sl) * a.gm.S;
  const int send = min(sbeg + a.gm.S, a.gm.V);
  const int c0 = sbeg + j * kBN + kChunk * max(half, 0);
  if (c0 >= send) return;
  const int c1 = min(c0 + (half < 0 ? kBN : kChunk), send);
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave_m(w),
            wn = wave_n(w);
  // this lane's rows' targets, loaded as in fwd_tiles
  int tgt[kMI];
  const auto load_row = [&](int mi, int ln) {
    if constexpr (kTop) tgt[mi] = a.yA[min(i0 + spread_row(wm, mi, ln), n_act - 1)];
  };
  const auto load_rows = [&]() {
#pragma unroll
    for (int mi = 0; mi < kTailRows; ++mi) load_row(mi, lane);
  };
  const RowsK A = rows_k_spread(a.hA + (size_t)i0 * a.H, min(n_act - i0, kBM) - 1, a.H);
  const RowsK B = rows_k(a.W + (size_t)c0 * a.H, c1 - 1 - c0, a.H);
  Acc acc;
  acc_zero(acc);
  if (half >= 0 && wn == 1) {
    gemm256<false, false, 0>(A, B, a.H / kBK, acc, lds);
    return;
  }
  gemm_rows(A, B, a.H / kBK, acc, lds, wm, min(n_act - i0, kBM), load_rows);

  const int cc0 = c0 + kChunk * wn;  // this wave's chunk
  const int width = min(cc0 + kChunk, c1) - cc0;
  if (width <= 0) return;
  const int ch = half < 0 ? wn : half, jc = 2 * j + ch;  // its number in the tile, in the split
  const int g = (a.gm.s0 + sl) * a.gm.cps + jc;
  int le = lane;  // an opaque copy, see fwd_tiles
  asm volatile("" : "+v"(le));
  const int rl = row_lane(le);
  const int lim = width - 4 * rl;  // value k is valid iff chunk_col(k) < lim
#pragma unroll
  for (int mi = kTailRows; mi < kMI; ++mi) load_row(mi, le);
  // the entries of row group rg in this tile
  int e0 = 0, e1 = 0;
  const uint32_t* ent = nullptr;
  const auto entries = [&](int rg) {
    const int32_t* off = a.ent_off + (size_t)rg * (kNSplit * a.tg.tps + 1) + (a.gm.s0 + sl) * a.tg.tps + j;
    e0 = __builtin_amdgcn_readfirstlane(off[0]);
    e1 = __builtin_amdgcn_readfirstlane(off[1]);
    ent = a.ent + (size_t)rg * kBucketRows * a.K;
  };
#pragma unroll
  for (int mi = 0; mi < kMI; ++mi) {
    const int b = spread_block(wm, mi), i_mi = i0 + kBlk * b;  // the row block and its first row
    if (i_mi >= n_act) continue;
    const int i = i_mi + le % kBlk;
    __builtin_amdgcn_sched_barrier(0);
    float v[kRowVals];
#pragma unroll
    for (int ni = 0; ni < kNI; ++ni)
#pragma unroll
      for (int r = 0; r < 4 * kQL; ++r)
        v[4 * kQL * ni + r] = kTop ? acc.c[mi][ni][r] : acc.c[mi][ni][r] * a.scale;
    // the wave's values in LDS (free once the engine has returned): lane l
    // holds its element k at float4 slot 64 (k >> 2) + l of the wave's slots
    float4* sl4 = reinterpret_cast<float4*>(lds) + 16 * kRowVals * w;
    const auto stage = [&]() {
#pragma unroll
      for (int q = 0; q < kRowVals / 4; ++q)
        sl4[64 * q + le] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
    };
    if constexpr (kTop) {
      if (a.z && i < n_act) {
        // whole chunks: the columns past the split's end hold logits of the
        // clamped last row, which no reader takes
        float* zr = a.z + (size_t)i * a.ldz + (size_t)kChunk * (sl * a.gm.cps + jc) + 4 * rl;
#pragma unroll
        for (int k = 0; k < kRowVals; k += 4)
          *reinterpret_cast<float4*>(zr + chunk_col(k)) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
      }
      const int tc = tgt[mi] - cc0;
      const bool hit = i < n_act && tc >= 0 && tc < width && ((tc >> 2) & (kLPR - 1)) == rl;
      if (__builtin_amdgcn_ballot_w64(hit)) {  // rare: see fwd_tiles
        stage();
        if (hit) {
          const int k = chunk_val(tc);
          a.zt[i] = reinterpret_cast<const float*>(sl4 + 64 * (k >> 2) + le)[k & 3];
        }
      }
    } else {
      bool staged = false;
      entries(i_mi / kBucketRows);
      for (int eb = e0; eb < e1; eb += 64) {
        const uint32_t x = eb + le < e1 ? ent[eb + le] : 0u;
        const int row = (x >> 8) & 255, col = x & 255;
        const bool mine = eb + le < e1 && row / kBlk == b && (col >> 7) == ch;
        if (!__builtin_amdgcn_ballot_w64(mine)) continue;
        if (!staged) {
          stage();
          // the wave's writes come before its lanes' reads of one another's values
          __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
          __builtin_amdgcn_wave_barrier();
          __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
          staged = true;
        }
        if (mine) {
          const int c = col & (kChunk - 1), k = chunk_val(c);
          const int from = row % kBlk + kBlk * ((c >> 2) & (kLPR - 1));
          a.z_ids[(size_t)(i0 + row) * a.K + (x >> 16)] = reinterpret_cast<const float*>(sl4 + 64 * (k >> 2) + from)[k & 3];
        }
      }
      // ... and the reads before the next row block's writes
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
    if (width < kChunk) {
#pragma unroll
      for (int k = 0; k < kRowVals; ++k)
        if (chunk_col(k) >= lim) v[k] = -INFINITY;
    }
    if constexpr (kTop) {
      const MSU st = chunk_stats_moment(v);
      if (rl == 0 && i < n_act) {
        a.rec[(size_t)g * a.rec_stride + i] = make_float2(st.m, st.s);
        a.rec_u[(size_t)g * a.rec_stride + i] = st.u;
      }
    } else {
      const float2 st = chunk_stats(v);
      if (rl == 0 && i < n_act) a.rec[(size_t)g * a.rec_stride + i] = st;
    }
  }
}

// -p (a + b (z - lse)), the softmax's share of dz; z already scaled.
// rowinfo = {lse, a, b, target}; b counts in the kTop instances only.
template <bool kTop>
__device__ __forceinline__ float minus_share(float z, const float4& r) {
  const float d = z - r.x;
  const float p = rlk_exp(d);
  if constexpr (kTop) return -(p * (r.y + r.z * fmaxf(d, kDeepest)));
  else return -(p * r.y);
}

#if RLK_MFMA == 16
// Waves wait for their own direct loads, all but the n issued last, and then
// for one another.
template <int n>
__device__ __forceinline__ void loads_then_barrier() {
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(n) : "memory");
  wait_lds();
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
}

// ---------------------------------------------------------------------------
// Few rows (T <= kFewRows): the same logits, statistics and dz with W streamed
// through a ring of LDS stages.
//
// With few rows the time is W's way from HBM, and that takes bytes in flight:
// about 2.9 us of them at full rate.  The engine has one tile per compute unit
// at a time, 1.5 k-blocks ahead, and gaps between tiles (256 rows of V =
// 151936: 4.3 TB/s).  Here a block stays on its unit and walks over chunks of
// 128 columns; two waves do nothing but issue the direct loads of stages
// (64 k of the chunk's W rows and of h, kSlots of them, kSlots - 1 in flight:
// 64 KB of W and more per unit) across the chunks' borders, and kC waves
// consume them, 32 rows each, while the next stages arrive.  A barrier per
// stage hands it over and its predecessor's slot back.  Every logit is the
// engine's MFMA chain (k ascending in steps of 32) in the engine's layout, so
// the statistics are the same bits.  Rows are those of the batch, in place: no
// compaction.
//
// One row, H = 4096: 223 - 230 us (5.4 - 5.6 TB/s of W; the copy's rate is 4.9
// read and written together); 48 rows of H = 2048: 146 (4.3 TB/s; the logits
// are 30 MB of stores besides).  W straight into registers took 225 at one row
// of H = 4096 but 335 at 64, and 193 at 48 of H = 2048; waves of 64 columns, or
// that split the rows, 465 and more (W's rows pass LDS once per wave).
// ---------------------------------------------------------------------------
constexpr int kFewRows = 128;

struct FewArgs {
  const uint16_t* h;  // [T, H]
  const uint16_t* W;
  int T, H;
  int chunks;  // of the launch: chunk c is chunk c % cps of split gm.s0 + c / cps
  SplitGeom gm;
  float scale;  // 1 / temperature; not applied by the kTop instances
  // logits
  size_t rec_stride;
  float2* rec;
  float* rec_u;
  float* z;     // row t, chunk c of the vocabulary at t * ldz + 128 c
  int64_t ldz;
  // dz
  const float4* rowinfo;  // [kFewRows] as for soft_dz_tiles; target kNoRow: zeros
  const float* rowg;
  BwdGeom bg;
  uint16_t* dZ;  // rows up to T's multiple of 64 are written
};

// Waves by consumers: 1, 2 or 4 for up to 32, 64 or 128 rows.
constexpr int few_consumers(int64_t T) { return T <= 32 ? 1 : T <= 64 ? 2 : 4; }
constexpr int few_threads(int consumers) { return 64 * (2 + consumers); }

template <bool kTop, bool kDz, int kC>
__global__ __launch_bounds__(few_threads(kC)) void few_tiles(FewArgs a) {
  constexpr uint32_t kWBytes = kChunk * 2 * kBK, kStage = kWBytes + 32 * kC * 2 * kBK;
  constexpr int kSlots = (160 << 10) / kStage, kLoads = 8 + 2 * kC;  // loads of a stage per loading wave
  static_assert((kSlots - 2) * kLoads < 64, "vmcnt");
  constexpr int kRB = 2, kCB = kChunk / 16;  // 16-row blocks of a wave, 16-column blocks
  __shared__ u32x4 lds[kSlots * kStage / 16];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nk = a.H / kBK;
  const int mine = (a.chunks - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;  // chunks b, b + grid, ...
  if (mine <= 0) return;
  // columns of chunk c: first one and how many (0 past the vocabulary)
  const auto chunk_at = [&](int c, int& s, int& j, int& c0) {
    s = c / a.gm.cps;
    j = c - s * a.gm.cps;
    const int sbeg = (a.gm.s0 + s) * a.gm.S;
    c0 = sbeg + j * kChunk;
    return max(0, min(kChunk, min(a.gm.S, a.gm.V - sbeg) - j * kChunk));
  };
  if (w >= kC) {
    // ---- loads: W rows 64 p + 8 i + lane / 8 of the chunk, h rows 16 kC p + 8 i + lane / 8
    const int p = w - kC, r8 = lane >> 3;
    uint32_t w_off[8], h_off[2 * kC];
#pragma unroll
    for (int i = 0; i < 2 * kC; ++i) {
      const int row = 16 * kC * p + 8 * i + r8;
      h_off[i] = 2u * ((uint32_t)min(row, a.T - 1) * a.H) + 16u * ((lane & 7) ^ ((row >> 1) & 7));
    }
    const char* wb = nullptr;
    int l_c = (int)blockIdx.x, l_kb = 0, l_left = mine;  // chunk and k-block of the stage loaded next
    const auto begin = [&]() {
      int s, j, c0;
      const int width = chunk_at(l_c, s, j, c0), last = max(width, 1) - 1;
      wb = reinterpret_cast<const char*>(a.W) + (size_t)__builtin_amdgcn_readfirstlane(width > 0 ? c0 : 0) * (2 * a.H);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int row = 64 * p + 8 * i + r8;
        w_off[i] = 2u * ((uint32_t)min(row, last) * a.H) + 16u * ((lane & 7) ^ ((row >> 1) & 7));
      }
    };
    begin();
    // Rows 4 KB apart, or a multiple of it, lie on few memory channels, and
    // blocks in step all ask for the same ones: they start up to 15 k-blocks
    // (0.8 us each) apart.  One row of H = 4096 256 -> 232 us, of 2048 139 ->
    // 124; at other widths waiting only costs (H = 4032: 213 -> 221).
    if (a.H % 2048 == 0 && a.chunks > (int)gridDim.x)
      for (int i = (int)(blockIdx.x >> 3) & 15; i > 0; --i) __builtin_amdgcn_s_sleep(26);
    const uint32_t lds0 = lds_addr(lds);
    const auto load = [&](int slot) {
      const uint32_t m0 = lds0 + kStage * slot;
      const size_t k2 = (size_t)l_kb * (2 * kBK);
#pragma unroll
      for (int i = 0; i < 8; ++i) dma16(wb + k2, w_off[i], m0 + 1024u * (8 * p + i));
#pragma unroll
      for (int i = 0; i < 2 * kC; ++i)
        dma16(reinterpret_cast<const char*>(a.h) + k2, h_off[i], m0 + kWBytes + 1024u * (2 * kC * p + i));
      if (l_kb + 1 < nk) {
        ++l_kb;
      } else if (l_left > 1) {  // (past the end: the last stage again, into a free slot)
        --l_left;
        l_kb = 0;
        l_c += (int)gridDim.x;
        begin();
      }
    };
#pragma unroll 1
    for (int i = 0; i + 1 < kSlots; ++i) load(i);
    int slot = 0;
#pragma unroll 1
    for (int i = 0; i < mine * nk; ++i) {
      loads_then_barrier<(kSlots - 2) * kLoads>();
      load(slot == 0 ? kSlots - 1 : slot - 1);  // the slot read last time
      slot = slot + 1 == kSlots ? 0 : slot + 1;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // nothing is loaded into LDS past the block's end
    return;
  }
  // ---- rows 32 w .. + 31
  const int r16 = lane & 15, rl = lane >> 4;
  int slot = 0;
#pragma unroll 1
  for (int n = 0; n < mine; ++n) {
    AccBlk acc[kRB][kCB];
#pragma unroll
    for (int m = 0; m < kRB; ++m)
#pragma unroll
      for (int b = 0; b < kCB; ++b) acc[m][b] = AccBlk{};
#pragma unroll 1
    for (int kt = 0; kt < nk; ++kt) {
      wait_lds();
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
      const char* st = reinterpret_cast<const char*>(lds) + kStage * slot;
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        bf16x8 x[kRB];
#pragma unroll
        for (int m = 0; m < kRB; ++m)
          x[m] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(
                                                st + kWBytes + 16u * slot_k(32 * w + 16 * m + r16, 4 * kk + rl)));
#pragma unroll
        for (int b = 0; b < kCB; ++b) {
          const bf16x8 y =
              __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(st + 16u * slot_k(16 * b + r16, 4 * kk + rl)));
#pragma unroll
          for (int m = 0; m < kRB; ++m) acc[m][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(y, x[m], acc[m][b], 0, 0, 0);
        }
      }
      slot = slot + 1 == kSlots ? 0 : slot + 1;
    }
    // lane l holds row 32 w + 16 m + l % 16, columns 16 b + 4 (l / 16) + e
    int s, j, c0;
    const int width = chunk_at((int)blockIdx.x + n * (int)gridDim.x, s, j, c0);
    if constexpr (kDz) {
      // (the last wave: zeros down to the rows' multiple of 64)
      const int rows = w + 1 < kC ? 32 : (a.T + 63) / 64 * 64 - 32 * w;
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        if (16 * m >= rows) continue;
        const int t = 32 * w + 16 * m + r16;
        const float4 ri = a.rowinfo[t];
        const int target = __float_as_int(ri.w), yl = target - c0;
        const bool on = m < kRB && target != kNoRow;
        const float g = kTop && on ? a.rowg[t] : 0.f;
#pragma unroll
        for (int b = 0; b < kCB; ++b) {
          const int c = 16 * b + 4 * rl;
          if (j * kChunk + c >= a.bg.S_pad) continue;  // the next split's columns
          float d[4] = {0.f, 0.f, 0.f, 0.f};
          if (m < kRB && on) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (c + e < width) {
                const float z = acc[m < kRB ? m : 0][b][e];
                const float x = minus_share<kTop>(kTop ? z : z * a.scale, ri);
                d[e] = kTop && c + e == yl ? g + x : x;
              }
          }
          *reinterpret_cast<uint2*>(a.dZ + (size_t)t * a.bg.ldz + (size_t)s * a.bg.S_pad + j * kChunk + c) =
              make_uint2(pack_bf16x2(d[0], d[1]), pack_bf16x2(d[2], d[3]));
        }
      }
    } else {
      if (width <= 0) continue;
      const int g = (a.gm.s0 + s) * a.gm.cps + j;
#pragma unroll
      for (int m = 0; m < kRB; ++m) {
        const int t = 32 * w + 16 * m + r16;
        float v[4 * kCB];
#pragma unroll
        for (int b = 0; b < kCB; ++b) {
          const int c = 16 * b + 4 * rl;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[4 * b + e] = kTop ? acc[m][b][e] : acc[m][b][e] * a.scale;
          if (t < a.T)  // whole chunks: what lies past the split's end is not read
            *reinterpret_cast<float4*>(a.z + (size_t)t * a.ldz + (size_t)g * kChunk + c) =
                make_float4(v[4 * b], v[4 * b + 1], v[4 * b + 2], v[4 * b + 3]);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (c + e >= width) v[4 * b + e] = -INFINITY;
        }
        const MSU st = chunk_stats_moment(v);
        if (rl == 0 && t < a.T) {
          a.rec[(size_t)g * a.rec_stride + t] = make_float2(st.m, st.s);
          if (kTop) a.rec_u[(size_t)g * a.rec_stride + t] = st.u;
        }
      }
    }
  }
}
#endif  // RLK_MFMA == 16

// ---------------------------------------------------------------------------
// Row gathers
// ---------------------------------------------------------------------------
// hA[i] = h[idx[i]] for active rows i < n_act, zero rows for n_act <= i <
// rows, and the K slots of the inactive rows t < T (act[t] == ignore):
// slot_logp = -inf, slot_ids (optional) = -1.  Block 256, 16-byte pieces.
struct GatherArgs {
  const uint16_t* h;
  const int32_t* idx;
  const int32_t* n_act;
  int T, rows, H;
  uint16_t* hA;
  const int32_t* act;
  int ignore_index;
  int K;
  float* slot_logp;
  int32_t* slot_ids;
};

__device__ __forceinline__ void gather_row(const uint16_t* h, const int32_t* idx, int n_act, int i, int H,
                                           uint16_t* hA) {
  u32x4* dst = reinterpret_cast<u32x4*>(hA + (size_t)i * H);
  if (i < n_act) {
    const u32x4* src = reinterpret_cast<const u32x4*>(h + (size_t)idx[i] * H);
    for (int p = threadIdx.x; p < H / 8; p += 256) dst[p] = src[p];
  } else {
    for (int p = threadIdx.x; p < H / 8; p += 256) dst[p] = u32x4{0u, 0u, 0u, 0u};
  }
}

__global__ __launch_bounds__(256) void gather_rows_fill(GatherArgs a) {
  const int n_act = *a.n_act;
  for (int i = blockIdx.x; i < a.rows; i += gridDim.x) {
    gather_row(a.h, a.idx, n_act, i, a.H, a.hA);
    if (i < a.T && a.act[i] == a.ignore_index) {
      for (int k = threadIdx.x; k < a.K; k += 256) {
        a.slot_logp[(size_t)i * a.K + k] = -INFINITY;
        if (a.slot_ids) a.slot_ids[(size_t)i * a.K + k] = -1;
      }
    }
  }
}

// hA as above, and per active row the coefficients of
//     dz_v = g [v == target] - p_v (a + b (z_v - lse)),  p_v = e(z_v - lse):
// rowinfo = {lse, a, b, target (bits)}, rowg = g; {0, 0, 0, -1} past n_act.
// top: a = g + b entropy, b = dL/dentropy.  distill: a = -(dL/dloss /
// temperature), b = 0, no target; the teacher's share of dz comes from
// distill_scatter.  A row without a defined loss (a target outside the
// vocabulary; see distill_row) gets NaN coefficients.
struct GatherGradArgs {
  const uint16_t* h;
  const int32_t* idx;
  const int32_t* n_act;
  int rows, H, V;
  uint16_t* hA;
  const float* lse;
  const float* g;           // may be NULL (top: zero)
  float4* rowinfo;
  float* rowg;
  // top
  const int32_t* y;
  const float* entropy;
  const float* g_entropy;   // may be NULL (zero)
  const int32_t* act;       // top: y; distill: the rows' states (distill_row)
  float scale;
};

template <bool kTop>
__device__ __forceinline__ float4 grad_row(const GatherGradArgs& a, int t, int state, float* g_out) {
  float4 ri = make_float4(a.lse[t], 0.f, 0.f, __int_as_float(-1));
  float gt = 0.f;
  if constexpr (kTop) {
    const int yt = a.y[t];
    gt = a.g ? a.g[t] : 0.f;
    const bool ok = yt >= 0 && yt < a.V;
    if (!ok) gt = __builtin_nanf("");
    ri.z = a.g_entropy ? a.g_entropy[t] : 0.f;
    ri.y = gt + ri.z * a.entropy[t];
    ri.w = __int_as_float(ok ? yt : -1);
  } else {
    ri.y = state == 1 ? __builtin_nanf("") : -(a.g[t] * a.scale);
  }
  *g_out = gt;
  return ri;
}

template <bool kTop>
__global__ __launch_bounds__(256) void gather_rows_grad(GatherGradArgs a) {
  const int n_act = *a.n_act;
  for (int i = blockIdx.x; i < a.rows; i += gridDim.x) {
    gather_row(a.h, a.idx, n_act, i, a.H, a.hA);
    if (threadIdx.x == 0)
      a.rowinfo[i] = i < n_act ? grad_row<kTop>(a, a.idx[i], kTop ? 0 : a.act[a.idx[i]], a.rowg + i) : make_float4(0.f, 0.f, 0.f, __int_as_float(-1));
  }
}

// ---------------------------------------------------------------------------
// The teacher's rows
// ---------------------------------------------------------------------------
// Slot k of a row is kept iff its id is >= 0 and its logit is not -inf.
__device__ __forceinline__ bool slot_kept(int id, float logit) { return id >= 0 && logit != -INFINITY; }

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) x = fmaxf(x, __shfl_xor(x, d));
  return x;
}
__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) x = x + __shfl_xor(x, d);
  return x;
}

// A teacher's row over a wave: lane l holds slots l and l + 64.
// q = softmax of the kept logits / temperature, lq = log q.  The max is taken
// off before the quotient: any finite logits are defined then (rows masked
// with the type's lowest value, under a temperature below 1), and a quotient's
// error is that of the distance to the max.  (distill_rows of 4096 rows of 64:
// 4 us.)
constexpr int kSlots2 = kMaxK / 64;
struct TeacherRow {
  int id[kSlots2];
  bool kept[kSlots2];
  float q[kSlots2], lq[kSlots2];
};

__device__ __forceinline__ TeacherRow teacher_row(const int32_t* ids, const float* logits, int K, float scale) {
  const int lane = threadIdx.x & 63;
  TeacherRow r;
  float x[kSlots2], m = -INFINITY;
  bool bad = false;  // fmaxf would drop a NaN
#pragma unroll
  for (int s = 0; s < kSlots2; ++s) {
    const int k = lane + 64 * s;
    r.id[s] = k < K ? ids[k] : -1;
    const float l = k < K ? logits[k] : -INFINITY;
    r.kept[s] = slot_kept(r.id[s], l);
    x[s] = r.kept[s] ? l : -INFINITY;
    m = fmaxf(m, x[s]);
    bad |= x[s] != x[s];
  }
  m = wave_max(m);
  if (__builtin_amdgcn_ballot_w64(bad)) m = __builtin_nanf("");
  float sum = 0.f;
#pragma unroll
  for (int s = 0; s < kSlots2; ++s) {
    x[s] = (x[s] - m) * scale;
    r.q[s] = r.kept[s] ? rlk_exp(x[s]) : 0.f;
    sum = sum + r.q[s];
  }
  sum = wave_sum(sum);
  const float L = rlk_log(sum);
#pragma unroll
  for (int s = 0; s < kSlots2; ++s) {
    r.lq[s] = r.kept[s] ? x[s] - L : 0.f;
    r.q[s] = r.kept[s] ? r.q[s] / sum : 0.f;
  }
  return r;
}

// The state of row t over a wave: -100 without a kept token, 1 where the loss
// is undefined (a kept token outside the vocabulary, or a logit that makes q
// NaN), else 0; q (optional): the teacher's distribution.
__device__ __forceinline__ int distill_row(const int32_t* ids, const float* logits, int t, int K, int V, float scale,
                                           float* q) {
  const int lane = threadIdx.x & 63;
  const TeacherRow r = teacher_row(ids + (size_t)t * K, logits + (size_t)t * K, K, scale);
  bool any = false, out = false;
#pragma unroll
  for (int s = 0; s < kSlots2; ++s) {
    any |= r.kept[s];
    out |= r.kept[s] && (r.id[s] >= V || r.q[s] != r.q[s]);
    if (q && lane + 64 * s < K) q[(size_t)t * K + lane + 64 * s] = r.q[s];
  }
  const bool any_w = __builtin_amdgcn_ballot_w64(any) != 0, out_w = __builtin_amdgcn_ballot_w64(out) != 0;
  return !any_w ? -100 : out_w ? 1 : 0;
}

// act[t] = the rows' states.  One wave per row.
__global__ __launch_bounds__(256) void distill_rows(const int32_t* __restrict__ ids, const float* __restrict__ logits,
                                                    int T, int K, int V, float scale, int32_t* __restrict__ act,
                                                    float* __restrict__ q) {
  for (int t = blockIdx.x * 4 + (threadIdx.x >> 6); t < T; t += gridDim.x * 4) {
    const int state = distill_row(ids, logits, t, K, V, scale, q);
    if ((threadIdx.x & 63) == 0) act[t] = state;
  }
}

// Few rows: the batch's rows in place.  hA[t] = h[t], zeros for inactive rows
// and past T (they meet dz = 0 in grad_W, and may hold anything in h);
// n_act = T.  distill: wave 0 finds the row's state first (and act, q for the
// kernels after this one).  Grid: `rows` blocks.
struct FewRowsArgs {
  GatherGradArgs ga;
  int T, ignore_index;
  int32_t* n_act;
  // distill
  const int32_t* ids;
  const float* logits;
  int K;
  int32_t* act;  // = ga.act
  float* q;
};

template <bool kTop>
__global__ __launch_bounds__(256) void few_rows_grad(FewRowsArgs f) {
  __shared__ int state_s;
  const GatherGradArgs& a = f.ga;
  const int t = blockIdx.x;
  int state = f.ignore_index;
  if constexpr (kTop) {
    if (t < f.T) state = a.act[t];
  } else {
    if (threadIdx.x < 64) {
      if (t < f.T) {
        state = distill_row(f.ids, f.logits, t, f.K, a.V, a.scale, f.q);
        if (threadIdx.x == 0) f.act[t] = state;
      }
      if (threadIdx.x == 0) state_s = state;
    }
    __syncthreads();
    state = state_s;
  }
  const bool on = t < f.T && state != f.ignore_index;
  u32x4* dst = reinterpret_cast<u32x4*>(a.hA + (size_t)t * a.H);
  const u32x4* src = reinterpret_cast<const u32x4*>(a.h + (size_t)t * a.H);
  for (int p = threadIdx.x; p < a.H / 8; p += 256) dst[p] = on ? src[p] : u32x4{0u, 0u, 0u, 0u};
  if (threadIdx.x == 0) {
    a.rowinfo[t] = on ? grad_row<kTop>(a, t, state, a.rowg + t) : make_float4(0.f, 0.f, 0.f, __int_as_float(kNoRow));
    if (t == 0) *f.n_act = f.T;
  }
}

// The entries of every kBucketRows active rows, grouped by the vocabulary
// tile their token lies in: off[rb][c] .. off[rb][c + 1] are those of tile c
// (= split * tps + tile of the split).  Within a tile the order is left open:
// every entry writes a place of its own.  One block per row group: small
// groups, since a teacher's tokens crowd in few tiles, whose counters take
// their entries one after the other (256 rows of 128 in one block: 38 us).
constexpr int kBucketThreads = 256;
constexpr int kMaxVTiles = 32768;  // 32 tps for the largest vocabulary: 31264
template <int kTiles>
__global__ __launch_bounds__(kBucketThreads) void bucket_entries(const int32_t* __restrict__ ids,
                                                                 const float* __restrict__ logits,
                                                                 const int32_t* __restrict__ idx,
                                                                 const int32_t* __restrict__ n_act_p, int K,
                                                                 SplitGeom gm, int tps, int32_t* __restrict__ off,
                                                                 uint32_t* __restrict__ ent) {
  __shared__ int32_t cnt[kTiles];
  __shared__ int32_t row_s[kBucketRows];
  __shared__ int32_t wave_tot[kBucketThreads / 64];
  const int rg = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int i0 = rg * kBucketRows, n = min(kBucketRows, *n_act_p - i0);
  if (n <= 0) return;
  const int C = kNSplit * tps;
  for (int c = tid; c < C; c += kBucketThreads) cnt[c] = 0;
  if (tid < n) row_s[tid] = idx[i0 + tid];
  __syncthreads();
  // thread tid takes slot tid % kp of rows tid / kp, + kBucketThreads / kp,
  // ... (kp: the power of two at or above K), kAhead of them at a time: the
  // loads unrolled, the loop not (see the row kernels below)
  const int kp = 1 << (32 - __builtin_clz(max(K - 1, 1))), shift = __builtin_ctz(kp);
  const int k = tid & (kp - 1), r0 = tid >> shift, step = kBucketThreads >> shift;
  const uint32_t rcp = (uint32_t)(((uint64_t(1) << 32) - 1) / (uint32_t)gm.S);
  constexpr int kAhead = 8;
  const auto each = [&](auto&& f) {
#pragma unroll 1
    for (int rb = r0; rb - r0 < n; rb += kAhead * step) {
      int id[kAhead];
      float lg[kAhead];
#pragma unroll
      for (int e = 0; e < kAhead; ++e) {
        const int r = rb + e * step;
        id[e] = -1;
        lg[e] = 0.f;
        if (r < n && k < K) {
          const size_t at = (size_t)row_s[r] * K + k;
          id[e] = ids[at];
          lg[e] = logits[at];
        }
      }
#pragma unroll
      for (int e = 0; e < kAhead; ++e) {
        if (id[e] >= gm.V || !slot_kept(id[e], lg[e])) continue;
        // id / S: the truncated reciprocal's quotient is short by at most one
        int q = (int)__umulhi((uint32_t)id[e], rcp), c = id[e] - q * gm.S;
        if (c >= gm.S) {
          c -= gm.S;
          ++q;
        }
        f(q * tps + (c >> 8), entry_of(c & 255, i0 % kBM + rb + e * step, k));
      }
    }
  };
  each([&](int bin, uint32_t) { atomicAdd(&cnt[bin], 1); });
  __syncthreads();
  // exclusive scan: thread tid takes `per` consecutive tiles
  const int per = (C + kBucketThreads - 1) / kBucketThreads;
  const int lo = min(tid * per, C), hi = min(lo + per, C);
  int sum = 0;
  for (int c = lo; c < hi; ++c) sum += cnt[c];
  int incl = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 63) wave_tot[wave] = incl;
  __syncthreads();
  int pos = incl - sum;
  for (int w = 0; w < wave; ++w) pos += wave_tot[w];
  int32_t* o = off + (size_t)rg * (C + 1);
  for (int c = lo; c < hi; ++c) {
    const int v = cnt[c];
    o[c] = pos;
    cnt[c] = pos;
    pos += v;
  }
  if (tid == kBucketThreads - 1) o[C] = pos;
  __syncthreads();
  uint32_t* e0 = ent + (size_t)rg * kBucketRows * K;
  each([&](int bin, uint32_t x) { e0[atomicAdd(&cnt[bin], 1)] = x; });
}

// ---------------------------------------------------------------------------
// Row kernels after the logits: a block per row, of one wave or two.  With one row
// they are latency alone, and most of that is instruction fetch: unrolled
// forms of these loops, which run through their code once, took 54 us where
// the rolled ones below take 17 (20 alternatives, V = 151936).  So loops stay
// rolled, what is loaded ahead goes through LDS, and only the loads are
// unrolled.  With the fold in a wave of its own one row takes 20 - 21 us with
// its alternatives.  A chunk's records of neighbouring rows share cache lines,
// so a die takes consecutive rows (xcd_tile): 3482 rows, 20 alternatives, 108
// us (51 MB of records and about 21 of a row's 1216 chunks of logits each);
// their divergences from 64 tokens 37 us.
// ---------------------------------------------------------------------------
// The lanes of a wave see one another's LDS writes.
__device__ __forceinline__ void wave_lds_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Place of token v's logit in a row of all chunks' logits.
__device__ __forceinline__ int logit_at(const SplitGeom& gm, int v) {
  const int s = v / gm.S;
  return s * gm.cps * kChunk + (v - s * gm.S);
}

// Chunks of split `s` that hold columns.
__device__ __forceinline__ int chunks_of(const SplitGeom& gm, int s) {
  const int cols = min(gm.S, gm.V - s * gm.S);
  return cols > 0 ? (cols + kChunk - 1) / kChunk : 0;
}

// Fold of active row i.  Lane s < 32 folds split s (chunks left to right);
// the splits then meet in a pairwise tree over the lanes (lane 2w j takes
// lane 2w j + w): the order, and for m and s the bits, of merge_splits.  All
// lanes load, kFoldAhead chunks of every split at a time, the next ones while
// these are folded.  The result is valid in lane 0.  buf: kFoldFloats floats.
constexpr int kFoldAhead = 16;
constexpr int kFoldFloats = 3 * kFoldAhead * kNSplit;
template <bool kMoment>
__device__ __forceinline__ MSU fold_row(const float2* rec, const float* rec_u, size_t stride, int i,
                                        const SplitGeom& gm, float* buf) {
  const int lane = threadIdx.x & 63, s = lane & (kNSplit - 1), half = lane / kNSplit;
  constexpr int kEach = kFoldAhead / 2;
  const int nj = chunks_of(gm, s);
  const size_t base = (size_t)s * gm.cps * stride + i;
  float2* b_ms = reinterpret_cast<float2*>(buf);
  float* b_u = buf + 2 * kFoldAhead * kNSplit;
  float2 ms[kEach];
  float u[kEach];
  const auto load = [&](int j0) {
#pragma unroll
    for (int b = 0; b < kEach; ++b) {
      const int j = j0 + half * kEach + b;
      if (j < nj) {
        ms[b] = rec[base + (size_t)j * stride];
        if (kMoment) u[b] = rec_u[base + (size_t)j * stride];
      }
    }
  };
  MSU r = msu_identity();
  load(0);
#pragma unroll 1
  for (int j0 = 0; j0 < gm.cps; j0 += kFoldAhead) {
#pragma unroll
    for (int b = 0; b < kEach; ++b) {
      b_ms[(half * kEach + b) * kNSplit + s] = ms[b];
      if (kMoment) b_u[(half * kEach + b) * kNSplit + s] = u[b];
    }
    wave_lds_sync();
    load(j0 + kFoldAhead);
    const int n = half ? 0 : min(kFoldAhead, nj - j0);
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
      const float2 x = b_ms[j * kNSplit + s];
      if constexpr (kMoment) {
        r = msu_combine(r, MSU{x.x, x.y, b_u[j * kNSplit + s]});
      } else {
        const MS t = ms_combine(MS{r.m, r.s}, MS{x.x, x.y});
        r.m = t.m;
        r.s = t.s;
      }
    }
    wave_lds_sync();
  }
#pragma unroll 1
  for (int w = 1; w < kNSplit; w <<= 1) {
    MSU b;
    b.m = __shfl_down(r.m, w);
    b.s = __shfl_down(r.s, w);
    b.u = kMoment ? __shfl_down(r.u, w) : 0.f;
    if constexpr (kMoment) {
      r = msu_combine(r, b);
    } else {
      const MS t = ms_combine(MS{r.m, r.s}, MS{b.m, b.s});
      r.m = t.m;
      r.s = t.s;
    }
  }
  return r;
}

// ---------------------------------------------------------------------------
// The K best of a row, ties to the lowest id.
//
// A logit and its id make one 64-bit key (the logit's bits in an order that
// integers keep, -0 as +0, then the id's complement): all keys of a row
// differ, and a larger key is a better alternative.  The chunks are dealt
// into 256 groups; tau = the K-th largest of the groups' maxima (bit by bit,
// counting the groups at or above).  K logits at least are >= tau, so the K
// best are, and they lie in the chunks whose max is >= tau: about
// -256 log(1 - K / 256) of them.  Their logits at or above tau go to a list,
// its K best come out by counting.  When the list fills up it is cut to its K
// best, and what is accepted to what beats the last of them.
//
// Lanes l and l + 32 hold the two halves of split l's chunks, at most
// kSelPer each; splits of more than 2 kSelPer chunks (vocabularies past
// 262144) take runs of R chunks as one.
// ---------------------------------------------------------------------------
constexpr int kSelPer = 32;                // runs per lane
constexpr int kSelGroups = 4;              // groups per lane
constexpr int kSelRuns = 64 * kSelPer;
constexpr int kSelList = 512;              // keys of a row in LDS
constexpr int kSelAhead = 16;              // chunks whose logits are loaded together
static_assert(kSelList >= kMaxK + 64, "room for a step after a cut");
static_assert(64 * kSelGroups >= kMaxK, "K groups");
static_assert(kSelAhead * kChunk <= kSelRuns, "one LDS array serves both");

__device__ __forceinline__ uint32_t ordered_bits(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t o) {
  return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// list[0..n) -> its min(n, K) best in descending order; returns their number.
__device__ __forceinline__ int keep_best(uint64_t* list, int n, int K) {
  const int lane = threadIdx.x & 63;
  constexpr int kPer = kSelList / 64;
  uint64_t x[kPer];
  int rank[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    x[e] = 64 * e + lane < n ? list[64 * e + lane] : 0;
    rank[e] = 0;
  }
#pragma unroll 1
  for (int j = 0; j < n; ++j) {
    const uint64_t b = list[j];
    rank[0] += b > x[0];
    if (n > 64) {
#pragma unroll
      for (int e = 1; e < kPer; ++e) rank[e] += b > x[e];
    }
  }
  wave_lds_sync();
#pragma unroll
  for (int e = 0; e < kPer; ++e)
    if (64 * e + lane < n && rank[e] < K) list[rank[e]] = x[e];
  wave_lds_sync();
  return min(n, K);
}

struct TopMergeArgs {
  const float2* rec;
  const float* rec_u;
  size_t rec_stride;
  const float* zt;       // NULL: the target's logit is in z
  const int32_t* idx;    // NULL: every row of the batch, in place
  const int32_t* n_act;
  int T, ignore_index;
  const int32_t* y;
  SplitGeom gm;    // gm.s0: first split of the group
  int G;           // splits of the group whose logits z holds
  int first, last; // is it the first / last group
  int R;           // chunks taken as one
  const float* z;
  int64_t ldz;
  int K;
  uint64_t* best;  // [active row][K] keys of the groups so far, best first
  float* logp;
  float* lse;      // may be NULL
  float* entropy;
  float* top_logp;
  int32_t* top_ids;
};

// Two waves a row: one picks the alternatives, the other folds the statistics
// (after the last group); the first then needs m and log s of the second.
__global__ __launch_bounds__(128) void top_merge(TopMergeArgs a) {
  __shared__ uint32_t pool[kSelRuns];  // run maxima, then logits
  __shared__ uint64_t list[kSelList];
  __shared__ uint16_t picks[kSelRuns];
  __shared__ float records[kFoldFloats];
  __shared__ float m_s, log_s;
  const int lane = threadIdx.x & 63, i = xcd_tile(a.idx ? *a.n_act : a.T, blockIdx.x);
  const bool folds = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) == 1;
  if (i < 0) return;
  const int t = a.idx ? a.idx[i] : i, yt = a.y[t];
  if (!a.idx && yt == a.ignore_index) {
    if (folds) return;
    if (lane == 0) {
      a.logp[t] = a.entropy[t] = 0.f;
      if (a.lse) a.lse[t] = 0.f;
    }
    for (int k = lane; k < a.K; k += 64) {
      a.top_ids[(size_t)t * a.K + k] = -1;
      a.top_logp[(size_t)t * a.K + k] = -INFINITY;
    }
    return;
  }
  if (folds) {
    if (!a.last) return;
    const MSU tot = fold_row<true>(a.rec, a.rec_u, a.rec_stride, i, a.gm, records);
    if (lane == 0) {
      const float m = tot.m, L = rlk_log(tot.s);
      float lp = __builtin_nanf("");
      if (yt >= 0 && yt < a.gm.V) {
        const float zt = a.zt ? a.zt[i] : a.z[(size_t)i * a.ldz + logit_at(a.gm, yt)];
        lp = (zt - m) - L;
      }
      a.logp[t] = lp;
      if (a.lse) a.lse[t] = m + L;
      a.entropy[t] = L - tot.u / tot.s;
      m_s = m;
      log_s = L;
    }
    __syncthreads();
    return;
  }
  int n = 0;
  if (a.K > 0) {
    // this lane's runs of R chunks: run e is chunks j0 + e R .. of split s0 + sl
    const int sl = lane & (kNSplit - 1), hs = ((a.gm.cps + a.R - 1) / a.R + 1) / 2;
    const int nj = sl < a.G ? chunks_of(a.gm, a.gm.s0 + sl) : 0;
    const int j0 = lane / kNSplit * hs * a.R;
    const float2* rec = a.rec + (size_t)(a.gm.s0 + sl) * a.gm.cps * a.rec_stride + i;
    uint32_t top[kSelGroups] = {0, 0, 0, 0};  // groups' maxima (0: no columns)
    constexpr int kLoads = 16;
#pragma unroll 1
    for (int e0 = 0; e0 < hs; e0 += kLoads) {
      float m[kLoads];
#pragma unroll
      for (int e = 0; e < kLoads; ++e) {
        const int j = j0 + (e0 + e) * a.R;
        if (e0 + e < hs && j < nj) m[e] = rec[(size_t)j * a.rec_stride].x;
      }
#pragma unroll
      for (int e = 0; e < kLoads; ++e) {
        const int j = j0 + (e0 + e) * a.R;
        if (e0 + e >= hs) continue;
        uint32_t x = j < nj ? ordered_bits(m[e]) : 0;
        for (int r = 1; r < a.R; ++r)
          if (j + r < nj) x = max(x, ordered_bits(rec[(size_t)(j + r) * a.rec_stride].x));
        pool[(e0 + e) * 64 + lane] = x;
        top[e % kSelGroups] = max(top[e % kSelGroups], x);
      }
    }
    // the largest tau that K groups reach (1, any logit, if fewer hold columns)
    uint32_t tau = 0;
#pragma unroll 1
    for (int b = 31; b >= 0; --b) {
      const uint32_t t = tau | (1u << b);
      int c = 0;
#pragma unroll
      for (int e = 0; e < kSelGroups; ++e) c += __builtin_popcountll(__builtin_amdgcn_ballot_w64(top[e] >= t));
      if (c >= a.K) tau = t;
      if (c == a.K) break;
    }
    tau = max(tau, 1u);
    // the runs that reach it
    int np = 0;
#pragma unroll 1
    for (int e = 0; e < hs; ++e) {
      const bool take = pool[e * 64 + lane] >= tau;
      const uint64_t mask = __builtin_amdgcn_ballot_w64(take);
      if (take) picks[np + __builtin_popcountll(mask & ((uint64_t(1) << lane) - 1))] = (uint16_t)(e * 64 + lane);
      np += __builtin_popcountll(mask);
    }
    uint64_t floor = (uint64_t)tau << 32;
    if (!a.first) {
      const uint64_t* b = a.best + (size_t)i * a.K;
      for (int k = lane; k < a.K; k += 64) list[k] = b[k];
      for (int k0 = 0; k0 < a.K; k0 += 64)
        n += __builtin_popcountll(__builtin_amdgcn_ballot_w64(k0 + lane < a.K && b[k0 + lane] != 0));
      if (n == a.K) floor = max(floor, b[a.K - 1]);
    }
    wave_lds_sync();
    // their logits, two columns a lane
    const float* zr = a.z + (size_t)i * a.ldz;
    float2* stage = reinterpret_cast<float2*>(pool);
    const int np_c = np * a.R;
    // chunk p of the picked runs: its split (of the group) and number there
    const auto chunk_at = [&](int p, int& ps, int& j) {
      const int q = __builtin_amdgcn_readfirstlane(picks[a.R == 1 ? p : p / a.R]);
      ps = q & (kNSplit - 1);
      j = ((q & 63) / kNSplit * hs + (q >> 6)) * a.R + (a.R == 1 ? 0 : p % a.R);
    };
#pragma unroll 1
    for (int p0 = 0; p0 < np_c; p0 += kSelAhead) {
      float2 v[kSelAhead];
#pragma unroll
      for (int e = 0; e < kSelAhead; ++e) {
        if (p0 + e >= np_c) continue;
        int ps, j;
        chunk_at(p0 + e, ps, j);
        if (j < a.gm.cps)
          v[e] = *reinterpret_cast<const float2*>(zr + (size_t)(ps * a.gm.cps + j) * kChunk + 2 * lane);
      }
#pragma unroll
      for (int e = 0; e < kSelAhead; ++e) stage[64 * e + lane] = v[e];
      wave_lds_sync();
#pragma unroll 1
      for (int e = 0; e < min(kSelAhead, np_c - p0); ++e) {
        int ps, j;
        chunk_at(p0 + e, ps, j);
        const int sbeg = (a.gm.s0 + ps) * a.gm.S;
        const int id0 = sbeg + j * kChunk + 2 * lane, end = min(sbeg + a.gm.S, a.gm.V);
        const float2 x2 = stage[64 * e + lane];
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          const int id = id0 + h;
          const float x = h ? x2.y : x2.x;
          const uint64_t key = (uint64_t)ordered_bits(x) << 32 | (0xFFFFFFFFu - (uint32_t)id);
          const bool take = id < end && x == x && key >= floor;
          const uint64_t mask = __builtin_amdgcn_ballot_w64(take);
          if (!mask) continue;
          if (n + __builtin_popcountll(mask) > kSelList) {
            wave_lds_sync();
            n = keep_best(list, n, a.K);
            floor = max(floor, list[a.K - 1]);  // n == K: the list held more
          }
          if (take) list[n + __builtin_popcountll(mask & ((uint64_t(1) << lane) - 1))] = key;
          n += __builtin_popcountll(mask);
        }
      }
      wave_lds_sync();
    }
    n = keep_best(list, n, a.K);
    if (!a.last)
      for (int k = lane; k < a.K; k += 64) a.best[(size_t)i * a.K + k] = k < n ? list[k] : 0;
  }
  if (!a.last) return;
  __syncthreads();
  const float m = m_s, L = log_s;
  for (int k = lane; k < a.K; k += 64) {
    const bool some = k < n;
    const uint64_t key = some ? list[k] : 0;
    a.top_ids[(size_t)t * a.K + k] = some ? (int32_t)(0xFFFFFFFFu - (uint32_t)key) : -1;
    a.top_logp[(size_t)t * a.K + k] = some ? (from_ordered((uint32_t)(key >> 32)) - m) - L : -INFINITY;
  }
}

// ---------------------------------------------------------------------------
// The divergence of a row: loss = sum_k q_k (log q_k - log p_k),
// log p_k = (z_k - m) - log s of the teacher's tokens.  One wave per row.
// ---------------------------------------------------------------------------
struct DistillMergeArgs {
  const float2* rec;
  size_t rec_stride;
  const int32_t* idx;
  const int32_t* n_act;
  SplitGeom gm;
  int K;
  float scale;
  const int32_t* ids;
  const float* logits;
  const float* z_ids;  // [active row][K], scaled; NULL: they are in z
  const float* z;      // (idx, n_act NULL: every row of the batch, in place)
  int64_t ldz;
  int T;
  float* loss;
  float* lse;
  float* logp_ids;
};

__global__ __launch_bounds__(64) void distill_merge(DistillMergeArgs a) {
  __shared__ float buf[kFoldFloats];
  const int lane = threadIdx.x, i = xcd_tile(a.idx ? *a.n_act : a.T, blockIdx.x);
  if (i < 0) return;
  const int t = a.idx ? a.idx[i] : i;
  const TeacherRow r = teacher_row(a.ids + (size_t)t * a.K, a.logits + (size_t)t * a.K, a.K, a.scale);
  if (!a.idx) {
    bool any = false;
#pragma unroll
    for (int s = 0; s < kSlots2; ++s) any |= r.kept[s];
    if (!__builtin_amdgcn_ballot_w64(any)) {
      if (lane == 0) a.loss[t] = a.lse[t] = 0.f;
      for (int k = lane; k < a.K; k += 64) a.logp_ids[(size_t)t * a.K + k] = -INFINITY;
      return;
    }
  }
  const MSU tot = fold_row<false>(a.rec, nullptr, a.rec_stride, i, a.gm, buf);
  const float m = __shfl(tot.m, 0), L = rlk_log(__shfl(tot.s, 0));
  float sum = 0.f;
#pragma unroll
  for (int s = 0; s < kSlots2; ++s) {
    const int k = lane + 64 * s;
    if (k >= a.K) continue;
    float lp = -INFINITY;
    if (r.kept[s]) {
      lp = __builtin_nanf("");
      if (r.id[s] < a.gm.V) {
        const float z = a.z_ids ? a.z_ids[(size_t)i * a.K + k] : a.z[(size_t)i * a.ldz + logit_at(a.gm, r.id[s])];
        lp = (z - m) - L;
      }
      // a token that the teacher gives no weight adds nothing, whatever the student gives it
      if (r.q[s] != 0.f || lp != lp) sum = sum + r.q[s] * (r.lq[s] - lp);
    }
    a.logp_ids[(size_t)t * a.K + k] = lp;
  }
  sum = wave_sum(sum);
  if (lane == 0) {
    a.loss[t] = sum;
    a.lse[t] = m + L;
  }
}

// ---------------------------------------------------------------------------
// dz of a group of splits from recomputed logits, bf16: tiles, staging and
// stores as in dz_tiles;
//     dz_v = g [v == target] - p_v (a + b (z_v - lse)),  p_v = e(z_v - lse),
// z scaled by 1 / temperature.  fp32, each operation rounded once, then bf16
// once: dz is an operand of the gradients' bf16 products, and two bf16 terms of
// it would double them (gradients 0.0023 - 0.0025 off 64 bits, where their own
// rounding to bf16 is 0.0017).
// kTop: with target and b; !kTop: a alone.
// Bound by the engine's MFMAs: 3482 active rows, H = 4096 (4.33 TFLOP) 3.00 -
// 3.11 ms (1.39 - 1.44 PFLOP/s), 3 % above the logits of the forward (1.1 GB
// of dz).
// ---------------------------------------------------------------------------
struct SoftDzArgs {
  const uint16_t* hA;
  const uint16_t* W;
  const float4* rowinfo;  // {lse, a, b, target (bits)}
  const float* rowg;      // g
  const int32_t* n_act;
  int H;
  int cus;                // see tile_of_block
  float scale;
  SplitGeom gm;
  TileGeom tg;
  BwdGeom bg;
  uint16_t* dZ;
};

template <bool kTop>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(RLK_WAVES / 4, RLK_WAVES / 4))) void soft_dz_tiles(
    SoftDzArgs a) {
  __shared__ u32x4 lds[kLdsU4];
  const int n_act = __builtin_amdgcn_readfirstlane(*a.n_act);
  const int rtiles = (n_act + kBM - 1) / kBM;
  const int C = a.bg.G * a.tg.tps;
  int id, half;
  if (!tile_of_block(rtiles * C, a.cus, blockIdx.x, id, half)) return;
  int rt, ct;
  grouped_tile(id, rtiles, rt, ct, C, row_group(rtiles));
  rt = __builtin_amdgcn_readfirstlane(rt);  // (tile addresses derive from them)
  ct = __builtin_amdgcn_readfirstlane(ct);
  const int i0 = rt * kBM;
  const int sc = __builtin_amdgcn_readfirstlane(ct / a.tg.tps), j = ct - sc * a.tg.tps;
  const int sbeg = (a.bg.c_lo + sc) * a.gm.S;
  const int valid_s = max(0, min(a.gm.S, a.gm.V - sbeg));  // columns of this split
  const int t0 = j * kBN + kChunk * max(half, 0), t1 = t0 + (half < 0 ? kBN : kChunk);  // the tile's, in the split
  if (t0 >= a.bg.S_pad) return;
  const int c0 = sbeg + t0;
  const int c1 = sbeg + min(t1, valid_s);
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave_m(w),
            wn = wave_n(w);
  float4 ri[kMI];  // loaded as in dz_tiles
  const auto load_rows = [&]() {
#pragma unroll
    for (int mi = 0; mi < kTailRows; ++mi) ri[mi] = a.rowinfo[i0 + spread_row(wm, mi, lane)];
  };
  // a tile past the vocabulary runs on W's first row and is written as zeros
  const RowsK A = rows_k_spread(a.hA + (size_t)i0 * a.H, min(n_act - i0, kBM) - 1, a.H);
  const RowsK B = c0 < c1 ? rows_k(a.W + (size_t)c0 * a.H, c1 - 1 - c0, a.H) : rows_k(a.W, 0, a.H);
  // rows whose dz is written: zeros up to a k-block of grad_W's product
  const int rows = min(n_act - i0, kBM), rows_out = (rows + kBK - 1) / kBK * kBK;
  char* stage = reinterpret_cast<char*>(lds);
  int le = lane;  // an opaque copy, see fwd_tiles
  Acc acc;
  acc_zero(acc);
  if (half >= 0 && wn == 1) {
    gemm256<false, false, 0>(A, B, a.H / kBK, acc, lds);
    asm volatile("" : "+v"(le));
  } else {
    gemm_rows(A, B, a.H / kBK, acc, lds, wm, rows, load_rows);
    asm volatile("" : "+v"(le));
#pragma unroll
    for (int mi = kTailRows; mi < kMI; ++mi) ri[mi] = a.rowinfo[i0 + spread_row(wm, mi, le)];
    // staging in LDS as in dz_tiles: 256 rows x 512 bytes, 16-byte unit u of row r at r * 512 + 16 (u ^ (r & 31))
    auto put = [&](int r, int c, const float (&d)[4]) {
      const uint32_t off = 512u * r + 16u * ((c >> 3) ^ (r & 31)) + 8u * ((c >> 2) & 1);
      *reinterpret_cast<uint2*>(stage + off) = make_uint2(pack_bf16x2(d[0], d[1]), pack_bf16x2(d[2], d[3]));
    };
    const auto share = [&](float z, const float4& r) { return minus_share<kTop>(kTop ? z : z * a.scale, r); };
    const int wc0 = t0 + 128 * wn;  // first column of the wave within the split
    const bool full_c = wc0 + 128 <= valid_s;
#pragma unroll
    for (int mi = 0; mi < kMI; ++mi) {
      const int r0 = kBlk * spread_block(wm, mi), r = r0 + le % kBlk;  // the row block's first row, this lane's
      if (r0 >= rows_out) continue;
      const bool rvalid = i0 + r < n_act;
      const int yl = kTop ? __float_as_int(ri[mi].w) - sbeg : -1;  // target column within the split
      const int tl = yl - wc0;
      const bool hit = kTop && tl >= 0 && tl < 128 && ((tl >> 2) & (kLPR - 1)) == row_lane(le);
      if (full_c && r0 + kBlk <= rows && !__builtin_amdgcn_ballot_w64(hit)) {
#pragma unroll
        for (int ni = 0; ni < kNI; ++ni)
#pragma unroll
          for (int q = 0; q < kQL; ++q) {
            float d[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) d[e] = share(acc.c[mi][ni][4 * q + e], ri[mi]);
            put(r, acc_col4(wn, ni, q, le), d);
          }
      } else {
        const float g = kTop ? a.rowg[i0 + r] : 0.f;
#pragma unroll
        for (int ni = 0; ni < kNI; ++ni)
#pragma unroll
          for (int q = 0; q < kQL; ++q) {
            if (t0 + 128 * wn + kBlk * ni + 4 * kLPR * q >= a.bg.S_pad) continue;  // never stored
            const int c = acc_col4(wn, ni, q, le);
            float d[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int vl = t0 + c + e;
              const float x = share(acc.c[mi][ni][4 * q + e], ri[mi]);
              d[e] = rvalid && vl < valid_s ? (kTop && vl == yl ? g + x : x) : 0.f;
            }
            put(r, c, d);
          }
      }
    }
  }
  __syncthreads();
  uint16_t* dzs = a.dZ + (size_t)sc * a.bg.S_pad;
  constexpr int kRowsW = kBM / kWaves;
  const int u = le & 31;
  const int col = t0 + 8 * u;  // column within the split
  if (col < min(t1, a.bg.S_pad)) {
#pragma unroll
    for (int it = 0; it < kRowsW / 2; ++it) {
      const int r = kRowsW * w + 2 * it + (le >> 5);
      if (r >= rows_out) continue;
      const u32x4 v = *reinterpret_cast<const u32x4*>(stage + 512u * r + 16u * (u ^ (r & 31)));
      __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(dzs + (size_t)(i0 + r) * a.bg.ldz + col));
    }
  }
}

// dz at the teacher's tokens of the group: a (q - p) with a = -dL/dloss /
// temperature and p = e(log p) of the forward.  A token in several slots of
// a row has the sum of their q, in slot order, written by the first of them.
// Block kMaxK, one thread per slot, rows strided over the grid.  Scattered
// two-byte stores into dz, 64 a row: 3482 rows 16 us, 257 rows 11.
struct ScatterArgs {
  const int32_t* ids;
  const float* q;         // [T][K], 0 for slots that are not kept
  const float* logp_ids;  // [T][K]
  const float* logits;
  const int32_t* idx;  // NULL: every row of the batch, in place
  const int32_t* n_act;
  const float4* rowinfo;
  int K;
  SplitGeom gm;
  BwdGeom bg;
  uint16_t* dZ;
};

__global__ __launch_bounds__(kMaxK) void distill_scatter(ScatterArgs a) {
  __shared__ int32_t id_s[kMaxK];
  __shared__ float q_s[kMaxK];
  const int k = threadIdx.x, n_act = *a.n_act;
  for (int i = blockIdx.x; i < n_act; i += gridDim.x) {
    const size_t at = (size_t)(a.idx ? a.idx[i] : i) * a.K + k;
    int id = -1;
    if (k < a.K && slot_kept(a.ids[at], a.logits[at])) id = a.ids[at];
    if (id >= a.gm.V) id = -1;
    __syncthreads();
    id_s[k] = id;
    q_s[k] = id >= 0 ? a.q[at] : 0.f;
    __syncthreads();
    if (id < 0) continue;
    const int s = id / a.gm.S - a.bg.c_lo;
    if (s < 0 || s >= a.bg.G) continue;
    bool first = true;
    float q = 0.f;
    for (int j = 0; j < a.K; ++j) {
      const bool same = id_s[j] == id;
      first &= !(same && j < k);
      if (same) q = q + q_s[j];
    }
    if (!first) continue;
    const float p = rlk_exp(a.logp_ids[at]);
    const float d = a.rowinfo[i].y * (q - p);
    const int c = id - (s + a.bg.c_lo) * a.gm.S;
    a.dZ[(size_t)i * a.bg.ldz + (size_t)s * a.bg.S_pad + c] = (uint16_t)pack_bf16x2(d, d);
  }
}

// ---------------------------------------------------------------------------
// Gradients of a group of splits.
//
// grad_h: the sum over the vocabulary is cut into parts of `per` splits each
// (part_splits: by H and V, whatever the batch); a part's sum is one fp32 MFMA
// chain per element, vocabulary ascending (it continues across groups through
// its place in `part`), and grad_h_sum adds the parts in order.  One chain
// over the whole vocabulary leaves most compute units without a grad_h tile
// where rows are few: at 257 rows, H = 4096, V = 151936 its tiles take 1.97
// ms.  (linear_logp_bwd keeps the one chain: its bits are its contract.)
// Four parts there: both gradients of that batch in 0.98 ms, of 4096 rows
// (3482 active) in 6.63 ms with grad_h_sum; two parts 1.68 and 6.49, eight
// 0.99 and 6.73 (the parts' sums pass through HBM).  3482 active rows: 6.33 -
// 6.55 ms for 8.67 TFLOP (1.32 - 1.37 PFLOP/s), bound by MFMAs and by the
// transposing reads of both products' operands.
// ---------------------------------------------------------------------------
constexpr int kMaxParts = kNSplit;

struct PartGradHArgs {
  const uint16_t* dZ;
  const uint16_t* W;
  int H;
  SplitGeom gm;
  BwdGeom bg;
  int n_tiles;         // 256-column tiles of H
  int per;             // splits of a part
  int part0, parts;    // parts of the group: part0 .. part0 + parts - 1
  int cus;
  float* part;         // [part][T][H], rows in active order; NULL: not wanted
  size_t part_stride;  // T * H
};

// At most a tile for every fourth compute unit (up to 256 rows): they are cut
// into their two 128-column halves.  Both gradients at 256 rows: 0.96 -> 0.85
// ms (H = 4096), 0.48 -> 0.42 (2048).  A half's loads are a tile's, and twice
// the tiles cut so cost: 257 rows 0.98 -> 1.17, 512 rows 1.15 -> 1.38.
__device__ __forceinline__ bool cut_tiles(int n, int cus) { return 4 * n <= cus; }

// kCont: the group starts inside its (one) part.
template <bool kCont>
__device__ __forceinline__ void gradh_part_tile(const PartGradHArgs& a, int id, int half, int rtiles, int n_act,
                                                u32x4* lds) {
  const int per = rtiles * a.n_tiles;
  const int q = __builtin_amdgcn_readfirstlane(id / per);  // part within the group
  int rt, nt;
  grouped_tile(id - q * per, rtiles, rt, nt, a.n_tiles, row_group(rtiles));
  rt = __builtin_amdgcn_readfirstlane(rt);  // (tile addresses derive from them)
  nt = __builtin_amdgcn_readfirstlane(nt);
  const int i0 = rt * kBM, n0 = nt * kBN + 128 * max(half, 0), n1 = min(n0 + (half < 0 ? kBN : 128), a.H);
  if (n0 >= n1) return;
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave_m(w),
            wn = wave_n(w);
  float* part = a.part + (size_t)(a.part0 + q) * a.part_stride;
  Acc acc;
  acc_zero(acc);
  if (kCont) {  // (clamped addresses outside the problem; never stored)
#pragma unroll
    for (int mi = 0; mi < kMI; ++mi) {
      const float* src = part + (size_t)min(i0 + acc_row(wm, mi, lane), n_act - 1) * a.H;
#pragma unroll
      for (int ni = 0; ni < kNI; ++ni)
#pragma unroll
        for (int p = 0; p < kQL; ++p) {
          const float4 v = *reinterpret_cast<const float4*>(src + min(n0 + acc_col4(wn, ni, p, lane), a.H - 4));
          acc.c[mi][ni][4 * p] = v.x;
          acc.c[mi][ni][4 * p + 1] = v.y;
          acc.c[mi][ni][4 * p + 2] = v.z;
          acc.c[mi][ni][4 * p + 3] = v.w;
        }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  // the accumulators enter the engine in accumulator registers (see gradh_tile)
#pragma unroll
  for (int mi = 0; mi < kMI; ++mi)
#pragma unroll
    for (int ni = 0; ni < kNI; ++ni) asm volatile("" : "+a"(acc.c[mi][ni]));
  const int s0 = q * a.per, splits = min(a.per, a.bg.G - s0);  // of the group
  // (a lone row tile does not fetch its padding: both gradients of 130 rows of
  // H = 4096 0.83 -> 0.72 ms; a second tile's gains nothing: 257 rows 0.97 -> 0.98)
  const RowsK A = rows_k(a.dZ + (size_t)i0 * a.bg.ldz + (size_t)s0 * a.bg.S_pad, rtiles > 1 ? kBM - 1 : n_act - 1,
                         a.bg.ldz);
  WRowsMN B;
  B.base = reinterpret_cast<const char*>(a.W + n0);
  B.H = a.H;
  B.S = a.gm.S;
  B.kbps = a.bg.S_pad / kBK;
  B.rcp = ((uint64_t(1) << 32) + (uint64_t)B.kbps - 1) / (uint64_t)B.kbps;
  B.c_lo = a.bg.c_lo + s0;
  B.V = a.gm.V;
#pragma unroll
  for (int i = 0; i < kDma; ++i) {
    B.col2[i] = 2 * (min(n0 + dma_mn_piece(dma_mn_krow(i)) * 8, n1 - 8) - n0);
    B.krow[i] = (uint32_t)dma_mn_krow(i);
  }
  if (half >= 0 && wn == 1) {
    gemm256<false, true, 0>(A, B, splits * B.kbps, acc, lds);
    return;
  }
  gemm256<false, true>(A, B, splits * B.kbps, acc, lds);
#pragma unroll
  for (int mi = 0; mi < kMI; ++mi) {
    const int i = i0 + acc_row(wm, mi, lane);
    if (i >= n_act) continue;
#pragma unroll
    for (int ni = 0; ni < kNI; ++ni)
#pragma unroll
      for (int p = 0; p < kQL; ++p) {
        if (n0 + 128 * wn + kBlk * ni + 4 * kLPR * p >= a.H) continue;  // wave-uniform
        const AccBlk& c = acc.c[mi][ni];
        *reinterpret_cast<float4*>(part + (size_t)i * a.H + n0 + acc_col4(wn, ni, p, lane)) =
            make_float4(c[4 * p], c[4 * p + 1], c[4 * p + 2], c[4 * p + 3]);
      }
  }
}

// gradw_tile (rlk_kernels.h) with a bf16 grad_W, each fp32 sum rounded once.
// The tile goes through LDS as dz does: straight from the accumulators a
// store would write 32-byte pieces of 16 rows.
__device__ __forceinline__ void gradw_bf16_tile(const GradWArgs& a, int id, int n_act, u32x4* lds) {
  int nt, vt;
  grouped_tile(id, a.n_tiles, nt, vt, a.bg.G * a.tps, min(kGradWGroup, a.n_tiles));
  nt = __builtin_amdgcn_readfirstlane(nt);  // (tile addresses derive from them)
  vt = __builtin_amdgcn_readfirstlane(vt);
  const int sc = __builtin_amdgcn_readfirstlane(vt / a.tps), j = vt - sc * a.tps;
  const int sbeg = (a.bg.c_lo + sc) * a.gm.S;
  const int valid_s = max(0, min(a.gm.S, a.gm.V - sbeg));
  const int v0 = j * kBM;  // within the split
  if (v0 >= valid_s) return;
  const int n0 = nt * kBN;
  const int tid = threadIdx.x;
  const ColsMN A = cols_mn(a.dZ + (size_t)sc * a.bg.S_pad, v0, a.bg.S_pad, a.bg.ldz);
  const ColsMN B = cols_mn(a.hA, n0, a.H, a.H);
  Acc acc;
  acc_zero(acc);
#pragma unroll
  for (int mi = 0; mi < kMI; ++mi)
#pragma unroll
    for (int ni = 0; ni < kNI; ++ni) asm volatile("" : "+a"(acc.c[mi][ni]));
  if (n_act > 0) gemm256<true, true>(A, B, (n_act + kBK - 1) / kBK, acc, lds);
  int le = tid & 63;  // an opaque copy, see fwd_tiles
  asm volatile("" : "+v"(le));
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave_m(w), wn = wave_n(w);
  char* stage = reinterpret_cast<char*>(lds);  // as in dz_tiles
#pragma unroll
  for (int mi = 0; mi < kMI; ++mi) {
    const int r = acc_row(wm, mi, le);
#pragma unroll
    for (int ni = 0; ni < kNI; ++ni)
#pragma unroll
      for (int q = 0; q < kQL; ++q) {
        const AccBlk& c = acc.c[mi][ni];
        const int col = acc_col4(wn, ni, q, le);
        *reinterpret_cast<uint2*>(stage + 512u * r + 16u * ((col >> 3) ^ (r & 31)) + 8u * ((col >> 2) & 1)) =
            make_uint2(pack_bf16x2(c[4 * q], c[4 * q + 1]), pack_bf16x2(c[4 * q + 2], c[4 * q + 3]));
      }
  }
  __syncthreads();
  constexpr int kRowsW = kBM / kWaves;
  const int u = le & 31, col = n0 + 8 * u;
  if (col < a.H) {
    uint16_t* out = reinterpret_cast<uint16_t*>(a.grad_W) + (size_t)sbeg * a.H + col;
#pragma unroll
    for (int it = 0; it < kRowsW / 2; ++it) {
      const int r = kRowsW * w + 2 * it + (le >> 5);
      if (v0 + r < valid_s)
        *reinterpret_cast<u32x4*>(out + (size_t)(v0 + r) * a.H) =
            *reinterpret_cast<const u32x4*>(stage + 512u * r + 16u * (u ^ (r & 31)));
    }
  }
}

// The group's grad_h tiles (long chains, first) and grad_W tiles in one
// launch, as in grad_tiles.
template <bool kBf16, bool kCont>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(RLK_WAVES / 4, RLK_WAVES / 4))) void part_grad_tiles(
    PartGradHArgs ha, GradWArgs wa) {
  __shared__ u32x4 lds[kLdsU4];
  const int n_act = __builtin_amdgcn_readfirstlane(*wa.n_act);
  const int rtiles = (n_act + kBM - 1) / kBM;
  const int nt = ha.part ? rtiles * ha.n_tiles * ha.parts : 0;
  const bool cut = cut_tiles(nt, ha.cus);
  const int nh = cut ? 2 * nt : nt;
  const int nh_blocks = 8 * ((nh + 7) >> 3);
  const int bid = blockIdx.x;
  if (bid < nh_blocks) {
    const int id = xcd_tile(nh, bid);
    if (id >= 0) gradh_part_tile<kCont>(ha, cut ? id >> 1 : id, cut ? id & 1 : -1, rtiles, n_act, lds);
    return;
  }
  const int nw = wa.grad_W ? wa.n_tiles * wa.bg.G * wa.tps : 0;
  const int id = xcd_tile(nw, bid - nh_blocks);
  if (id < 0) return;
  if constexpr (kBf16) gradw_bf16_tile(wa, id, n_act, lds);
  else gradw_tile(wa, id, n_act, lds);
}

#if RLK_MFMA == 16
// ---------------------------------------------------------------------------
// Gradients of few rows.  Both are bound by W's traffic (grad_h reads it,
// grad_W has its size), and the 256 x 256 tiles leave that far off: 64 of
// them for grad_h at H = 4096, each as long as its part, and for grad_W one
// tile at a time per compute unit, loads, MFMAs and stores in turn.  Together
// they took 0.92 ms at 64 rows of H = 4096; the kernels below take 0.52.
// ---------------------------------------------------------------------------
// Eight k of one column for each lane, from two transposing reads: `base` is
// where the lane's 4 columns of k-row 8 (l / 16) + (l % 16) / 4 lie, kr the
// bytes of 4 k-rows (which keep the swizzle; see frag_at).
__device__ __forceinline__ bf16x8 tr_frag(const char* base, uint32_t kr4) {
  const lds_bf16x4* p0 = (const lds_bf16x4*)base;
  const lds_bf16x4* p1 = (const lds_bf16x4*)(base + kr4);
  const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(const_cast<lds_bf16x4*>(p0));
  const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(const_cast<lds_bf16x4*>(p1));
  return bf16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
}

// grad_h of up to 128 rows: a block takes 64 columns of one part and streams
// the part's W through a ring of kSlots LDS stages of 64 vocabulary rows
// (8 KB, and the dz block they meet), kSlots - 1 in flight.  Its four waves
// take 16 columns each, or (above 64 rows, where reading dz from LDS counts)
// 32 columns and half of the rows.  The same chains as gradh_part_tile.
// Bound by W's way from HBM up to 64 rows: 257 - 274 us at H = 4096 (4.5 - 4.8
// TB/s), 126 - 140 at 2048; above, by reading dz from LDS: 354 and 181 at 128
// rows.  A form for 256 rows took 544.
// A stage: W as 64 k-rows of 128 bytes, 32-byte units xor-ed with
// (row >> 1 & 1) + 2 (row >> 3 & 1): the 8 k-rows of a transposing pass fall
// on distinct banks; dz as rows of 128 bytes in the engine's K layout (slot_k).
struct FewGradHArgs {
  const uint16_t* dZ;  // 16 kRB rows at least
  const uint16_t* W;
  const int32_t* n_act;
  int H;
  SplitGeom gm;
  BwdGeom bg;
  int per, part0, parts;
  float* part;         // as in PartGradHArgs
  size_t part_stride;
};

template <int kRB, bool kCont>
__global__ __launch_bounds__(256) void few_grad_h(FewGradHArgs a) {
  constexpr int kRows = 16 * (kRB < 2 ? 2 : kRB);  // dz rows of a stage (32 at least: every wave loads as many)
  constexpr uint32_t kWBytes = 64 * 128, kStage = kWBytes + kRows * 128;
  constexpr int kSlots = (160 << 10) / kStage, kLoads = 2 + kRows / 32;
  static_assert((kSlots - 2) * kLoads < 64, "vmcnt");
  constexpr int kC = kRB >= 8 ? 2 : 1, kR = kRB / kC;  // 16-column and 16-row blocks of a wave
  __shared__ u32x4 lds[kSlots * kStage / 16];
  const int n_act = __builtin_amdgcn_readfirstlane(*a.n_act);
  const int n_tiles = a.H / 64;
  const int id = n_act > 0 ? xcd_tile(n_tiles * a.parts, blockIdx.x) : -1;
  if (id < 0) return;
  const int q = __builtin_amdgcn_readfirstlane(id / n_tiles), n0 = 64 * (id - q * n_tiles);
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, rl = lane >> 4;
  const int wc = kC == 1 ? 16 * w : 32 * (w & 1), wr = kC == 1 ? 0 : 16 * kR * (w >> 1);  // first column, row
  const int s0 = q * a.per, splits = min(a.per, a.bg.G - s0), kbps = a.bg.S_pad / kBK;
  const int nk = splits * kbps;
  // direct loads of this lane: W rows 16 w + 8 i + lane / 8, dz rows 8 (w + 4 i) + lane / 8
  uint32_t w_row[2], w_col[2], dz_off[kRows / 32];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = 16 * w + 8 * i + (lane >> 3), p = lane & 7;
    const int f = ((row >> 1) & 1) | ((row >> 2) & 2);
    w_row[i] = row;
    w_col[i] = 2 * n0 + 16 * ((((p >> 1) ^ f) << 1) | (p & 1));
  }
#pragma unroll
  for (int i = 0; i < kRows / 32; ++i) {
    const int row = 8 * (w + 4 * i) + (lane >> 3);
    dz_off[i] = 2u * ((uint32_t)row * (uint32_t)a.bg.ldz) + 16u * ((lane & 7) ^ ((row >> 1) & 7));
  }
  const char* dz = reinterpret_cast<const char*>(a.dZ + (size_t)s0 * a.bg.S_pad);
  const uint32_t lds0 = lds_addr(lds);
  int l_sc = 0, l_kb = 0, l_kt = 0;  // the stage loaded next: split, k-block of it, k-block of the part
  const auto load = [&](int slot) {
    const uint32_t m0 = lds0 + kStage * slot;
    const int r0 = min((a.bg.c_lo + s0 + l_sc) * a.gm.S + kBK * l_kb, a.gm.V - 1);
    const uint32_t last = (uint32_t)(a.gm.V - 1 - r0);  // (rows past it meet dz = 0)
    const char* wb = reinterpret_cast<const char*>(a.W) + (size_t)r0 * (2 * a.H);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      dma16(wb, min(w_row[i], last) * (uint32_t)(2 * a.H) + w_col[i], m0 + 1024u * (2 * w + i));
#pragma unroll
    for (int i = 0; i < kRows / 32; ++i)
      dma16(dz + (size_t)l_kt * (2 * kBK), dz_off[i], m0 + kWBytes + 1024u * (w + 4 * i));
    if (l_kt + 1 < nk) {  // (past the end: the last stage again, into a free slot)
      ++l_kt;
      if (++l_kb == kbps) {
        l_kb = 0;
        ++l_sc;
      }
    }
  };
  AccBlk acc[kR][kC];
  float* part = a.part + (size_t)(a.part0 + q) * a.part_stride + n0 + wc + 4 * rl;
#pragma unroll
  for (int m = 0; m < kR; ++m)
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      acc[m][c] = AccBlk{};
      if (kCont) {
        const float4 v = *reinterpret_cast<const float4*>(part + (size_t)min(wr + 16 * m + r16, n_act - 1) * a.H + 16 * c);
        acc[m][c] = AccBlk{v.x, v.y, v.z, v.w};
      }
    }
  // this lane's W fragments within a stage: k step kk 32 k-rows further (the swizzle stays, as for k-rows + 4)
  const int krow = 8 * rl + (r16 >> 2), f = ((krow >> 1) & 1) | ((krow >> 2) & 2);
  uint32_t w_at[kC];
#pragma unroll
  for (int c = 0; c < kC; ++c) w_at[c] = 128u * krow + 32u * (((wc >> 4) + c) ^ f) + 8u * (r16 & 3);
  if (kCont) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // (the loads below are counted)
#pragma unroll 1
  for (int i = 0; i + 1 < kSlots; ++i) load(i);
  int slot = 0;
#pragma unroll 1
  for (int kt = 0; kt < nk; ++kt) {
    loads_then_barrier<(kSlots - 2) * kLoads>();
    load(slot == 0 ? kSlots - 1 : slot - 1);  // the slot read last time
    const char* st = reinterpret_cast<const char*>(lds) + kStage * slot;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      bf16x8 y[kC];
#pragma unroll
      for (int c = 0; c < kC; ++c) y[c] = tr_frag(st + w_at[c] + 128u * 32 * kk, 128u * 4);
#pragma unroll
      for (int m = 0; m < kR; ++m) {
        const bf16x8 x = __builtin_bit_cast(
            bf16x8, *reinterpret_cast<const u32x4*>(st + kWBytes + 16u * slot_k(wr + 16 * m + r16, 4 * kk + rl)));
#pragma unroll
        for (int c = 0; c < kC; ++c) acc[m][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(y[c], x, acc[m][c], 0, 0, 0);
      }
    }
    slot = slot + 1 == kSlots ? 0 : slot + 1;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // nothing is loaded into LDS past the block's end
#pragma unroll
  for (int m = 0; m < kR; ++m) {
    const int t = wr + 16 * m + r16;
    if (t >= n_act) continue;
#pragma unroll
    for (int c = 0; c < kC; ++c)
      *reinterpret_cast<float4*>(part + (size_t)t * a.H + 16 * c) =
          make_float4(acc[m][c][0], acc[m][c][1], acc[m][c][2], acc[m][c][3]);
  }
}

// grad_W of up to 64 kKB rows: a block takes a chunk of 128 vocabulary rows
// and all of H, 128 columns at a time; its four waves take 64 x 64 of that
// each.  dz's fragments are read once, through LDS, and stay in registers
// (32 kKB of them); h comes in stages of 64 rows x 128 columns, two LDS slots.
// Block b starts with the b-th 128 columns: rows of grad_W lie 2 H or 4 H bytes
// apart, and blocks in step would all write to the same few memory channels.
// Several blocks per compute unit overlap one's stores with another's loads
// and MFMAs.  The same chains as gradw_tile (rows ascending).
// Bound by grad_W's stores: bf16, up to 128 rows, 250 us at H = 4096 (5.0 TB/s;
// 300 with all blocks starting at column 0), 111 - 134 at 2048.  A form for
// 256 rows took 480 beside the tiles' 950 for both gradients, of which grad_h
// alone is 745.
// A lane's columns of an MFMA block are free to choose, four by four.  For a
// bf16 grad_W block n of a wave's four takes, in lanes r = l / 16, columns
// 32 (n / 2) + 8 r + 4 (n % 2) .. + 3: two blocks make 8 consecutive columns
// of a lane and 32 (64 bytes) of a row's four lanes, one store.
// LDS: rows (k) of 256 bytes, their 32-byte units xor-ed with
// (row & 3) + 4 (row >> 3 & 1), as in mn_pos; with the columns so chosen h's
// 64-byte units with row & 3 instead (two lanes then meet at a bank, the
// least there is: each lane of a pass reads the same half of a piece).
struct FewGradWArgs {
  const uint16_t* dZ;
  const uint16_t* hA;  // zero rows past the active ones, to a multiple of 64 at least
  const int32_t* n_act;  // <= 64 kKB
  int H;
  SplitGeom gm;
  BwdGeom bg;
  void* grad_W;
};

template <int kKB, bool kBf16>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2))) void few_grad_w(FewGradWArgs a) {
  constexpr uint32_t kTile = 64 * 256;
  __shared__ u32x4 lds[2 * kTile / 16];
  const int s = blockIdx.x / a.gm.cps, j = blockIdx.x - s * a.gm.cps;
  const int sbeg = (a.bg.c_lo + s) * a.gm.S, v0 = kChunk * j;
  const int rows = min(kChunk, min(a.gm.S, a.gm.V - sbeg) - v0);  // vocabulary rows of the chunk
  if (rows <= 0) return;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, rl = lane >> 4, wv = 64 * (w & 1), wc = 64 * (w >> 1);
  const int n_act = __builtin_amdgcn_readfirstlane(*a.n_act);
  const int kb = (n_act + 63) / 64;  // k-blocks (none: grad_W is zero)
  const uint32_t lds0 = lds_addr(lds);
  // direct loads: k-rows 16 w + 4 i + lane / 16 of a 64-row tile, piece lane % 16
  uint32_t dz_off[4], h_off[4];
  int h_piece[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 16 * w + 4 * i + rl, p = r16;
    const int f = (row & 3) | ((row >> 1) & 4);
    const int pd = (((p >> 1) ^ f) << 1) | (p & 1);
    dz_off[i] = 2u * ((uint32_t)row * (uint32_t)a.bg.ldz + (uint32_t)min(v0 + 8 * pd, a.bg.S_pad - 8));
    h_off[i] = 2u * (uint32_t)row * (uint32_t)a.H;
    h_piece[i] = kBf16 ? p ^ ((row & 3) << 2) : pd;
  }
  const char* dz = reinterpret_cast<const char*>(a.dZ + (size_t)s * a.bg.S_pad);
  const char* hb = reinterpret_cast<const char*>(a.hA);
  // this lane's fragments: k-row 8 rl + r16 / 4, k step kk 32 rows further
  const int krow = 8 * rl + (r16 >> 2), q4 = r16 & 3, f_row = (krow & 3) | ((krow >> 1) & 4);
  bf16x8 x[kKB][2][4];
#pragma unroll
  for (int k = 0; k < kKB; ++k) {
    if (k < kb) {
      const uint32_t slot = lds0 + kTile * (k & 1);
#pragma unroll
      for (int i = 0; i < 4; ++i) dma16(dz + (size_t)k * 128 * a.bg.ldz, dz_off[i], slot + 1024u * (4 * w + i));
      loads_then_barrier<0>();
#pragma unroll
      for (int kk = 0; kk < 2; ++kk)
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const uint32_t at = 256u * (krow + 32 * kk) + 32u * (((wv >> 4) + m) ^ f_row) + 8u * q4;
          x[k][kk][m] = tr_frag(reinterpret_cast<const char*>(lds) + kTile * (k & 1) + at, 256u * 4);
        }
    } else {
#pragma unroll
      for (int kk = 0; kk < 2; ++kk)
#pragma unroll
        for (int m = 0; m < 4; ++m) x[k][kk][m] = bf16x8{};
    }
  }
  loads_then_barrier<0>();  // every wave has its fragments: the slots are free
  const int steps = (a.H + 127) / 128;
  const int first = (int)blockIdx.x % steps;
  int l_n = first, l_k = 0;
  const auto load = [&](uint32_t slot) {
    const char* base = hb + (size_t)l_k * 128 * a.H;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      dma16(base, h_off[i] + 2u * (uint32_t)min(128 * l_n + 8 * h_piece[i], a.H - 8), slot + 1024u * (4 * w + i));
    if (++l_k >= kb) {
      l_k = 0;
      l_n = l_n + 1 < steps ? l_n + 1 : 0;
    }
  };
  load(lds0);
  using Out = std::conditional_t<kBf16, uint16_t, float>;
  Out* out = reinterpret_cast<Out*>(a.grad_W) + (size_t)(sbeg + v0) * a.H;
  uint32_t slot = 0;
#pragma unroll 1
  for (int i = 0, n = first; i < steps; ++i, n = n + 1 < steps ? n + 1 : 0) {
    AccBlk acc[4][4];
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int b = 0; b < 4; ++b) acc[m][b] = AccBlk{};
#pragma unroll
    for (int k = 0; k < kKB; ++k) {
      if (k >= kb) break;
      loads_then_barrier<0>();
      load(lds0 + (slot ^ kTile));
      const char* th = reinterpret_cast<const char*>(lds) + slot;
#pragma unroll
      for (int kk = 0; kk < 2; ++kk)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          // this lane's four columns of block b, k-row krow
          const int c64 = wc >> 6;
          const uint32_t in_row = kBf16 ? 16u * ((8 * c64 + 4 * (b >> 1) + q4) ^ ((krow & 3) << 2)) + 8u * (b & 1)
                                        : 32u * ((4 * c64 + b) ^ f_row) + 8u * q4;
          const bf16x8 y = tr_frag(th + 256u * (krow + 32 * kk) + in_row, 256u * 4);
#pragma unroll
          for (int m = 0; m < 4; ++m)
            acc[m][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(y, x[k][kk][m], acc[m][b], 0, 0, 0);
        }
      slot ^= kTile;
    }
    const int c0 = 128 * n + wc;
    if (c0 >= a.H) continue;  // (H % 128 == 64: the last step's second half)
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int v = wv + 16 * m + r16;
      if (v >= rows) continue;
      if constexpr (kBf16) {
        Out* to = out + (size_t)v * a.H + c0 + 8 * rl;
#pragma unroll
        for (int b = 0; b < 4; b += 2)
          *reinterpret_cast<u32x4*>(to + 16 * b) =
              u32x4{pack_bf16x2(acc[m][b][0], acc[m][b][1]), pack_bf16x2(acc[m][b][2], acc[m][b][3]),
                    pack_bf16x2(acc[m][b + 1][0], acc[m][b + 1][1]), pack_bf16x2(acc[m][b + 1][2], acc[m][b + 1][3])};
      } else {
        Out* to = out + (size_t)v * a.H + c0 + 4 * rl;
#pragma unroll
        for (int b = 0; b < 4; ++b)
          *reinterpret_cast<float4*>(to + 16 * b) = make_float4(acc[m][b][0], acc[m][b][1], acc[m][b][2], acc[m][b][3]);
      }
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // nothing is loaded into LDS past the block's end
}
#endif  // RLK_MFMA == 16

// grad_h[idx[i]] = the parts' sum, left to right, rounded to bf16 once; zero
// rows for inactive rows.  Block b takes active row b and row b of the batch
// (idx NULL: they are the same).  HBM: 3482 rows of four parts, H = 4096 (0.26
// GB), 57 us.
__global__ __launch_bounds__(256) void grad_h_sum(const float* __restrict__ part, size_t part_stride, int parts,
                                                  const int32_t* __restrict__ idx,
                                                  const int32_t* __restrict__ n_act_p, const int32_t* __restrict__ act,
                                                  int ignore_index, int T, int H, uint16_t* __restrict__ grad_h) {
  const int n_act = *n_act_p;
  for (int i = blockIdx.x; i < T; i += gridDim.x) {
    const bool off = act[i] == ignore_index;
    if (off)
      for (int c = 4 * threadIdx.x; c < H; c += 1024)
        *reinterpret_cast<uint2*>(grad_h + (size_t)i * H + c) = make_uint2(0u, 0u);
    if (i >= n_act || (!idx && off)) continue;
    uint16_t* out = grad_h + (size_t)(idx ? idx[i] : i) * H;
    for (int c = 4 * threadIdx.x; c < H; c += 1024) {
      const float* src = part + (size_t)i * H + c;
      float4 s = *reinterpret_cast<const float4*>(src);
      constexpr int kAhead = 4;
      for (int q0 = 1; q0 < parts; q0 += kAhead) {
        float4 v[kAhead];
#pragma unroll
        for (int q = 0; q < kAhead; ++q)
          if (q0 + q < parts) v[q] = *reinterpret_cast<const float4*>(src + (q0 + q) * part_stride);
#pragma unroll
        for (int q = 0; q < kAhead; ++q)
          if (q0 + q < parts) s = make_float4(s.x + v[q].x, s.y + v[q].y, s.z + v[q].z, s.w + v[q].w);
      }
      *reinterpret_cast<uint2*>(out + c) = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
    }
  }
}

}  // namespace vocab
}  // namespace rlk
