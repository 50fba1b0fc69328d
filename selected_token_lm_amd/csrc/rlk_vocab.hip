// The operators of include/rlk/vocab_ops.h: their kernels, on the eight-wave
// tile engine, and their C entry points.  Everything is enqueued on the
// caller's stream; nothing here allocates device memory or synchronises.
#ifdef RLK_WAVES
#undef RLK_WAVES
#endif
#define RLK_WAVES 8
#define RLK_ENGINE_W8
#define RLK_ENGINE_PARTS
#include "rlk/vocab_ops.h"

#include "rlk_host.h"
#include "rlk_rows.h"
#include "rlk_vocab.h"

namespace rlk {
namespace vocab {

// Zeroes n16 16-byte words (T == 0: grad_W).
__global__ __launch_bounds__(256) void zero_bytes(u32x4* p, int64_t n16) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n16; i += (int64_t)gridDim.x * 256)
    p[i] = u32x4{0u, 0u, 0u, 0u};
}

}  // namespace vocab
}  // namespace rlk

namespace {

using namespace rlk::vocab;
static_assert(RLK_MAX_K == kMaxK, "the header's limit");
static_assert(rlk::kThreads == rlk::kThreadsW8, "eight-wave kernels");

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Consecutive pieces of a workspace, each at a multiple of 256 bytes.
struct Pieces {
  size_t total = 0;
  size_t take(size_t bytes) {
    const size_t at = total;
    total = align256(total + bytes);
    return at;
  }
};

inline int64_t padded_rows(int64_t T) { return ceil_div(std::max<int64_t>(T, 1), rlk::kBM) * rlk::kBM; }

// Few rows: every logit of the batch is kept (in fp32, within the budget).
#if RLK_MFMA == 16
inline int64_t few_ldz(int64_t V) { return rlk::kNSplit * geom_of(V).cps * rlk::kChunk; }
inline bool few_rows(int64_t T, int64_t V) { return T <= kFewRows && 4 * T * few_ldz(V) <= dz_budget_bytes(); }
#else
inline int64_t few_ldz(int64_t) { return 0; }
inline bool few_rows(int64_t, int64_t) { return false; }
#endif

// linear_logp_top, forward: G splits of logits at a time.
struct TopFwdWs {
  size_t idx, yA, n_act, zt, hA, rec, rec_u, z, best, total;
  int64_t T_pad, G, ldz;
};

inline TopFwdWs top_fwd_layout(int64_t T, int64_t H, int64_t V, int64_t K) {
  const Geom g = geom_of(V);
  TopFwdWs w;
  w.T_pad = padded_rows(T);
  w.G = rlk::kNSplit;
  if (K > 0) {
    const int64_t per_split = 4 * T * g.cps * rlk::kChunk, budget = dz_budget_bytes();
    while (w.G > 1 && w.G * per_split > budget) w.G /= 2;
  }
  w.ldz = w.G * g.cps * rlk::kChunk;
  Pieces p;
  w.idx = p.take(sizeof(int32_t) * T);
  w.yA = p.take(sizeof(int32_t) * T);
  w.n_act = p.take(sizeof(int32_t));
  w.zt = p.take(sizeof(float) * T);
  w.hA = p.take(2 * (size_t)w.T_pad * H);
  const size_t records = (size_t)rlk::kNSplit * g.cps * T;
  w.rec = p.take(sizeof(float2) * records);
  w.rec_u = p.take(sizeof(float) * records);
  w.z = p.take(K > 0 || few_rows(T, V) ? sizeof(float) * (size_t)T * w.ldz : 0);
  w.best = p.take(w.G < rlk::kNSplit ? sizeof(uint64_t) * (size_t)T * K : 0);
  w.total = p.total;
  return w;
}

struct DistillFwdWs {
  size_t act, idx, n_act, hA, rec, off, ent, z_ids, z, total;
  int64_t T_pad;
};

inline DistillFwdWs distill_fwd_layout(int64_t T, int64_t H, int64_t V, int64_t K) {
  const Geom g = geom_of(V);
  DistillFwdWs w;
  w.T_pad = padded_rows(T);
  Pieces p;
  w.act = p.take(sizeof(int32_t) * T);
  w.idx = p.take(sizeof(int32_t) * T);
  w.n_act = p.take(sizeof(int32_t));
  w.hA = p.take(2 * (size_t)w.T_pad * H);
  w.rec = p.take(sizeof(float2) * (size_t)rlk::kNSplit * g.cps * T);
  w.off = p.take(sizeof(int32_t) * (size_t)(w.T_pad / kBucketRows) * (rlk::kNSplit * ceil_div(g.S, rlk::kBN) + 1));
  w.ent = p.take(sizeof(uint32_t) * (size_t)w.T_pad * K);
  w.z_ids = p.take(sizeof(float) * (size_t)T * K);
  w.z = p.take(few_rows(T, V) ? sizeof(float) * (size_t)T * few_ldz(V) : 0);
  w.total = p.total;
  return w;
}

// Splits of one of grad_h's parts: 32 / parts.  grad_h's bits depend on them,
// so they go by H and V alone.  Parts are work items, so narrow heads want more
// of them: 256 blocks of 64 columns, one for each of the part's units, are 4
// parts at H = 4096 and 32 at 512.  Their sums pass through HBM (P T H floats
// beside a product of 2 T H V), so a part has 4096 columns at least, four
// parts aside.  Both sides of that border, a backward with both gradients in
// us at T = 32, 300, 2000: V = 132000 in 16 and 32 parts at H = 512 129, 260,
// 884 and 125, 228, 891, at H = 256 105, 213, 583 and 92, 156, 615; V = 66000
// in 8 and 16 at H = 512 95, 174, 453 and 82, 135, 481; V = 33000 in 4 and 8
// 80, 152, 257 and 66, 103, 252 (in 16 60, 86, 272; in 32 59, 86, 309).
constexpr int64_t kPartColumns = 4096;
int part_splits(int64_t H, int64_t V) {
  int parts = 4;
  while (parts < kMaxParts && 2 * parts * H <= 256 * 64 && 2 * parts * kPartColumns <= V) parts *= 2;
  return rlk::kNSplit / parts;
}

// Both backwards: G splits of dz at a time, grad_h's parts, and (distill,
// K > 0) the teacher's rows.
struct SoftBwdWs {
  size_t idx, n_act, rowinfo, rowg, hA, dZ, part, act, q, total;
  int64_t T_pad, S_pad, G;
};

inline SoftBwdWs soft_bwd_layout(int64_t T, int64_t H, int64_t V, int64_t K) {
  const BwdWs b = bwd_layout(T, H, V);
  SoftBwdWs w;
  w.T_pad = b.T_pad;
  w.S_pad = b.S_pad;
  w.G = b.G;
  Pieces p;
  w.idx = p.take(sizeof(int32_t) * T);
  w.n_act = p.take(sizeof(int32_t));
  w.rowinfo = p.take(16 * (size_t)w.T_pad);
  w.rowg = p.take(sizeof(float) * w.T_pad);
  w.hA = p.take(2 * (size_t)w.T_pad * H);
  w.dZ = p.take(2 * (size_t)w.T_pad * w.G * w.S_pad);
  w.part = p.take(sizeof(float) * (size_t)(rlk::kNSplit / part_splits(H, V)) * T * H);
  w.act = p.take(K > 0 ? sizeof(int32_t) * T : 0);
  w.q = p.take(sizeof(float) * (size_t)T * K);
  w.total = p.total;
  return w;
}

template <class T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

// Rows: the row kernels take up to 128 threads each, 2^31 - 1 to a launch.
constexpr int64_t kMaxRows = int64_t(1) << 23;

inline rlk_status check_sizes(int64_t T, int64_t H, int64_t V, int64_t K, int64_t least_k) {
  if (T < 0 || T > kMaxRows) return fail(RLK_ERR_BAD_SHAPE, "T=%lld out of [0, 2^23]", (long long)T);
  if (H <= 0 || H > kMaxH || H % 64 != 0)
    return fail(RLK_ERR_BAD_SHAPE, "H=%lld must be a positive multiple of 64 up to 65536", (long long)H);
  if (V <= 0 || V > kMaxV) return fail(RLK_ERR_BAD_SHAPE, "V=%lld out of [1, 8000000]", (long long)V);
  if (K < least_k || K > kMaxK)
    return fail(RLK_ERR_BAD_SHAPE, "K=%lld out of [%lld, %d]", (long long)K, (long long)least_k, kMaxK);
  return RLK_OK;
}

// 1 / temperature; the kernels multiply by it.
inline rlk_status check_temperature(float t, float* scale) {
  *scale = 1.f / t;
  if (!(t > 0.f) || !(t <= 3.402823466e38f) || !(*scale > 0.f && *scale <= 3.402823466e38f))
    return fail(RLK_ERR_BAD_ARG, "temperature=%g must be positive and finite, and so its reciprocal", (double)t);
  return RLK_OK;
}

inline rlk::SplitGeom split_geom(int64_t V) {
  const Geom g = geom_of(V);
  rlk::SplitGeom gm;
  gm.V = (int)g.V;
  gm.S = (int)g.S;
  gm.cps = (int)g.cps;
  gm.s0 = 0;
  gm.vocab_start = 0;
  return gm;
}

// The last split that holds columns.
inline int last_split(const rlk::SplitGeom& gm) { return (gm.V - 1) / gm.S; }

// Blocks for up to n tiles dealt by tile_of_block.
inline int64_t tile_blocks(int64_t n, int cus) { return 8 * ceil_div(n + cus / 2, 8); }
// (tile_of_block deals whole rounds to the dies: their units, a multiple of 8)
inline int tile_units() { return device_cus() % 8 == 0 ? device_cus() : 8; }

#define RLK_LAUNCH_V(kern, grid, block, st, ...) RLK_LAUNCH(vocab::kern, grid, block, st, __VA_ARGS__)

inline rlk_status compact(hipStream_t st, const int32_t* y, int64_t T, int32_t ignore, int32_t* idx, int32_t* yA,
                          int32_t* n_act, float* z0, float* z1, float* z2) {
  {
    ProfScope _ps("compact_rows", st);
    rlk::launch_compact_rows(st, y, (int)T, ignore, idx, yA, n_act, z0, z1, z2);
  }
  return launched("compact_rows");
}

inline dim3 row_grid(int64_t rows) { return dim3((unsigned)std::min(rows, kRowBlocks)); }

#if RLK_MFMA == 16
template <bool kTop, bool kDz>
rlk_status launch_few(const FewArgs& a, hipStream_t st) {
  typedef void (*Fn)(FewArgs);
  const int c = few_consumers(a.T);
  const Fn fn = c == 1 ? few_tiles<kTop, kDz, 1> : c == 2 ? few_tiles<kTop, kDz, 2> : few_tiles<kTop, kDz, 4>;
  RLK_LAUNCH_FN(kDz ? "few_tiles (dz)" : "few_tiles", fn, dim3((unsigned)std::min(a.chunks, device_cus())),
                dim3((unsigned)few_threads(c)), st, a);
  return RLK_OK;
}

// The logits, and chunk statistics, of a few rows.
template <bool kTop>
rlk_status few_logits(const void* h, const void* W, int64_t T, int64_t H, int64_t V, float scale, float2* rec,
                      float* rec_u, float* z, hipStream_t st) {
  FewArgs a{};
  a.h = static_cast<const uint16_t*>(h);
  a.W = static_cast<const uint16_t*>(W);
  a.T = (int)T;
  a.H = (int)H;
  a.gm = split_geom(V);
  a.scale = scale;
  a.rec_stride = (size_t)T;
  a.rec = rec;
  a.rec_u = rec_u;
  a.z = z;
  a.ldz = few_ldz(V);
  a.chunks = (last_split(a.gm) + 1) * a.gm.cps;
  return launch_few<kTop, false>(a, st);
}
#endif

rlk_status run_top_fwd(const void* h, const void* W, const int32_t* y, int64_t T, int64_t H, int64_t V, int32_t ignore,
                       int64_t K, float* logp, float* lse, float* entropy, float* top_logp, int32_t* top_ids, void* ws,
                       hipStream_t st) {
  const TopFwdWs L = top_fwd_layout(T, H, V, K);
  int32_t* idx = at<int32_t>(ws, L.idx);
  int32_t* yA = at<int32_t>(ws, L.yA);
  int32_t* n_act = at<int32_t>(ws, L.n_act);
  LogitArgs la{};
  la.gm = split_geom(V);
  la.tg.tps = (int)ceil_div(la.gm.S, rlk::kBN);
  la.cus = tile_units();
  const int64_t blocks = tile_blocks(ceil_div(T, rlk::kBM) * L.G * la.tg.tps, la.cus);
  RLK_TRY(check_grid(blocks));
  TopMergeArgs ma{};
  ma.rec = at<float2>(ws, L.rec);
  ma.rec_u = at<float>(ws, L.rec_u);
  ma.rec_stride = (size_t)T;
  ma.T = (int)T;
  ma.ignore_index = ignore;
  ma.y = y;
  ma.gm = la.gm;
  ma.G = (int)L.G;
  ma.first = ma.last = 1;
  ma.R = (int)ceil_div(la.gm.cps, 2 * kSelPer);
  ma.z = at<float>(ws, L.z);
  ma.ldz = L.ldz;
  ma.K = (int)K;
  ma.best = at<uint64_t>(ws, L.best);
  ma.logp = logp;
  ma.lse = lse;
  ma.entropy = entropy;
  ma.top_logp = top_logp;
  ma.top_ids = top_ids;
  const dim3 merge_grid((unsigned)(8 * ceil_div(T, 8)));
#if RLK_MFMA == 16
  if (few_rows(T, V)) {
    RLK_TRY(few_logits<true>(h, W, T, H, V, 1.f, at<float2>(ws, L.rec), at<float>(ws, L.rec_u), at<float>(ws, L.z), st));
    RLK_LAUNCH_V(top_merge, merge_grid, dim3(128), st, ma);
    return RLK_OK;
  }
#endif
  RLK_TRY(compact(st, y, T, ignore, idx, yA, n_act, logp, lse, entropy));
  GatherArgs ga{};
  ga.h = static_cast<const uint16_t*>(h);
  ga.idx = idx;
  ga.n_act = n_act;
  ga.T = (int)T;
  ga.rows = (int)L.T_pad;
  ga.H = (int)H;
  ga.hA = at<uint16_t>(ws, L.hA);
  ga.act = y;
  ga.ignore_index = ignore;
  ga.K = (int)K;
  ga.slot_logp = top_logp;
  ga.slot_ids = top_ids;
  RLK_LAUNCH_V(gather_rows_fill, row_grid(L.T_pad), dim3(256), st, ga);
  la.hA = ga.hA;
  la.W = static_cast<const uint16_t*>(W);
  la.n_act = n_act;
  la.H = (int)H;
  la.G = (int)L.G;
  la.rec_stride = (size_t)T;
  la.rec = at<float2>(ws, L.rec);
  la.yA = yA;
  la.zt = at<float>(ws, L.zt);
  la.rec_u = at<float>(ws, L.rec_u);
  la.z = K > 0 ? at<float>(ws, L.z) : nullptr;
  la.ldz = L.ldz;
  ma.zt = la.zt;
  ma.idx = idx;
  ma.n_act = n_act;
  const int last = last_split(la.gm);
  for (int c = 0; c <= last; c += (int)L.G) {
    la.gm.s0 = c;
    RLK_LAUNCH_FN("logit_tiles", (rlk::vocab::logit_tiles<true>), dim3((unsigned)blocks), dim3(rlk::kThreads), st, la);
    ma.gm = la.gm;
    ma.first = c == 0;
    ma.last = c + L.G > last;
    RLK_LAUNCH_V(top_merge, merge_grid, dim3(128), st, ma);
  }
  return RLK_OK;
}

rlk_status run_distill_fwd(const void* h, const void* W, const int32_t* ids, const float* logits, int64_t T, int64_t H,
                           int64_t V, int64_t K, float scale, float* loss, float* lse, float* logp_ids, void* ws,
                           hipStream_t st) {
  const DistillFwdWs L = distill_fwd_layout(T, H, V, K);
  int32_t* act = at<int32_t>(ws, L.act);
  int32_t* idx = at<int32_t>(ws, L.idx);
  int32_t* n_act = at<int32_t>(ws, L.n_act);
  LogitArgs la{};
  la.gm = split_geom(V);
  la.tg.tps = (int)ceil_div(la.gm.S, rlk::kBN);
  const int64_t row_tiles = ceil_div(T, rlk::kBM);
  la.cus = tile_units();
  const int64_t blocks = tile_blocks(row_tiles * rlk::kNSplit * la.tg.tps, la.cus);
  RLK_TRY(check_grid(blocks));
  DistillMergeArgs ma{};
  ma.rec = at<float2>(ws, L.rec);
  ma.rec_stride = (size_t)T;
  ma.gm = la.gm;
  ma.K = (int)K;
  ma.T = (int)T;
  ma.scale = scale;
  ma.ids = ids;
  ma.logits = logits;
  ma.loss = loss;
  ma.lse = lse;
  ma.logp_ids = logp_ids;
  const dim3 merge_grid((unsigned)(8 * ceil_div(T, 8)));
#if RLK_MFMA == 16
  if (few_rows(T, V)) {
    ma.z = at<float>(ws, L.z);
    ma.ldz = few_ldz(V);
    RLK_TRY(few_logits<false>(h, W, T, H, V, scale, at<float2>(ws, L.rec), nullptr, at<float>(ws, L.z), st));
    RLK_LAUNCH_V(distill_merge, merge_grid, dim3(64), st, ma);
    return RLK_OK;
  }
#endif
  RLK_LAUNCH_V(distill_rows, row_grid(ceil_div(T, 4)), dim3(256), st, ids, logits, (int)T, (int)K, (int)V, scale, act,
               nullptr);
  RLK_TRY(compact(st, act, T, -100, idx, nullptr, n_act, loss, lse, nullptr));
  GatherArgs ga{};
  ga.h = static_cast<const uint16_t*>(h);
  ga.idx = idx;
  ga.n_act = n_act;
  ga.T = (int)T;
  ga.rows = (int)L.T_pad;
  ga.H = (int)H;
  ga.hA = at<uint16_t>(ws, L.hA);
  ga.act = act;
  ga.ignore_index = -100;
  ga.K = (int)K;
  ga.slot_logp = logp_ids;
  RLK_LAUNCH_V(gather_rows_fill, row_grid(L.T_pad), dim3(256), st, ga);
  la.ent_off = at<int32_t>(ws, L.off);
  la.ent = at<uint32_t>(ws, L.ent);
  const auto bucket = rlk::kNSplit * la.tg.tps <= 4096 ? rlk::vocab::bucket_entries<4096> : rlk::vocab::bucket_entries<kMaxVTiles>;
  RLK_LAUNCH_FN("bucket_entries", bucket, dim3((unsigned)ceil_div(T, kBucketRows)), dim3(kBucketThreads), st, ids, logits,
                idx, n_act, (int)K, la.gm, la.tg.tps, at<int32_t>(ws, L.off), at<uint32_t>(ws, L.ent));
  la.hA = ga.hA;
  la.W = static_cast<const uint16_t*>(W);
  la.n_act = n_act;
  la.H = (int)H;
  la.G = rlk::kNSplit;
  la.rec_stride = (size_t)T;
  la.rec = at<float2>(ws, L.rec);
  la.scale = scale;
  la.K = (int)K;
  la.z_ids = at<float>(ws, L.z_ids);
  RLK_LAUNCH_FN("logit_tiles", (rlk::vocab::logit_tiles<false>), dim3((unsigned)blocks), dim3(rlk::kThreads), st, la);
  ma.idx = idx;
  ma.n_act = n_act;
  ma.z_ids = la.z_ids;
  RLK_LAUNCH_V(distill_merge, merge_grid, dim3(64), st, ma);
  return RLK_OK;
}

#if RLK_MFMA == 16
// Both gradients in their few-row kernels up to kFewRows rows: 0.60 ms
// together at 128 rows (H = 4096, V = 151936) against the tiles' 0.94; forms
// for 256 rows took 1.02 against 0.95.
rlk_status launch_few_grad_h(const FewGradHArgs& a, int64_t T, bool cont, hipStream_t st) {
  typedef void (*Fn)(FewGradHArgs);
  static constexpr Fn fns[2][4] = {
      {few_grad_h<1, false>, few_grad_h<2, false>, few_grad_h<4, false>, few_grad_h<8, false>},
      {few_grad_h<1, true>, few_grad_h<2, true>, few_grad_h<4, true>, few_grad_h<8, true>}};
  const int64_t blocks = 8 * ceil_div(a.H / 64 * a.parts, 8);
  int f = 0;
  while ((int64_t)16 << f < T) ++f;
  RLK_LAUNCH_FN("few_grad_h", fns[cont][f], dim3((unsigned)blocks), dim3(256), st, a);
  return RLK_OK;
}

rlk_status launch_few_grad_w(const FewGradWArgs& a, int64_t T, bool bf16, int64_t blocks, hipStream_t st) {
  typedef void (*Fn)(FewGradWArgs);
  static constexpr Fn fns[2][2] = {{few_grad_w<1, false>, few_grad_w<2, false>},
                                   {few_grad_w<1, true>, few_grad_w<2, true>}};
  RLK_LAUNCH_FN("few_grad_w", fns[bf16][T <= 64 ? 0 : 1], dim3((unsigned)blocks), dim3(256), st, a);
  return RLK_OK;
}
#endif

// What the two backwards have in common: gradients of dz in groups of
// splits; `act` marks the inactive rows with `ignore`.  ids != NULL: distill.
struct SoftBwd {
  const void *h, *W;
  const int32_t* act;
  int32_t ignore;
  int64_t T, H, V, K;
  float scale;
  const float *lse, *g, *entropy, *g_entropy;
  const int32_t* ids;
  const float *logits, *logp_ids;
  void *grad_h, *grad_W;
  int32_t dtype;
};

rlk_status run_soft_bwd(const SoftBwd& b, const SoftBwdWs& L, void* ws, hipStream_t st) {
  const bool top = b.ids == nullptr;
  int32_t* idx = at<int32_t>(ws, L.idx);
  int32_t* n_act = at<int32_t>(ws, L.n_act);
  float* part = at<float>(ws, L.part);
  const rlk::SplitGeom gm = split_geom(b.V);
  const int tps = (int)ceil_div(gm.S, rlk::kBN), n_tiles = (int)ceil_div(b.H, rlk::kBN), G = (int)L.G;
  const int64_t row_tiles = ceil_div(b.T, rlk::kBM);
  const int64_t dz_blocks = tile_blocks(row_tiles * G * tps, tile_units());
  const int per = part_splits(b.H, b.V), group_parts = (int)ceil_div(G, per);
  const int64_t gh_tiles = row_tiles * n_tiles * group_parts;  // (or up to cus / 2 halves: cut_tiles)
  const int64_t gh_blocks =
      b.grad_h ? 8 * ceil_div(std::max(gh_tiles, std::min<int64_t>(2 * gh_tiles, device_cus() / 2)), 8) : 0;
  const int64_t gw_blocks = b.grad_W ? 8 * ceil_div((int64_t)n_tiles * G * tps, 8) : 0;
  RLK_TRY(check_grid(dz_blocks));
  RLK_TRY(check_grid(gh_blocks + gw_blocks));
#if RLK_MFMA == 16
  const bool few = b.T <= kFewRows;
#else
  const bool few = false;
#endif
  if (!top && !few)
    RLK_LAUNCH_V(distill_rows, row_grid(ceil_div(b.T, 4)), dim3(256), st, b.ids, b.logits, (int)b.T, (int)b.K,
                 (int)b.V, b.scale, at<int32_t>(ws, L.act), at<float>(ws, L.q));
  if (few) idx = nullptr;  // the batch's rows in place
  else RLK_TRY(compact(st, b.act, b.T, b.ignore, idx, nullptr, n_act, nullptr, nullptr, nullptr));
  GatherGradArgs ga{};
  ga.h = static_cast<const uint16_t*>(b.h);
  ga.idx = idx;
  ga.n_act = n_act;
  ga.rows = (int)L.T_pad;
  ga.H = (int)b.H;
  ga.V = (int)b.V;
  ga.hA = at<uint16_t>(ws, L.hA);
  ga.lse = b.lse;
  ga.g = b.g;
  ga.rowinfo = at<float4>(ws, L.rowinfo);
  ga.rowg = at<float>(ws, L.rowg);
  ga.y = top ? b.act : nullptr;
  ga.entropy = b.entropy;
  ga.g_entropy = b.g_entropy;
  ga.act = b.act;
  ga.scale = b.scale;
#if RLK_MFMA == 16
  FewRowsArgs ra{};
  ra.ga = ga;
  ra.T = (int)b.T;
  ra.ignore_index = b.ignore;
  ra.n_act = n_act;
  ra.ids = b.ids;
  ra.logits = b.logits;
  ra.K = (int)b.K;
  ra.act = at<int32_t>(ws, L.act);
  ra.q = at<float>(ws, L.q);
  if (few && top)
    RLK_LAUNCH_FN("few_rows_grad", (rlk::vocab::few_rows_grad<true>), dim3(kFewRows), dim3(256), st, ra);
  else if (few)
    RLK_LAUNCH_FN("few_rows_grad", (rlk::vocab::few_rows_grad<false>), dim3(kFewRows), dim3(256), st, ra);
  else
#endif
  if (top)
    RLK_LAUNCH_FN("gather_rows_grad", (rlk::vocab::gather_rows_grad<true>), row_grid(L.T_pad), dim3(256), st, ga);
  else
    RLK_LAUNCH_FN("gather_rows_grad", (rlk::vocab::gather_rows_grad<false>), row_grid(L.T_pad), dim3(256), st, ga);
  const int last = last_split(gm);
  for (int c = 0; c <= last; c += G) {
    rlk::BwdGeom bg;
    bg.c_lo = c;
    bg.G = G;
    bg.S_pad = (int)L.S_pad;
    bg.ldz = (int)(G * L.S_pad);
    bg.T_pad = (int)L.T_pad;
    SoftDzArgs da{};
    da.hA = ga.hA;
    da.W = static_cast<const uint16_t*>(b.W);
    da.rowinfo = ga.rowinfo;
    da.rowg = ga.rowg;
    da.n_act = n_act;
    da.H = (int)b.H;
    da.cus = tile_units();
    da.scale = b.scale;
    da.gm = gm;
    da.tg.tps = tps;
    da.bg = bg;
    da.dZ = at<uint16_t>(ws, L.dZ);
    const dim3 grid((unsigned)dz_blocks), block(rlk::kThreads);
#if RLK_MFMA == 16
    if (few) {
      FewArgs fa{};
      fa.h = ga.h;
      fa.W = da.W;
      fa.T = (int)b.T;
      fa.H = (int)b.H;
      fa.gm = gm;
      fa.gm.s0 = c;
      fa.scale = b.scale;
      fa.rowinfo = ga.rowinfo;
      fa.rowg = ga.rowg;
      fa.bg = bg;
      fa.dZ = da.dZ;
      fa.chunks = G * gm.cps;
      if (top) RLK_TRY((launch_few<true, true>(fa, st)));
      else RLK_TRY((launch_few<false, true>(fa, st)));
    } else
#endif
    if (top)
      RLK_LAUNCH_FN("soft_dz_tiles", (rlk::vocab::soft_dz_tiles<true>), grid, block, st, da);
    else
      RLK_LAUNCH_FN("soft_dz_tiles", (rlk::vocab::soft_dz_tiles<false>), grid, block, st, da);
    if (!top) {
      ScatterArgs sa{};
      sa.ids = b.ids;
      sa.q = at<float>(ws, L.q);
      sa.logp_ids = b.logp_ids;
      sa.logits = b.logits;
      sa.idx = idx;
      sa.n_act = n_act;
      sa.rowinfo = ga.rowinfo;
      sa.K = (int)b.K;
      sa.gm = gm;
      sa.bg = bg;
      sa.dZ = da.dZ;
      RLK_LAUNCH_V(distill_scatter, row_grid(b.T), dim3(kMaxK), st, sa);
    }
    rlk::GradWArgs wa{};
    wa.dZ = da.dZ;
    wa.hA = ga.hA;
    wa.n_act = n_act;
    wa.H = (int)b.H;
    wa.gm = gm;
    wa.bg = bg;
    wa.tps = tps;
    wa.n_tiles = n_tiles;
    wa.grad_W = static_cast<float*>(b.grad_W);
    PartGradHArgs ha{};
    ha.dZ = da.dZ;
    ha.W = da.W;
    ha.H = (int)b.H;
    ha.gm = gm;
    ha.bg = bg;
    ha.n_tiles = n_tiles;
    ha.per = per;
    ha.cus = device_cus();
    ha.part0 = c / per;
    ha.parts = std::min(group_parts, last / per + 1 - ha.part0);
    ha.part = b.grad_h ? part : nullptr;
    ha.part_stride = (size_t)b.T * b.H;
    const bool cont = c % per != 0;
#if RLK_MFMA == 16
    if (few && b.grad_h) {
      FewGradHArgs fh{};
      fh.dZ = da.dZ;
      fh.W = da.W;
      fh.n_act = n_act;
      fh.H = (int)b.H;
      fh.gm = gm;
      fh.bg = bg;
      fh.per = per;
      fh.part0 = ha.part0;
      fh.parts = ha.parts;
      fh.part = part;
      fh.part_stride = ha.part_stride;
      RLK_TRY(launch_few_grad_h(fh, b.T, cont, st));
      ha.part = nullptr;
    }
    if (few && b.grad_W) {
      FewGradWArgs fw{};
      fw.dZ = da.dZ;
      fw.hA = ga.hA;
      fw.n_act = n_act;
      fw.H = (int)b.H;
      fw.gm = gm;
      fw.bg = bg;
      fw.grad_W = b.grad_W;
      RLK_TRY(launch_few_grad_w(fw, b.T, b.dtype == RLK_DT_BF16, (int64_t)G * gm.cps, st));
      wa.grad_W = nullptr;
    }
    if (!ha.part && !wa.grad_W) continue;
#endif
    const dim3 gg((unsigned)((ha.part ? gh_blocks : 0) + (wa.grad_W ? gw_blocks : 0)));
    if (b.dtype == RLK_DT_BF16) {
      if (cont) RLK_LAUNCH_FN("part_grad_tiles", (rlk::vocab::part_grad_tiles<true, true>), gg, block, st, ha, wa);
      else RLK_LAUNCH_FN("part_grad_tiles", (rlk::vocab::part_grad_tiles<true, false>), gg, block, st, ha, wa);
    } else {
      if (cont) RLK_LAUNCH_FN("part_grad_tiles", (rlk::vocab::part_grad_tiles<false, true>), gg, block, st, ha, wa);
      else RLK_LAUNCH_FN("part_grad_tiles", (rlk::vocab::part_grad_tiles<false, false>), gg, block, st, ha, wa);
    }
  }
  if (b.grad_h)
    RLK_LAUNCH_V(grad_h_sum, row_grid(b.T), dim3(256), st, part, (size_t)b.T * b.H, last / per + 1, idx, n_act,
                 b.act, b.ignore, (int)b.T, (int)b.H, static_cast<uint16_t*>(b.grad_h));
  return RLK_OK;
}

// Checks of the gradients' outputs; T == 0 zeroes grad_W (the sum over no
// rows) and is done (*done).
rlk_status check_grads(int64_t T, int64_t H, int64_t V, const void* grad_h, void* grad_W, int32_t dtype,
                       hipStream_t st, bool* done) {
  *done = false;
  if (dtype != RLK_DT_F32 && dtype != RLK_DT_BF16) return fail(RLK_ERR_BAD_ARG, "grad_W_dtype=%d", dtype);
  if ((grad_h && !aligned16(grad_h)) || (grad_W && !aligned16(grad_W)))
    return fail(RLK_ERR_BAD_ALIGNMENT, "grad_h, grad_W must be 16-byte aligned");
  if (T > 0) return RLK_OK;
  *done = true;
  if (!grad_W) return RLK_OK;
  RLK_TRY(check_device());
  const int64_t n16 = V * H * (dtype == RLK_DT_F32 ? 4 : 2) / 16;  // H % 64 == 0
  RLK_LAUNCH_V(zero_bytes, row_grid(ceil_div(n16, 256)), dim3(256), st,
               static_cast<rlk::u32x4*>(grad_W), n16);
  return RLK_OK;
}

}  // namespace

extern "C" {

size_t rlk_vocab_workspace_bytes(int32_t op, int64_t T, int64_t H, int64_t V, int64_t K) {
  if (T < 0 || T > kMaxRows || H <= 0 || H > kMaxH || H % 64 != 0 || V <= 0 || V > kMaxV || K < 0 || K > kMaxK) return 0;
  switch (op) {
    case RLK_VOP_TOP_FWD: return top_fwd_layout(T, H, V, K).total;
    case RLK_VOP_TOP_BWD: return soft_bwd_layout(T, H, V, 0).total;
    case RLK_VOP_DISTILL_FWD: return K > 0 ? distill_fwd_layout(T, H, V, K).total : 0;
    case RLK_VOP_DISTILL_BWD: return K > 0 ? soft_bwd_layout(T, H, V, K).total : 0;
    default: return 0;
  }
}

rlk_status rlk_linear_logp_top_fwd(const void* h, const void* W, const int32_t* y, int64_t T, int64_t H, int64_t V,
                                   int32_t ignore_index, int64_t K, float* logp, float* lse, float* entropy,
                                   float* top_logp, int32_t* top_ids, void* ws, size_t ws_bytes, void* stream) {
  RLK_TRY(check_sizes(T, H, V, K, 0));
  if (T == 0) return ok();
  if (!h || !W || !y || !logp || !entropy || !ws || (K > 0 && (!top_logp || !top_ids)))
    return fail(RLK_ERR_NULL_ARG, "h, W, y, logp, entropy, ws (and top_logp, top_ids when K > 0) are required");
  if (!aligned16(h) || !aligned16(W) || !aligned16(ws) || !aligned4(y) || !aligned4(logp) || !aligned4(lse) ||
      !aligned4(entropy) || !aligned4(top_logp) || !aligned4(top_ids))
    return fail(RLK_ERR_BAD_ALIGNMENT, "h, W, ws must be 16-byte aligned, the row arrays 4-byte");
  const size_t need = top_fwd_layout(T, H, V, K).total;
  if (ws_bytes < need) return fail(RLK_ERR_WORKSPACE_TOO_SMALL, "need %zu bytes, got %zu", need, ws_bytes);
  RLK_TRY(check_device());
  RLK_TRY(run_top_fwd(h, W, y, T, H, V, ignore_index, K, logp, lse, entropy, top_logp, top_ids, ws,
                      static_cast<hipStream_t>(stream)));
  return ok();
}

rlk_status rlk_linear_logp_top_bwd(const void* h, const void* W, const int32_t* y, const float* lse,
                                   const float* entropy, const float* g, const float* g_entropy, int64_t T, int64_t H,
                                   int64_t V, int32_t ignore_index, void* grad_h, void* grad_W, int32_t grad_W_dtype,
                                   void* ws, size_t ws_bytes, void* stream) {
  RLK_TRY(check_sizes(T, H, V, 0, 0));
  hipStream_t st = static_cast<hipStream_t>(stream);
  bool done;
  RLK_TRY(check_grads(T, H, V, grad_h, grad_W, grad_W_dtype, st, &done));
  if (done) return ok();
  if (!h || !W || !y || !lse || !entropy || !ws)
    return fail(RLK_ERR_NULL_ARG, "h, W, y, lse, entropy and ws are required");
  if (!aligned16(h) || !aligned16(W) || !aligned16(ws) || !aligned4(y) || !aligned4(lse) || !aligned4(entropy) ||
      !aligned4(g) || !aligned4(g_entropy))
    return fail(RLK_ERR_BAD_ALIGNMENT, "h, W, ws must be 16-byte aligned, the row arrays 4-byte");
  const SoftBwdWs S = soft_bwd_layout(T, H, V, 0);
  if (ws_bytes < S.total) return fail(RLK_ERR_WORKSPACE_TOO_SMALL, "need %zu bytes, got %zu", S.total, ws_bytes);
  if (!grad_h && !grad_W) return ok();
  RLK_TRY(check_device());
  SoftBwd b{};
  b.h = h;
  b.W = W;
  b.act = y;
  b.ignore = ignore_index;
  b.T = T;
  b.H = H;
  b.V = V;
  b.scale = 1.f;
  b.lse = lse;
  b.g = g;
  b.entropy = entropy;
  b.g_entropy = g_entropy;
  b.grad_h = grad_h;
  b.grad_W = grad_W;
  b.dtype = grad_W_dtype;
  RLK_TRY(run_soft_bwd(b, S, ws, st));
  return ok();
}

rlk_status rlk_linear_distill_fwd(const void* h, const void* W, const int32_t* ids, const float* logits, int64_t T,
                                  int64_t H, int64_t V, int64_t K, float temperature, float* loss, float* lse,
                                  float* logp_ids, void* ws, size_t ws_bytes, void* stream) {
  RLK_TRY(check_sizes(T, H, V, K, 1));
  float scale;
  RLK_TRY(check_temperature(temperature, &scale));
  if (T == 0) return ok();
  if (!h || !W || !ids || !logits || !loss || !lse || !logp_ids || !ws)
    return fail(RLK_ERR_NULL_ARG, "h, W, ids, logits, loss, lse, logp_ids and ws are required");
  if (!aligned16(h) || !aligned16(W) || !aligned16(ws) || !aligned4(ids) || !aligned4(logits) || !aligned4(loss) ||
      !aligned4(lse) || !aligned4(logp_ids))
    return fail(RLK_ERR_BAD_ALIGNMENT, "h, W, ws must be 16-byte aligned, the row arrays 4-byte");
  const size_t need = distill_fwd_layout(T, H, V, K).total;
  if (ws_bytes < need) return fail(RLK_ERR_WORKSPACE_TOO_SMALL, "need %zu bytes, got %zu", need, ws_bytes);
  RLK_TRY(check_device());
  RLK_TRY(run_distill_fwd(h, W, ids, logits, T, H, V, K, scale, loss, lse, logp_ids, ws,
                          static_cast<hipStream_t>(stream)));
  return ok();
}

rlk_status rlk_linear_distill_bwd(const void* h, const void* W, const int32_t* ids, const float* logits,
                                  const float* lse, const float* logp_ids, const float* g, int64_t T, int64_t H,
                                  int64_t V, int64_t K, float temperature, void* grad_h, void* grad_W,
                                  int32_t grad_W_dtype, void* ws, size_t ws_bytes, void* stream) {
  RLK_TRY(check_sizes(T, H, V, K, 1));
  SoftBwd b{};
  RLK_TRY(check_temperature(temperature, &b.scale));
  hipStream_t st = static_cast<hipStream_t>(stream);
  bool done;
  RLK_TRY(check_grads(T, H, V, grad_h, grad_W, grad_W_dtype, st, &done));
  if (done) return ok();
  if (!h || !W || !ids || !logits || !lse || !logp_ids || !g || !ws)
    return fail(RLK_ERR_NULL_ARG, "h, W, ids, logits, lse, logp_ids, g and ws are required");
  if (!aligned16(h) || !aligned16(W) || !aligned16(ws) || !aligned4(ids) || !aligned4(logits) || !aligned4(lse) ||
      !aligned4(logp_ids) || !aligned4(g))
    return fail(RLK_ERR_BAD_ALIGNMENT, "h, W, ws must be 16-byte aligned, the row arrays 4-byte");
  const SoftBwdWs S = soft_bwd_layout(T, H, V, K);
  if (ws_bytes < S.total) return fail(RLK_ERR_WORKSPACE_TOO_SMALL, "need %zu bytes, got %zu", S.total, ws_bytes);
  if (!grad_h && !grad_W) return ok();
  RLK_TRY(check_device());
  b.h = h;
  b.W = W;
  b.act = at<int32_t>(ws, S.act);
  b.ignore = -100;
  b.T = T;
  b.H = H;
  b.V = V;
  b.K = K;
  b.lse = lse;
  b.g = g;
  b.ids = ids;
  b.logits = logits;
  b.logp_ids = logp_ids;
  b.grad_h = grad_h;
  b.grad_W = grad_W;
  b.dtype = grad_W_dtype;
  RLK_TRY(run_soft_bwd(b, S, ws, st));
  return ok();
}

}  // extern "C"
