// The C entry points of include/rlk/step_ops.h.  Everything is enqueued on
// the caller's stream; nothing here allocates device memory or synchronises.
#ifdef RLK_WAVES
#undef RLK_WAVES
#endif
#define RLK_WAVES 8
#define RLK_ENGINE_W8
#define RLK_ENGINE_PARTS
#include "rlk/step_ops.h"

#include <new>

#include "rlk_host.h"
#include "rlk_step.h"

namespace {

using namespace rlk::step;

constexpr int64_t kMaxRows = int64_t(1) << 23;
constexpr int64_t kMaxStride = int64_t(1) << 40;
constexpr int64_t kMaxTensors = int64_t(1) << 20;
// of a tensor: a launch's chunks stay below 2^31
constexpr int64_t kMaxElems = int64_t(1) << 36;
static_assert(kTensors * (kMaxElems / kScaleElems) < INT32_MAX, "chunk indices");

inline bool is_dtype(int32_t d) { return d == RLK_DT_F32 || d == RLK_DT_BF16; }
inline bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline size_t size_of(int32_t dtype) { return dtype == RLK_DT_F32 ? 4 : 2; }
inline bool aligned_as(const void* p, int32_t dtype) { return aligned_to(p, size_of(dtype)); }
inline bool finite(float f) { return f >= -3.402823466e38f && f <= 3.402823466e38f; }

// Blocks of a grid whose kernel strides over `n` work items.
inline unsigned blocks_for(int64_t n, int threads = 256) {
  return (unsigned)std::max<int64_t>(1, std::min(n, (int64_t)INT32_MAX / threads));
}

inline rlk_status check_rows(int64_t T, int64_t H) {
  if (T < 0 || T > kMaxRows) return fail(RLK_ERR_BAD_SHAPE, "T=%lld out of [0, 2^23]", (long long)T);
  if (H < 1 || H > kMaxH) return fail(RLK_ERR_BAD_SHAPE, "H=%lld out of [1, 65536]", (long long)H);
  return RLK_OK;
}

inline rlk_status check_ld(const char* name, int64_t ld) {
  if (ld < 0 || ld > kMaxStride) return fail(RLK_ERR_BAD_SHAPE, "%s=%lld out of [0, 2^40]", name, (long long)ld);
  return RLK_OK;
}

inline rlk_status check_ws(const void* ws, size_t got, size_t need) {
  if (!ws) return fail(RLK_ERR_NULL_ARG, "ws is required");
  if (!aligned16(ws)) return fail(RLK_ERR_BAD_ALIGNMENT, "ws must be 16-byte aligned");
  if (got < need) return fail(RLK_ERR_WORKSPACE_TOO_SMALL, "need %zu bytes, got %zu", need, got);
  return RLK_OK;
}

#define RLK_DTYPE(d, what) \
  do {                     \
    if (!is_dtype(d)) return fail(RLK_ERR_BAD_ARG, what "=%d", (int)(d)); \
  } while (0)

// --- norms ---------------------------------------------------------------------
// Rows a backward's block works on at a time, and the blocks (parts of the
// weight's gradient): by T and H alone.
// Widths above these: the *_wide kernels, where the others would spill.
constexpr int64_t kWideFwd = 16384, kWideBwd = 8192;
inline int norm_row_group(int64_t H) { return H <= 128 ? 16 : H <= 256 ? 8 : H <= 1024 ? 4 : 1; }
inline int64_t norm_parts(int64_t T, int64_t H) {
  // 512 blocks, two a unit, keep more rows in flight; 256 write fewer parts.  The
  // whole backward of layer_norm (both launches), bf16, 256 and 512 parts, us:
  //   H to 2048   8192 x 2048 33 and 26, 16384 x 2048 59 and 42 (fp32 72 and 68),
  //               20000 x 1000 33 and 29; but 1000 x 2048 10.7 and 12.8
  //   to 4096     rows of 2050, 3000, 4096: 1000 rows 14.8 and 16.6, 15.4 and 17.8,
  //               15.4 and 18.4; 1536 rows of 2050 18.1 and 18.2; 2048 rows 20.9 and
  //               19.3, 18.7 and 18.3, 19.4 and 20.3; 8192 rows 67 and 43, 45 and
  //               36, 44.5 and 43.5 (above 1536 rows 256 do better by more than 5 %
  //               for fp32 rows near 4096 only: 8192 rows 66 and 71)
  //   to 8192     4096 x 6144 34 and 40, 16384 x 6144 112 and 123, 8192 x 8192 82
  //               and 89
  // Wider rows' sums have a launch of their own, with blocks along H too; 32, 64
  // and 128 parts: 1024 x 12000 41, 35 and 35, 512 x 65536 fp32 168, 172 and 184.
  const int64_t most = H > kWideBwd ? 64 : H > 4096 || (H > 2048 && T <= 1536) ? 256 : 512;
  static_assert(kMaxParts == 512, "what norm_grad_sum folds");
  return std::max<int64_t>(1, std::min(most, ceil_div(T, norm_row_group(H))));
}
inline int64_t padded_width(int64_t H) { return ceil_div(H, 8) * 8; }
inline size_t norm_bwd_bytes(int64_t T, int64_t H) {
  return align256(2 * sizeof(float) * (size_t)norm_parts(T, H) * padded_width(H));
}

template <class X, class Y, bool kCenter, int R, int E>
rlk_status launch_norm_fwd(const NormFwdArgs& a, hipStream_t st) {
  RLK_LAUNCH_FN("norm_fwd", (norm_fwd<X, Y, kCenter, R, E>),
                dim3(blocks_for(ceil_div(a.T, norm_rows(R)), norm_block(R))), dim3(norm_block(R)), st, a);
  return RLK_OK;
}

template <class X, class Y, bool kCenter>
rlk_status norm_fwd_by_width(const NormFwdArgs& a, hipStream_t st) {
  if (a.H <= 128) return launch_norm_fwd<X, Y, kCenter, 16, 8>(a, st);
  if (a.H <= 256) return launch_norm_fwd<X, Y, kCenter, 32, 8>(a, st);
  if (a.H <= 512) return launch_norm_fwd<X, Y, kCenter, 64, 8>(a, st);
  if (a.H <= 1024) return launch_norm_fwd<X, Y, kCenter, 64, 16>(a, st);
  if (a.H <= 2048) return launch_norm_fwd<X, Y, kCenter, 256, 8>(a, st);
  if (a.H <= 4096) return launch_norm_fwd<X, Y, kCenter, 256, 16>(a, st);
  if (a.H <= 8192) return launch_norm_fwd<X, Y, kCenter, 512, 16>(a, st);
  if (a.H <= kWideFwd) return launch_norm_fwd<X, Y, kCenter, 1024, 16>(a, st);
  RLK_LAUNCH_FN("norm_fwd_wide", (norm_fwd_wide<X, Y, kCenter>), dim3(blocks_for(a.T, 1024)), dim3(1024), st, a);
  return RLK_OK;
}

template <bool kCenter>
rlk_status norm_forward(const void* x, int32_t x_dtype, int64_t ldx, const void* w, const void* b, int32_t w_dtype,
                        int64_t T, int64_t H, float eps, void* y, int32_t y_dtype, float* mean, float* rstd,
                        hipStream_t st) {
  RLK_TRY(check_rows(T, H));
  RLK_TRY(check_ld("ldx", ldx));
  RLK_DTYPE(x_dtype, "x_dtype");
  RLK_DTYPE(y_dtype, "y_dtype");
  if (w || b) RLK_DTYPE(w_dtype, "w_dtype");
  if (!(eps >= 0.f) || !finite(eps)) return fail(RLK_ERR_BAD_ARG, "eps=%g must be finite and not negative", (double)eps);
  if (T == 0) return ok();
  if (!x || !y) return fail(RLK_ERR_NULL_ARG, "x and y are required");
  if (!aligned_as(x, x_dtype) || !aligned_as(y, y_dtype) || !aligned_as(w, w_dtype) || !aligned_as(b, w_dtype) ||
      !aligned_to(mean, 4) || !aligned_to(rstd, 4))
    return fail(RLK_ERR_BAD_ALIGNMENT, "arrays must be aligned to their elements");
  RLK_TRY(check_device());
  NormFwdArgs a{};
  a.x = x;
  a.w = w;
  a.b = b;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  a.ldx = ldx;
  a.T = (int)T;
  a.H = (int)H;
  a.eps = eps;
  a.w_f32 = w_dtype == RLK_DT_F32;
  const bool xf = x_dtype == RLK_DT_F32, yf = y_dtype == RLK_DT_F32;
  RLK_TRY(xf ? (yf ? norm_fwd_by_width<float, float, kCenter>(a, st) : norm_fwd_by_width<float, uint16_t, kCenter>(a, st))
             : (yf ? norm_fwd_by_width<uint16_t, float, kCenter>(a, st)
                   : norm_fwd_by_width<uint16_t, uint16_t, kCenter>(a, st)));
  return ok();
}

template <class X, class G, bool kCenter, int R, int E>
rlk_status launch_norm_bwd(const NormBwdArgs& a, int64_t parts, bool sums, hipStream_t st) {
  if (sums)
    RLK_LAUNCH_FN("norm_bwd", (norm_bwd<X, G, kCenter, true, R, E>), dim3((unsigned)parts), dim3(norm_block(R)), st, a);
  else
    RLK_LAUNCH_FN("norm_bwd", (norm_bwd<X, G, kCenter, false, R, E>), dim3((unsigned)parts), dim3(norm_block(R)), st, a);
  return RLK_OK;
}

template <class X, class G, bool kCenter>
rlk_status norm_bwd_by_width(const NormBwdArgs& a, int64_t parts, bool sums, hipStream_t st) {
  if (a.H > kWideBwd) {
    if (a.grad_x)
      RLK_LAUNCH_FN("norm_bwd_wide", (norm_bwd_wide<X, G, kCenter>), dim3(blocks_for(a.T, 1024)), dim3(1024), st, a);
    if (sums)
      RLK_LAUNCH_FN("norm_sums_wide", (norm_sums_wide<X, G, kCenter>),
                    dim3((unsigned)ceil_div(a.H, 256 * width_of<X, G>()), (unsigned)parts), dim3(256), st, a);
    return RLK_OK;
  }
  if (a.H <= 128) return launch_norm_bwd<X, G, kCenter, 16, 8>(a, parts, sums, st);
  if (a.H <= 256) return launch_norm_bwd<X, G, kCenter, 32, 8>(a, parts, sums, st);
  if (a.H <= 512) return launch_norm_bwd<X, G, kCenter, 64, 8>(a, parts, sums, st);
  if (a.H <= 1024) return launch_norm_bwd<X, G, kCenter, 64, 16>(a, parts, sums, st);
  if (a.H <= 2048) return launch_norm_bwd<X, G, kCenter, 256, 8>(a, parts, sums, st);
  if (a.H <= 4096) return launch_norm_bwd<X, G, kCenter, 256, 16>(a, parts, sums, st);
  return launch_norm_bwd<X, G, kCenter, 512, 16>(a, parts, sums, st);
}

template <bool kCenter>
rlk_status norm_backward(const void* x, int32_t x_dtype, int64_t ldx, const void* w, int32_t w_dtype,
                         const float* mean, const float* rstd, const void* g, int32_t g_dtype, int64_t ldg, int64_t T,
                         int64_t H, void* grad_x, void* grad_weight, void* grad_bias, int32_t grad_dtype, void* ws,
                         size_t ws_bytes, hipStream_t st) {
  RLK_TRY(check_rows(T, H));
  RLK_TRY(check_ld("ldx", ldx));
  RLK_TRY(check_ld("ldg", ldg));
  RLK_DTYPE(x_dtype, "x_dtype");
  RLK_DTYPE(g_dtype, "g_dtype");
  if (w) RLK_DTYPE(w_dtype, "w_dtype");
  const bool sums = grad_weight || grad_bias;
  if (sums) RLK_DTYPE(grad_dtype, "grad_dtype");
  if (!sums && (T == 0 || !grad_x)) return ok();
  if (T > 0 && (!x || !g || !rstd || (kCenter && !mean)))
    return fail(RLK_ERR_NULL_ARG, "x, g, %srstd are required", kCenter ? "mean, " : "");
  if (!aligned_as(x, x_dtype) || !aligned_as(grad_x, x_dtype) || !aligned_as(g, g_dtype) || !aligned_as(w, w_dtype) ||
      !aligned_to(mean, 4) || !aligned_to(rstd, 4) || !aligned_as(grad_weight, grad_dtype) ||
      !aligned_as(grad_bias, grad_dtype))
    return fail(RLK_ERR_BAD_ALIGNMENT, "arrays must be aligned to their elements");
  if (sums) RLK_TRY(check_ws(ws, ws_bytes, norm_bwd_bytes(T, H)));
  RLK_TRY(check_device());
  const int64_t parts = T > 0 ? norm_parts(T, H) : 0;
  NormBwdArgs a{};
  a.x = x;
  a.w = w;
  a.g = g;
  a.mean = mean;
  a.rstd = rstd;
  a.grad_x = grad_x;
  a.part = static_cast<float*>(ws);
  a.ldx = ldx;
  a.ldg = ldg;
  a.T = (int)T;
  a.H = (int)H;
  a.Hp = (int)padded_width(H);
  a.w_f32 = w_dtype == RLK_DT_F32;
  if (T > 0) {
    const bool xf = x_dtype == RLK_DT_F32, gf = g_dtype == RLK_DT_F32;
    RLK_TRY(xf ? (gf ? norm_bwd_by_width<float, float, kCenter>(a, parts, sums, st)
                     : norm_bwd_by_width<float, uint16_t, kCenter>(a, parts, sums, st))
               : (gf ? norm_bwd_by_width<uint16_t, float, kCenter>(a, parts, sums, st)
                     : norm_bwd_by_width<uint16_t, uint16_t, kCenter>(a, parts, sums, st)));
  }
  if (sums) {
    NormSumArgs s{};
    s.part = a.part;
    s.P = (int)parts;
    s.H = a.H;
    s.Hp = a.Hp;
    s.out[0] = grad_weight;
    s.out[1] = grad_bias;
    s.f32 = grad_dtype == RLK_DT_F32;
    RLK_LAUNCH(step::norm_grad_sum, dim3((unsigned)ceil_div(H, 32), kCenter ? 2 : 1), dim3(256), st, s);
  }
  return ok();
}

// --- token embeddings ------------------------------------------------------------
inline int key_bits(int64_t V) {
  int b = 1;
  while ((int64_t(1) << b) <= V) ++b;  // keys 0 .. V
  return b;
}

struct EmbedWs {
  size_t keys[2], perm[2], hist, total_, part, total;
  int64_t tiles, runs;
  int passes;
};

inline EmbedWs embed_layout(int64_t T, int64_t H, int64_t V) {
  EmbedWs w;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align256(off + bytes);
    return at;
  };
  const bool radix = T > kRankRows;
  w.tiles = ceil_div(T, kTile);
  w.passes = radix ? (int)ceil_div(key_bits(V), 9) : 0;
  for (int i = 0; i < 2; ++i) {
    w.keys[i] = take(i < std::max(1, w.passes) ? sizeof(int32_t) * T : 0);
    w.perm[i] = take(i < std::max(1, w.passes) ? sizeof(int32_t) * T : 0);
  }
  w.hist = take(radix ? sizeof(int32_t) * kBins * w.tiles : 0);
  w.total_ = take(radix ? sizeof(int32_t) * kBins : 0);
  w.runs = ceil_div(T, kRun);
  w.part = take(T > kRun ? 2 * sizeof(float) * (size_t)w.runs * H : 0);
  w.total = std::max<size_t>(off, 256);
  return w;
}

inline rlk_status check_embed(const void* ids, int32_t id_bytes, int64_t T, int64_t H, int64_t V, float scale) {
  RLK_TRY(check_rows(T, H));
  if (V <= 0 || V > kMaxV) return fail(RLK_ERR_BAD_SHAPE, "V=%lld out of [1, 8000000]", (long long)V);
  if (id_bytes != 4 && id_bytes != 8) return fail(RLK_ERR_BAD_ARG, "id_bytes=%d", id_bytes);
  if (!finite(scale)) return fail(RLK_ERR_BAD_ARG, "scale=%g must be finite", (double)scale);
  if (T > 0 && !ids) return fail(RLK_ERR_NULL_ARG, "ids are required");
  if (!aligned_to(ids, id_bytes)) return fail(RLK_ERR_BAD_ALIGNMENT, "ids must be aligned to their elements");
  return RLK_OK;
}

template <class E, class O>
rlk_status launch_embed(EmbedArgs a, hipStream_t st) {
  const int64_t vectors = ceil_div(a.H, 64 * width_of<E, O>());
  const int vecs = a.T * vectors <= 8192 ? 1 : 4;
  a.slices = (int)ceil_div(vectors, vecs);
  RLK_LAUNCH_FN("embed_rows", (vecs == 1 ? embed_rows<E, O, 1> : embed_rows<E, O, 4>),
                dim3(blocks_for(ceil_div((int64_t)a.T * a.slices, 4))), dim3(256), st, a);
  return RLK_OK;
}

template <class G, class O>
rlk_status launch_embed_grad(EmbedGradArgs a, hipStream_t st) {
  if (a.T == 0) return RLK_OK;
  a.slices = (int)ceil_div(a.H, 64 * grad_width<O>());
  // windows of up to 16 positions while they leave 32 waves to a unit (16384
  // rows of H = 2048, bf16: 20 us with windows of 16, 32 with windows of 1)
  a.window = 1;
  while (a.window < kRun && (int64_t)a.T * a.slices > 8192 * a.window) a.window *= 2;
  RLK_LAUNCH_FN("embed_grad", (embed_grad<G, O>),
                dim3(blocks_for(ceil_div(ceil_div(a.T, a.window) * a.slices, 4))), dim3(256), st, a);
  if (a.T > kRun)
    RLK_LAUNCH_FN("embed_grad_join", (embed_grad_join<O>),
                  dim3((unsigned)ceil_div(a.T, 128), (unsigned)ceil_div(a.H, 256)), dim3(512), st, a);
  return RLK_OK;
}

// Sorts the tokens by (key, t) and zeroes zero.p on the way.
rlk_status sort_tokens(const IdsArg& ids, int64_t T, int64_t V, const ZeroArgs& zero, const EmbedWs& L, void* ws,
                       const int32_t** keys, const int32_t** perm, KeyMap* map, hipStream_t st) {
  char* base = static_cast<char*>(ws);
  int32_t* k[2];
  int32_t* p[2];
  for (int i = 0; i < 2; ++i) {
    k[i] = reinterpret_cast<int32_t*>(base + L.keys[i]);
    p[i] = reinterpret_cast<int32_t*>(base + L.perm[i]);
  }
  *keys = k[0];
  *perm = p[0];
  map->V = (int)V;
  // blocks that zero: 4 KB each, which is faster (6.7 TB/s) than fewer blocks
  // that stride (4.3 to 5.4)
  const int64_t zero_blocks = zero.p ? std::min<int64_t>(kRowBlocks, ceil_div(zero.bytes, 4096)) : 0;
  if (T <= kRankRows) {
    map->low = kBucketBits;
    map->high = std::max(0, key_bits(V - 1) - kBucketBits);
    map->none = 1 << (map->low + map->high);
    RankArgs a{};
    a.ids = ids;
    a.map = *map;
    a.keys = k[0];
    a.perm = p[0];
    a.T = (int)T;
    a.zero = zero;
    // small blocks for few tokens, and beside blocks that zero (4096 tokens take
    // 7.4 us in small blocks, 8192 in large ones 7; zeroes 6.7 TB/s by small
    // blocks, 6.2 by large)
    const bool few = T <= (zero.p ? 4096 : 1024);
    a.blocks = (int)ceil_div(T, few ? 16 : 64);
    const int64_t zeroing = few ? zero_blocks : ceil_div(zero_blocks, 4);
    if (a.blocks + zeroing == 0) return RLK_OK;
    if (few)
      RLK_LAUNCH_FN("embed_rank", (embed_rank<16>), dim3((unsigned)(a.blocks + zeroing)), dim3(256), st, a);
    else
      RLK_LAUNCH_FN("embed_rank", (embed_rank<64>), dim3((unsigned)(a.blocks + zeroing)), dim3(1024), st, a);
    return RLK_OK;
  }
  const int bits = (int)ceil_div(key_bits(V), L.passes);
  map->low = 24;  // keys are tokens
  map->high = 0;
  map->none = (int)V;
  RadixArgs a{};
  a.ids = ids;
  a.map = *map;
  a.T = (int)T;
  a.tiles = (int)L.tiles;
  a.hist = reinterpret_cast<int32_t*>(base + L.hist);
  a.total = reinterpret_cast<int32_t*>(base + L.total_);
  a.bits = bits;
  a.zero = zero;
  for (int pass = 0; pass < L.passes; ++pass) {
    const int to = pass & 1;
    a.first = pass == 0;
    a.shift = pass * bits;
    a.keys_in = k[1 - to];
    a.perm_in = p[1 - to];
    a.keys = k[to];
    a.perm = p[to];
    RLK_LAUNCH(step::radix_count, dim3((unsigned)(L.tiles + (a.first ? zero_blocks : 0))), dim3(256), st, a);
    RLK_LAUNCH(step::radix_scan, dim3(1u << bits), dim3(256), st, a);
    RLK_LAUNCH(step::radix_scatter, dim3((unsigned)L.tiles), dim3(256), st, a);
    *keys = a.keys;
    *perm = a.perm;
  }
  return RLK_OK;
}

// --- gradients of a step -----------------------------------------------------------
// Parts of the sum of squares: 2048 blocks fill the card; many launches share them.
constexpr int64_t kGradParts = 2048;
// the parts, and the factor behind them
inline size_t grads_parts_bytes(int64_t n) { return sizeof(double) * (size_t)(kGradParts + ceil_div(n, kTensors) + 1); }
inline size_t grads_bytes(int64_t n) { return align256(grads_parts_bytes(n) + sizeof(float)); }

struct Span {
  uintptr_t lo, hi;
  bool write;
};

rlk_status check_tensors(const void* const* grads, const int64_t* sizes, const int32_t* dtypes, int32_t n) {
  if (n < 0 || n > kMaxTensors) return fail(RLK_ERR_BAD_SHAPE, "n=%d out of [0, 2^20]", n);
  if (n == 0) return RLK_OK;
  if (!grads || !sizes || !dtypes) return fail(RLK_ERR_NULL_ARG, "grads, sizes and dtypes are required");
  for (int32_t i = 0; i < n; ++i) {
    if (!is_dtype(dtypes[i])) return fail(RLK_ERR_BAD_ARG, "dtypes[%d]=%d", i, dtypes[i]);
    if (sizes[i] < 0 || sizes[i] > kMaxElems)
      return fail(RLK_ERR_BAD_SHAPE, "sizes[%d]=%lld out of [0, 2^36]", i, (long long)sizes[i]);
    if (sizes[i] > 0 && !grads[i]) return fail(RLK_ERR_NULL_ARG, "grads[%d] is NULL", i);
    if (!aligned_as(grads[i], dtypes[i]))
      return fail(RLK_ERR_BAD_ALIGNMENT, "grads[%d] must be aligned to its elements", i);
  }
  return RLK_OK;
}

rlk_status check_outputs(const void* const* grads, const int64_t* sizes, const int32_t* dtypes, int32_t n,
                         void* const* out, const int32_t* out_dtypes) {
  if (n == 0) return RLK_OK;
  if (!out || !out_dtypes) return fail(RLK_ERR_NULL_ARG, "out and out_dtypes are required");
  Span* s = new (std::nothrow) Span[2 * (size_t)n];
  if (!s) return fail(RLK_ERR_HIP, "out of host memory");
  rlk_status r = RLK_OK;
  size_t m = 0;
  for (int32_t i = 0; i < n && r == RLK_OK; ++i) {
    if (!is_dtype(out_dtypes[i])) r = fail(RLK_ERR_BAD_ARG, "out_dtypes[%d]=%d", i, out_dtypes[i]);
    else if (sizes[i] > 0 && !out[i]) r = fail(RLK_ERR_NULL_ARG, "out[%d] is NULL", i);
    else if (!aligned_as(out[i], out_dtypes[i]))
      r = fail(RLK_ERR_BAD_ALIGNMENT, "out[%d] must be aligned to its elements", i);
    if (r != RLK_OK || sizes[i] == 0) continue;
    const uintptr_t o = reinterpret_cast<uintptr_t>(out[i]), g = reinterpret_cast<uintptr_t>(grads[i]);
    s[m++] = Span{o, o + (uintptr_t)sizes[i] * size_of(out_dtypes[i]), true};
    if (o != g || out_dtypes[i] != dtypes[i]) s[m++] = Span{g, g + (uintptr_t)sizes[i] * size_of(dtypes[i]), false};
  }
  if (r == RLK_OK) {
    std::sort(s, s + m, [](const Span& a, const Span& b) { return a.lo < b.lo; });
    uintptr_t any = 0, written = 0;
    for (size_t i = 0; i < m && r == RLK_OK; ++i) {
      if (s[i].lo < (s[i].write ? any : written))
        r = fail(RLK_ERR_BAD_ARG, "an output overlaps another output, or a gradient that is not its own");
      any = std::max(any, s[i].hi);
      if (s[i].write) written = std::max(written, s[i].hi);
    }
  }
  delete[] s;
  return r;
}

// Launches over up to kTensors tensors each: fills the arguments, calls
// f(args, chunks).
template <class F>
rlk_status each_batch(const void* const* grads, const int64_t* sizes, const int32_t* dtypes, int32_t n,
                      void* const* out, const int32_t* out_dtypes, int64_t chunk, F f) {
  for (int32_t i = 0; i < n;) {
    TensorsArgs a{};
    int64_t chunks = 0;
    for (; i < n && a.count < kTensors; ++i) {
      const int64_t c = ceil_div(sizes[i], chunk);
      if (c == 0) continue;
      const int k = a.count++;
      a.in[k] = grads[i];
      a.n[k] = sizes[i];
      a.first[k] = (int32_t)chunks;
      if (dtypes[i] == RLK_DT_F32) a.in_f32[k / 32] |= 1u << (k % 32);
      if (out) {
        a.out[k] = out[i];
        if (out_dtypes[i] == RLK_DT_F32) a.out_f32[k / 32] |= 1u << (k % 32);
      }
      chunks += c;
    }
    if (!a.count) break;
    a.first[a.count] = (int32_t)chunks;
    RLK_TRY(f(a, chunks));
  }
  return RLK_OK;
}

// The parts of the sum of squares; their number in *parts.
rlk_status square_parts(const void* const* grads, const int64_t* sizes, const int32_t* dtypes, int32_t n, double* part,
                        int* parts, hipStream_t st) {
  const int64_t most = std::max<int64_t>(1, kGradParts / std::max<int64_t>(1, ceil_div(n, kTensors)));
  *parts = 0;
  return each_batch(grads, sizes, dtypes, n, nullptr, nullptr, kSquareElems, [&](TensorsArgs& a, int64_t chunks) {
    const int blocks = (int)std::min(chunks, most);
    a.part = part + *parts;
    *parts += blocks;
    RLK_LAUNCH(step::grads_square, dim3((unsigned)blocks), dim3(256), st, a);
    return (rlk_status)RLK_OK;
  });
}

}  // namespace

extern "C" {

size_t rlk_step_workspace_bytes(int32_t op, int64_t T, int64_t H, int64_t V) {
  if (op == RLK_SOP_GRADS) return T < 0 || T > kMaxTensors ? 0 : grads_bytes(T);
  if (T < 0 || T > kMaxRows || H < 1 || H > kMaxH) return 0;
  if (op == RLK_SOP_NORM_BWD) return norm_bwd_bytes(T, H);
  if (op == RLK_SOP_EMBED_BWD) return V <= 0 || V > kMaxV ? 0 : embed_layout(T, H, V).total;
  return 0;
}

rlk_status rlk_layer_norm_fwd(const void* x, int32_t x_dtype, int64_t ldx, const void* weight, const void* bias,
                              int32_t w_dtype, int64_t T, int64_t H, float eps, void* y, int32_t y_dtype, float* mean,
                              float* rstd, void* stream) {
  return norm_forward<true>(x, x_dtype, ldx, weight, bias, w_dtype, T, H, eps, y, y_dtype, mean, rstd,
                            static_cast<hipStream_t>(stream));
}

rlk_status rlk_rms_norm_fwd(const void* x, int32_t x_dtype, int64_t ldx, const void* weight, int32_t w_dtype,
                            int64_t T, int64_t H, float eps, void* y, int32_t y_dtype, float* rstd, void* stream) {
  return norm_forward<false>(x, x_dtype, ldx, weight, nullptr, w_dtype, T, H, eps, y, y_dtype, nullptr, rstd,
                             static_cast<hipStream_t>(stream));
}

rlk_status rlk_layer_norm_bwd(const void* x, int32_t x_dtype, int64_t ldx, const void* weight, int32_t w_dtype,
                              const float* mean, const float* rstd, const void* g, int32_t g_dtype, int64_t ldg,
                              int64_t T, int64_t H, void* grad_x, void* grad_weight, void* grad_bias,
                              int32_t grad_dtype, void* ws, size_t ws_bytes, void* stream) {
  return norm_backward<true>(x, x_dtype, ldx, weight, w_dtype, mean, rstd, g, g_dtype, ldg, T, H, grad_x, grad_weight,
                             grad_bias, grad_dtype, ws, ws_bytes, static_cast<hipStream_t>(stream));
}

rlk_status rlk_rms_norm_bwd(const void* x, int32_t x_dtype, int64_t ldx, const void* weight, int32_t w_dtype,
                            const float* rstd, const void* g, int32_t g_dtype, int64_t ldg, int64_t T, int64_t H,
                            void* grad_x, void* grad_weight, int32_t grad_dtype, void* ws, size_t ws_bytes,
                            void* stream) {
  return norm_backward<false>(x, x_dtype, ldx, weight, w_dtype, nullptr, rstd, g, g_dtype, ldg, T, H, grad_x,
                              grad_weight, nullptr, grad_dtype, ws, ws_bytes, static_cast<hipStream_t>(stream));
}

rlk_status rlk_embed_fwd(const void* ids, int32_t id_bytes, const void* E, int32_t E_dtype, int64_t T, int64_t H,
                         int64_t V, int64_t ignore_index, float scale, void* out, int32_t out_dtype, void* stream) {
  RLK_TRY(check_embed(ids, id_bytes, T, H, V, scale));
  RLK_DTYPE(E_dtype, "E_dtype");
  RLK_DTYPE(out_dtype, "out_dtype");
  if (T == 0) return ok();
  if (!E || !out) return fail(RLK_ERR_NULL_ARG, "E and out are required");
  if (!aligned_as(E, E_dtype) || !aligned_as(out, out_dtype))
    return fail(RLK_ERR_BAD_ALIGNMENT, "arrays must be aligned to their elements");
  RLK_TRY(check_device());
  EmbedArgs a{};
  a.ids = IdsArg{ids, ignore_index, id_bytes == 8};
  a.E = E;
  a.out = out;
  a.T = (int)T;
  a.H = (int)H;
  a.V = (int)V;
  a.scale = scale;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const bool ef = E_dtype == RLK_DT_F32, of = out_dtype == RLK_DT_F32;
  RLK_TRY(ef ? (of ? launch_embed<float, float>(a, st) : launch_embed<float, uint16_t>(a, st))
             : (of ? launch_embed<uint16_t, float>(a, st) : launch_embed<uint16_t, uint16_t>(a, st)));
  return ok();
}

rlk_status rlk_embed_bwd(const void* ids, int32_t id_bytes, const void* g, int32_t g_dtype, int64_t ldg, int64_t T,
                         int64_t H, int64_t V, int64_t ignore_index, float scale, void* grad_E, int32_t grad_dtype,
                         int32_t accumulate, void* ws, size_t ws_bytes, void* stream) {
  RLK_TRY(check_embed(ids, id_bytes, T, H, V, scale));
  RLK_TRY(check_ld("ldg", ldg));
  RLK_DTYPE(g_dtype, "g_dtype");
  RLK_DTYPE(grad_dtype, "grad_dtype");
  if (accumulate != 0 && accumulate != 1) return fail(RLK_ERR_BAD_ARG, "accumulate=%d", accumulate);
  if (T == 0 && accumulate) return ok();
  if ((T > 0 && !g) || !grad_E) return fail(RLK_ERR_NULL_ARG, "g and grad_E are required");
  if (!aligned_as(g, g_dtype) || !aligned_as(grad_E, grad_dtype))
    return fail(RLK_ERR_BAD_ALIGNMENT, "arrays must be aligned to their elements");
  const EmbedWs L = embed_layout(T, H, V);
  if (T > 0) RLK_TRY(check_ws(ws, ws_bytes, L.total));
  RLK_TRY(check_device());
  hipStream_t st = static_cast<hipStream_t>(stream);
  EmbedGradArgs a{};
  const ZeroArgs zero{accumulate ? nullptr : static_cast<char*>(grad_E), (int64_t)size_of(grad_dtype) * V * H};
  RLK_TRY(sort_tokens(IdsArg{ids, ignore_index, id_bytes == 8}, T, V, zero, L, ws, &a.keys, &a.perm, &a.map, st));
  a.g = g;
  a.ldg = ldg;
  a.grad = grad_E;
  a.part = T > 0 ? reinterpret_cast<float*>(static_cast<char*>(ws) + L.part) : nullptr;
  a.runs = (int)L.runs;
  a.T = (int)T;
  a.H = (int)H;
  a.scale = scale;
  a.accumulate = accumulate;
  const bool gf = g_dtype == RLK_DT_F32, of = grad_dtype == RLK_DT_F32;
  RLK_TRY(gf ? (of ? launch_embed_grad<float, float>(a, st) : launch_embed_grad<float, uint16_t>(a, st))
             : (of ? launch_embed_grad<uint16_t, float>(a, st) : launch_embed_grad<uint16_t, uint16_t>(a, st)));
  return ok();
}

rlk_status rlk_grad_norm(const void* const* grads, const int64_t* sizes, const int32_t* dtypes, int32_t n, float* norm,
                         void* ws, size_t ws_bytes, void* stream) {
  RLK_TRY(check_tensors(grads, sizes, dtypes, n));
  if (!norm) return fail(RLK_ERR_NULL_ARG, "norm is required");
  if (!aligned_to(norm, 4)) return fail(RLK_ERR_BAD_ALIGNMENT, "norm must be aligned to its element");
  RLK_TRY(check_ws(ws, ws_bytes, grads_bytes(n)));
  RLK_TRY(check_device());
  hipStream_t st = static_cast<hipStream_t>(stream);
  double* part = static_cast<double*>(ws);
  int parts = 0;
  RLK_TRY(square_parts(grads, sizes, dtypes, n, part, &parts, st));
  RLK_LAUNCH(step::grads_norm, dim3(1), dim3(256), st, part, parts, norm, static_cast<float*>(nullptr), 0.f);
  return ok();
}

rlk_status rlk_clip_grads(const void* const* grads, const int64_t* sizes, const int32_t* dtypes, int32_t n,
                          float max_norm, void* const* out, const int32_t* out_dtypes, float* norm, void* ws,
                          size_t ws_bytes, void* stream) {
  RLK_TRY(check_tensors(grads, sizes, dtypes, n));
  RLK_TRY(check_outputs(grads, sizes, dtypes, n, out, out_dtypes));
  if (!(max_norm >= 0.f)) return fail(RLK_ERR_BAD_ARG, "max_norm=%g must not be negative", (double)max_norm);
  if (!norm) return fail(RLK_ERR_NULL_ARG, "norm is required");
  if (!aligned_to(norm, 4)) return fail(RLK_ERR_BAD_ALIGNMENT, "norm must be aligned to its element");
  RLK_TRY(check_ws(ws, ws_bytes, grads_bytes(n)));
  RLK_TRY(check_device());
  hipStream_t st = static_cast<hipStream_t>(stream);
  double* part = static_cast<double*>(ws);
  int parts = 0;
  RLK_TRY(square_parts(grads, sizes, dtypes, n, part, &parts, st));
  // the factor has a launch of its own where more blocks than the card holds
  // at once would find it for themselves (or none would)
  int64_t blocks = 0;
  for (int32_t i = 0; i < n; ++i) blocks += ceil_div(sizes[i], kScaleElems);
  const bool apart = blocks == 0 || blocks > kGradParts;
  float* c = reinterpret_cast<float*>(static_cast<char*>(ws) + grads_parts_bytes(n));
  if (apart) RLK_LAUNCH(step::grads_norm, dim3(1), dim3(256), st, part, parts, norm, c, max_norm);
  bool first = true;
  RLK_TRY(each_batch(grads, sizes, dtypes, n, out, out_dtypes, kScaleElems, [&](TensorsArgs& a, int64_t chunks) {
    a.part = part;
    a.parts = apart ? 0 : parts;
    a.norm = first ? norm : nullptr;
    a.c = c;
    a.max_norm = max_norm;
    first = false;
    RLK_LAUNCH(step::grads_scale, dim3(blocks_for(chunks)), dim3(256), st, a);
    return (rlk_status)RLK_OK;
  }));
  return ok();
}

}  // extern "C"
