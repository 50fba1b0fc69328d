// Host-side helpers of the C ABI, shared by its translation units: errors,
// workspace layouts, the device check, launches and their optional timing,
// and the argument checks that every LM-head entry point makes.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <vector>

#include "rlk.h"
#include "rlk_args.h"
#include "rlk_kernels.h"
#include "rlk_tiles_w8.h"

// State shared by the translation units.
namespace rlk_state {
#define RLK_HIDDEN __attribute__((visibility("hidden"))) inline
// the calling thread's last error text (a fixed buffer: no entry point can
// throw over it)
RLK_HIDDEN thread_local char g_last_error[512];
RLK_HIDDEN std::mutex g_dev_mu;
RLK_HIDDEN int g_dev_ok[64];   // 0 unknown, 1 gfx950, -1 other
RLK_HIDDEN int g_dev_cus[64];  // compute units of a checked device
struct ProfRec {
  const char* name;
  hipEvent_t start, stop;
};
RLK_HIDDEN std::mutex g_prof_mu;
// read without the lock on every launch: when timing is off (the normal
// case) a launch takes no lock at all
RLK_HIDDEN std::atomic<bool> g_prof_on{false};
RLK_HIDDEN std::vector<ProfRec> g_prof_recs;
RLK_HIDDEN std::vector<hipEvent_t> g_prof_pool;
#undef RLK_HIDDEN
}  // namespace rlk_state

namespace {

using namespace rlk_state;

inline rlk_status fail(rlk_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
inline rlk_status fail(rlk_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
  va_end(ap);
  return s;
}

inline rlk_status ok() {
  g_last_error[0] = 0;
  return RLK_OK;
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Limits that keep every 32-bit index inside the kernels in range.
constexpr int64_t kMaxT = int64_t(1) << 24;
constexpr int64_t kMaxH = 1 << 16;
constexpr int64_t kMaxV = 8000000;  // 32 splits x chunks stay within one grid dimension
constexpr int64_t kMaxGemmMN = int64_t(1) << 24;
constexpr int64_t kMaxGemmK = int64_t(1) << 20;  // 255 rows x K x 2 bytes stay below 2^32

struct Geom {
  int64_t V, S, cps, S_pad;
};

inline Geom geom_of(int64_t V_global) {
  Geom g;
  g.V = V_global;
  g.S = ceil_div(V_global, rlk::kNSplit);
  g.cps = ceil_div(g.S, rlk::kChunk);
  g.S_pad = g.cps * rlk::kChunk;
  return g;
}

// --- workspace layouts -------------------------------------------------------
struct FwdWs {
  size_t idx, yA, n_act, zt, hA, rec, total;
  int64_t rec_chunks, T_pad;
};

// Record slots: one per (chunk of the full vocabulary of V rows, row).
inline FwdWs fwd_layout(int64_t T, int64_t H, int64_t V) {
  FwdWs w;
  w.T_pad = ceil_div(std::max<int64_t>(T, 1), rlk::kBM) * rlk::kBM;
  size_t off = 0;
  w.idx = off;
  off = align256(off + sizeof(int32_t) * T);
  w.yA = off;
  off = align256(off + sizeof(int32_t) * T);
  w.n_act = off;
  off = align256(off + sizeof(int32_t));
  w.zt = off;
  off = align256(off + sizeof(float) * T);
  w.hA = off;
  off = align256(off + 2 * (size_t)w.T_pad * H);
  w.rec_chunks = rlk::kNSplit * geom_of(V).cps;
  w.rec = off;
  off = align256(off + sizeof(float2) * (size_t)w.rec_chunks * (size_t)T);
  w.total = off;
  return w;
}

// Splits per backward group: the largest power of two G <= 32 whose dz
// block (T_pad x G x S_pad bf16) fits the budget (default 2.5 GiB, env
// RLK_DZ_BUDGET_MB overrides it, at most 3.5 GiB).  G changes no result
// bit, only the workspace size and the number of launches.  The cap keeps
// the per-lane byte offsets of a 256-row dz tile (255 rows x G x S_pad x
// 2 B, less than the block since T_pad >= 256) inside the 32 unsigned bits
// the tile loaders use.
inline int64_t dz_budget_bytes() {
  constexpr int64_t kMaxBudget = int64_t(3584) << 20;
  const char* e = std::getenv("RLK_DZ_BUDGET_MB");
  if (e && *e) {
    const long long mb = std::atoll(e);
    if (mb > 0) return std::min<int64_t>((int64_t)mb << 20, kMaxBudget);
  }
  return (int64_t)2560 << 20;
}

struct BwdWs {
  size_t idx, n_act, rowinfo, hA, dZ, ghacc, total;
  int64_t T_pad, S_pad, G;
};

inline BwdWs bwd_layout(int64_t T, int64_t H, int64_t V) {
  const Geom g = geom_of(V);
  BwdWs w;
  w.T_pad = ceil_div(std::max<int64_t>(T, 1), rlk::kBM) * rlk::kBM;
  w.S_pad = ceil_div(g.S, 64) * 64;
  const int64_t per_split = 2 * w.T_pad * w.S_pad;
  const int64_t budget = dz_budget_bytes();
  w.G = 1;
  while (w.G < rlk::kNSplit && 2 * w.G * per_split <= budget) w.G *= 2;
  size_t off = 0;
  w.idx = off;
  off = align256(off + sizeof(int32_t) * T);
  w.n_act = off;
  off = align256(off + sizeof(int32_t));
  w.rowinfo = off;
  off = align256(off + 16 * (size_t)w.T_pad);
  w.hA = off;
  off = align256(off + 2 * (size_t)w.T_pad * H);
  w.dZ = off;
  off = align256(off + (size_t)per_split * w.G);
  w.ghacc = off;
  if (w.G < rlk::kNSplit) off = align256(off + 4 * (size_t)T * H);
  w.total = off;
  return w;
}

// --- device check ----------------------------------------------------------------
inline rlk_status check_device() {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return fail(RLK_ERR_HIP, "hipGetDevice: %s", hipGetErrorString(e));
  if (dev < 0 || dev >= 64) return fail(RLK_ERR_UNSUPPORTED_DEVICE, "device index %d", dev);
  std::lock_guard<std::mutex> lk(g_dev_mu);
  if (g_dev_ok[dev] == 0) {
    hipDeviceProp_t prop;
    e = hipGetDeviceProperties(&prop, dev);
    if (e != hipSuccess) return fail(RLK_ERR_HIP, "hipGetDeviceProperties: %s", hipGetErrorString(e));
    g_dev_ok[dev] = (std::strncmp(prop.gcnArchName, "gfx950", 6) == 0) ? 1 : -1;
    g_dev_cus[dev] = prop.multiProcessorCount;
    if (g_dev_ok[dev] < 0) return fail(RLK_ERR_UNSUPPORTED_DEVICE, "device %d is %s, not gfx950", dev, prop.gcnArchName);
  }
  if (g_dev_ok[dev] < 0) return fail(RLK_ERR_UNSUPPORTED_DEVICE, "device %d is not gfx950", dev);
  return RLK_OK;
}

// Compute units of the current device (after check_device succeeded on it).
inline int device_cus() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
  std::lock_guard<std::mutex> lk(g_dev_mu);
  return g_dev_cus[dev] > 0 ? g_dev_cus[dev] : 256;
}

// grad_h in two row passes (gradh_tile's kPart) when its whole tiles would
// leave most compute units idle while each runs the vocabulary-long chain:
// a pass's chain takes ~70 % of a tile's and the passes add ~40 % to
// grad_h's work, which pays while three times the tile count fits on the
// units (the grad_W tiles fill the rest).  The environment variable
// RLK_GRAD_H_PASSES = 0 / 1 forces either form (results are the same bits;
// tests use it).
inline bool grad_h_passes(int64_t row_tiles, int64_t n_tiles) {
  const char* e = std::getenv("RLK_GRAD_H_PASSES");
  if (e && *e) return std::atoi(e) != 0;
  return 3 * row_tiles * n_tiles <= device_cus();
}

// Tile grids stay within the 2^31 - 1 threads a launch holds along x
// (checked for the larger of the two block sizes).  Row-wise kernels take
// at most kRowBlocks blocks and stride over the rows.
constexpr int64_t kRowBlocks = int64_t(1) << 22;  // 256-thread blocks: 2^30 threads
constexpr int64_t kRowBlocksY = 65535;            // the limit along y
inline rlk_status check_grid(int64_t blocks) {
  if (blocks * std::max(rlk::kThreads, rlk::kThreadsW8) > (int64_t)INT32_MAX)
    return fail(RLK_ERR_BAD_SHAPE, "problem needs %lld tile blocks, more than one launch holds", (long long)blocks);
  return RLK_OK;
}

inline rlk_status launched(const char* what) {
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(RLK_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
  return RLK_OK;
}

// --- optional per-kernel timing (rlk_profile_begin / rlk_profile_end) ---------
inline hipEvent_t prof_event() {
  if (!g_prof_pool.empty()) {
    hipEvent_t e = g_prof_pool.back();
    g_prof_pool.pop_back();
    return e;
  }
  hipEvent_t e = nullptr;
  if (hipEventCreate(&e) != hipSuccess) return nullptr;
  return e;
}

// Brackets one launch with events on its stream when timing is enabled.
struct ProfScope {
  const char* name;
  hipStream_t st;
  hipEvent_t a = nullptr, b = nullptr;
  ProfScope(const char* n, hipStream_t s) : name(n), st(s) {
    if (!g_prof_on.load(std::memory_order_relaxed)) return;
    std::lock_guard<std::mutex> lk(g_prof_mu);
    if (!g_prof_on.load(std::memory_order_relaxed)) return;
    a = prof_event();
    b = prof_event();
    if (a && b) {
      (void)hipEventRecord(a, st);
    } else {  // event creation failed: this launch goes untimed
      if (a) g_prof_pool.push_back(a);
      if (b) g_prof_pool.push_back(b);
      a = b = nullptr;
    }
  }
  ~ProfScope() {
    if (!a || !b) return;
    std::lock_guard<std::mutex> lk(g_prof_mu);
    (void)hipEventRecord(b, st);
    g_prof_recs.push_back(ProfRec{name, a, b});
  }
};

#define RLK_TRY(x)                  \
  do {                              \
    rlk_status _s = (x);            \
    if (_s != RLK_OK) return _s;    \
  } while (0)

// Launch a kernel on stream `st`, timed when profiling is on; return on error.
#define RLK_LAUNCH(kern, grid, block, st, ...)                        \
  do {                                                                \
    {                                                                 \
      ProfScope _ps(#kern, st);                                       \
      hipLaunchKernelGGL(rlk::kern, grid, block, 0, st, __VA_ARGS__); \
    }                                                                 \
    RLK_TRY(launched(#kern));                                         \
  } while (0)

// Same for a kernel given as a function pointer, timed under `name`.
#define RLK_LAUNCH_FN(name, fn, grid, block, st, ...)           \
  do {                                                          \
    {                                                           \
      ProfScope _ps(name, st);                                  \
      hipLaunchKernelGGL(fn, grid, block, 0, st, __VA_ARGS__);  \
    }                                                           \
    RLK_TRY(launched(name));                                    \
  } while (0)

// Same for a launch made by a launcher of the eight-wave unit
// (rlk_tiles_w8.h), timed under `name`.
#define RLK_LAUNCH_W8(name, launcher, grid, st, args) \
  do {                                                \
    {                                                 \
      ProfScope _ps(name, st);                        \
      rlk::launcher(grid, st, args);                  \
    }                                                 \
    RLK_TRY(launched(name));                          \
  } while (0)

// Shapes first; with T == 0 there is nothing to read or write, so the
// pointers are not checked (empty tensors may carry NULL).
inline rlk_status check_common(const void* h, const void* W, const int32_t* y, int64_t T, int64_t H, int64_t V) {
  if (T < 0 || T > kMaxT) return fail(RLK_ERR_BAD_SHAPE, "T=%lld out of [0, 2^24]", (long long)T);
  if (H <= 0 || H > kMaxH || H % 64 != 0)
    return fail(RLK_ERR_BAD_SHAPE, "H=%lld must be a positive multiple of 64 up to 65536", (long long)H);
  if (V <= 0 || V > kMaxV) return fail(RLK_ERR_BAD_SHAPE, "V=%lld out of [1, 8000000]", (long long)V);
  if (T == 0) return RLK_OK;
  if (!h || !W || !y) return fail(RLK_ERR_NULL_ARG, "h, W and y are required");
  if (!aligned16(h) || !aligned16(W) || !aligned16(y)) return fail(RLK_ERR_BAD_ALIGNMENT, "h, W, y must be 16-byte aligned");
  return RLK_OK;
}

}  // namespace
