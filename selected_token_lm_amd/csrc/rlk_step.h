// Kernels of include/rlk/step_ops.h: norms, token embeddings, gradient norm
// and clipping.  All of them are bound by HBM (a few operations an element)
// or, for a few rows, by latency; there is no product for the matrix units.
//
// Elements move in vectors of eight (16 bytes of bf16, 32 of fp32).  Rows may
// start at any element (odd widths, strides): the hardware loads and stores
// 16 bytes at any address, so one path serves every alignment and a row's
// sums keep their order; only a row's last, short vector goes by elements.
#pragma once

#include "rlk_device.h"

namespace rlk {
namespace step {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

struct F8 {
  float v[8];
};

// Eight elements as they lie in memory.
template <class T>
struct Raw {
  u32x4 q[sizeof(T) / 2];
};

__device__ __forceinline__ float bf16_to_f32(uint32_t b) { return __uint_as_float(b << 16); }

__device__ __forceinline__ F8 widen(const Raw<uint16_t>& r) {
  F8 f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f.v[2 * i] = __uint_as_float(r.q[0][i] << 16);
    f.v[2 * i + 1] = __uint_as_float(r.q[0][i] & 0xffff0000u);
  }
  return f;
}
__device__ __forceinline__ F8 widen(const Raw<float>& r) {
  F8 f;
#pragma unroll
  for (int i = 0; i < 8; ++i) f.v[i] = __uint_as_float(r.q[i >> 2][i & 3]);
  return f;
}

// Elements p[0 .. n), n <= 8 (the rest zero; nothing is read where n <= 0).
template <class T>
__device__ __forceinline__ Raw<T> load(const T* p, int n) {
  Raw<T> r;
  if (n >= 8) {
    __builtin_memcpy(&r, p, sizeof(r));
    return r;
  }
  r = Raw<T>{};
#pragma unroll
  for (int i = 0; i < 7; ++i) {
    if (i < n) {
      if constexpr (sizeof(T) == 4) r.q[i >> 2][i & 3] = __float_as_uint(p[i]);
      else r.q[0][i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
    }
  }
  return r;
}

__device__ __forceinline__ void store(uint16_t* p, const F8& f, int n) {
  u32x4 q;
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = pack_bf16x2(f.v[2 * i], f.v[2 * i + 1]);
  if (n >= 8) {
    __builtin_memcpy(p, &q, 16);
    return;
  }
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (i < n) p[i] = (uint16_t)(q[i >> 1] >> (16 * (i & 1)));
}
__device__ __forceinline__ void store(float* p, const F8& f, int n) {
  if (n >= 8) {
    __builtin_memcpy(p, &f, 32);
    return;
  }
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (i < n) p[i] = f.v[i];
}

// Eight elements of an array whose type is known at run time (uniform).
__device__ __forceinline__ F8 load_any(const void* p, bool f32, int64_t at, int n) {
  if (f32) return widen(load(static_cast<const float*>(p) + at, n));
  return widen(load(static_cast<const uint16_t*>(p) + at, n));
}
__device__ __forceinline__ void store_any(void* p, bool f32, int64_t at, const F8& f, int n) {
  if (f32) store(static_cast<float*>(p) + at, f, n);
  else store(static_cast<uint16_t*>(p) + at, f, n);
}

// Sum over a wave, in every lane: pairs 1, 2, then mirrored quads and octets
// (lanes 4 and 8 apart hold sums of four and eight), rows of 16, halves.
template <int kCtrl>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(v), kCtrl, 0xf, 0xf, true));
}
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp<0xb1>(v);   // quad_perm [1, 0, 3, 2]
  v += dpp<0x4e>(v);   // quad_perm [2, 3, 0, 1]
  v += dpp<0x141>(v);  // row_half_mirror
  v += dpp<0x140>(v);  // row_mirror
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  float lo, hi;
  lane_halves(v, lo, hi);
  return lo + hi;
}

// --- norms -------------------------------------------------------------------
// R threads hold a row in registers, N vectors each: vector i * R + lane.  The
// split goes by H alone, so a row's sums have one order.
template <int R>
struct RowSum {
  static constexpr int kWaves = R / 64;
  // red: kWaves floats for each of the kVals sums; consecutive calls take
  // different ones (one barrier a call).
  template <int kVals>
  static __device__ __forceinline__ void run(float (&v)[kVals], float* red) {
#pragma unroll
    for (int k = 0; k < kVals; ++k) v[k] = wave_sum(v[k]);
    if constexpr (R > 64) {
      const int wave = threadIdx.x / 64;
      if (threadIdx.x % 64 == 0) {
#pragma unroll
        for (int k = 0; k < kVals; ++k) red[k * kWaves + wave] = v[k];
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kVals; ++k) {
        float s = red[k * kWaves];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) s += red[k * kWaves + w];
        v[k] = s;
      }
    }
  }
};

constexpr int norm_block(int R) { return R < 256 ? 256 : R; }
constexpr int norm_rows(int R) { return norm_block(R) / R; }

struct NormFwdArgs {
  const void* x;
  const void* w;
  const void* b;
  void* y;
  float* mean;
  float* rstd;
  int64_t ldx;
  int T, H;
  float eps;
  int w_f32;
};

// y = (x - mean) rstd w + b (kCenter), or x rstd w.  The row is read once; the
// variance is taken about the mean (a second sum over registers).
template <class X, class Y, bool kCenter, int R, int N>
__global__ __launch_bounds__(norm_block(R)) void norm_fwd(NormFwdArgs a) {
  constexpr int kRows = norm_rows(R);
  constexpr int kWaves = R / 64;
  __shared__ float red[2 * kWaves];
  const int lane = threadIdx.x % R;
  const float fH = (float)a.H;
  for (int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / R; row < a.T; row += (int64_t)gridDim.x * kRows) {
    const X* x = static_cast<const X*>(a.x) + row * a.ldx;
    Raw<X> raw[N];
#pragma unroll
    for (int i = 0; i < N; ++i) raw[i] = load(x + 8 * (i * R + lane), a.H - 8 * (i * R + lane));
    F8 v[N];
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = widen(raw[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[0] += kCenter ? v[i].v[j] : v[i].v[j] * v[i].v[j];
    }
    RowSum<R>::run(s, red);
    float mean = 0.f;
    if constexpr (kCenter) {
      mean = s[0] / fH;
      s[0] = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int n = a.H - 8 * (i * R + lane);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[i].v[j] = j < n ? v[i].v[j] - mean : 0.f;
          s[0] += v[i].v[j] * v[i].v[j];
        }
      }
      RowSum<R>::run(s, red + kWaves);
    }
    const float rstd = 1.f / __builtin_sqrtf(s[0] / fH + a.eps);
    if (lane == 0) {
      if (kCenter && a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    Y* y = static_cast<Y*>(a.y) + row * a.H;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = 8 * (i * R + lane), n = a.H - c;
      if (n <= 0) continue;
      F8 o;
#pragma unroll
      for (int j = 0; j < 8; ++j) o.v[j] = v[i].v[j] * rstd;
      if (a.w) {
        const F8 w = load_any(a.w, a.w_f32, c, n);
#pragma unroll
        for (int j = 0; j < 8; ++j) o.v[j] *= w.v[j];
      }
      if (kCenter && a.b) {
        const F8 b = load_any(a.b, a.w_f32, c, n);
#pragma unroll
        for (int j = 0; j < 8; ++j) o.v[j] += b.v[j];
      }
      store(y + c, o, n);
    }
    if (!kCenter && R > 64) __syncthreads();  // red is free again
  }
}

struct NormBwdArgs {
  const void* x;
  const void* w;
  const void* g;
  const float* mean;
  const float* rstd;
  void* grad_x;   // may be NULL
  float* part;    // [2][P][Hp]: a block's sums of g n and of g
  int64_t ldx, ldg;
  int T, H, Hp;
  int w_f32;
};

// A block takes rows b, b + P, ...: grad_x of each, and the block's sums for
// the weight's and bias's gradients in registers.  The next row's loads are
// issued before the current row's sums are exchanged.
template <class X, class G, bool kCenter, bool kSums, int R, int N>
__global__ __launch_bounds__(norm_block(R)) void norm_bwd(NormBwdArgs a) {
  constexpr int kRows = norm_rows(R);
  constexpr int kVals = kCenter ? 2 : 1;
  constexpr int kWaves = R / 64;
  __shared__ float red[2][kVals * kWaves];
  const int lane = threadIdx.x % R;
  const float fH = (float)a.H;
  F8 w[N], dw[N], db[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = 8 * (i * R + lane), n = a.H - c;
    if (a.w) w[i] = load_any(a.w, a.w_f32, c, n);
    else w[i] = F8{{1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f}};
    dw[i] = db[i] = F8{};
  }
  Raw<X> xr[N];
  Raw<G> gr[N];
  float mean = 0.f, rstd = 0.f;
  int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / R;
  const int64_t stride = (int64_t)gridDim.x * kRows;
  auto fetch = [&](int64_t t) {
    const X* x = static_cast<const X*>(a.x) + t * a.ldx;
    const G* g = static_cast<const G*>(a.g) + t * a.ldg;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = 8 * (i * R + lane);
      xr[i] = load(x + c, a.H - c);
      gr[i] = load(g + c, a.H - c);
    }
    if (kCenter) mean = a.mean[t];
    rstd = a.rstd[t];
  };
  if (row < a.T) fetch(row);
  int turn = 0;
  for (; row < a.T; row += stride, turn ^= 1) {
    F8 nv[N], gw[N];
    float s[kVals] = {};
    const float r = rstd, mu = mean;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const F8 xv = widen(xr[i]), gv = widen(gr[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = kCenter ? (xv.v[j] - mu) * r : xv.v[j] * r;
        const float g = gv.v[j];
        nv[i].v[j] = n;
        gw[i].v[j] = g * w[i].v[j];
        if (kSums) {
          dw[i].v[j] = __builtin_fmaf(g, n, dw[i].v[j]);
          if (kCenter) db[i].v[j] += g;
        }
        s[0] = __builtin_fmaf(gw[i].v[j], n, s[0]);
        if constexpr (kCenter) s[1] += gw[i].v[j];
      }
    }
    if (row + stride < a.T) fetch(row + stride);
    if (!a.grad_x) continue;
    RowSum<R>::run(s, red[turn]);
    const float c1 = s[0] / fH;
    float c2 = 0.f;
    if constexpr (kCenter) c2 = s[1] / fH;
    X* gx = static_cast<X*>(a.grad_x) + row * a.H;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = 8 * (i * R + lane);
      if (c >= a.H) continue;
      F8 o;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float t = kCenter ? gw[i].v[j] - c2 : gw[i].v[j];
        o.v[j] = r * (t - nv[i].v[j] * c1);
      }
      store(gx + c, o, a.H - c);
    }
  }
  if constexpr (kSums) {
    float* part = a.part + (int64_t)blockIdx.x * a.Hp;
    const int64_t second = (int64_t)gridDim.x * a.Hp;
    if constexpr (kRows > 1) {
      // the row groups' sums in order, through LDS
      __shared__ float4 lds[kRows][R * N * 2];
#pragma unroll
      for (int k = 0; k < kVals; ++k) {
        if (k) __syncthreads();
        const F8* d = k ? db : dw;
        const int q = threadIdx.x / R;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          lds[q][2 * (i * R + lane)] = make_float4(d[i].v[0], d[i].v[1], d[i].v[2], d[i].v[3]);
          lds[q][2 * (i * R + lane) + 1] = make_float4(d[i].v[4], d[i].v[5], d[i].v[6], d[i].v[7]);
        }
        __syncthreads();
        for (int e = threadIdx.x; e < 2 * R * N; e += norm_block(R)) {
          if (4 * e >= a.Hp) continue;
          float4 t = lds[0][e];
#pragma unroll
          for (int m = 1; m < kRows; ++m) {
            t.x += lds[m][e].x;
            t.y += lds[m][e].y;
            t.z += lds[m][e].z;
            t.w += lds[m][e].w;
          }
          *reinterpret_cast<float4*>(part + k * second + 4 * e) = t;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = 8 * (i * R + lane);
        if (c >= a.H) continue;
        store(part + c, dw[i], 8);
        if (kCenter) store(part + second + c, db[i], 8);
      }
    }
  }
}

// Rows wider than the registers hold: a pass over the row for each sum (the
// row comes from L2 then) and one for the result.
template <class X, class Y, bool kCenter>
__global__ __launch_bounds__(1024) void norm_fwd_wide(NormFwdArgs a) {
  constexpr int R = 1024;
  __shared__ float red[2][R / 64];
  const float fH = (float)a.H;
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
    const X* x = static_cast<const X*>(a.x) + row * a.ldx;
    float mean = 0.f, s[1] = {0.f};
    if constexpr (kCenter) {
      for (int c = 8 * threadIdx.x; c < a.H; c += 8 * R) {
        const F8 f = widen(load(x + c, a.H - c));
#pragma unroll
        for (int j = 0; j < 8; ++j) s[0] += f.v[j];
      }
      RowSum<R>::run(s, red[0]);
      mean = s[0] / fH;
      s[0] = 0.f;
    }
    for (int c = 8 * threadIdx.x; c < a.H; c += 8 * R) {
      const F8 f = widen(load(x + c, a.H - c));
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = c + j < a.H ? f.v[j] - mean : 0.f;
        s[0] += d * d;
      }
    }
    RowSum<R>::run(s, red[1]);
    const float rstd = 1.f / __builtin_sqrtf(s[0] / fH + a.eps);
    if (threadIdx.x == 0) {
      if (kCenter && a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    Y* y = static_cast<Y*>(a.y) + row * a.H;
    for (int c = 8 * threadIdx.x; c < a.H; c += 8 * R) {
      F8 o = widen(load(x + c, a.H - c));
#pragma unroll
      for (int j = 0; j < 8; ++j) o.v[j] = (kCenter ? o.v[j] - mean : o.v[j]) * rstd;
      if (a.w) {
        const F8 w = load_any(a.w, a.w_f32, c, a.H - c);
#pragma unroll
        for (int j = 0; j < 8; ++j) o.v[j] *= w.v[j];
      }
      if (kCenter && a.b) {
        const F8 b = load_any(a.b, a.w_f32, c, a.H - c);
#pragma unroll
        for (int j = 0; j < 8; ++j) o.v[j] += b.v[j];
      }
      store(y + c, o, a.H - c);
    }
    if (!kCenter) __syncthreads();  // red[1] is free again
  }
}

// The backward of such rows: one pass for its sums, one for grad_x.
template <class X, class G, bool kCenter>
__global__ __launch_bounds__(1024) void norm_bwd_wide(NormBwdArgs a) {
  constexpr int R = 1024, kVals = kCenter ? 2 : 1;
  __shared__ float red[2][kVals * (R / 64)];
  const float fH = (float)a.H;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x, turn ^= 1) {
    const X* x = static_cast<const X*>(a.x) + row * a.ldx;
    const G* g = static_cast<const G*>(a.g) + row * a.ldg;
    const float mu = kCenter ? a.mean[row] : 0.f, r = a.rstd[row];
    auto values = [&](int c, F8& nv, F8& gw) {
      nv = widen(load(x + c, a.H - c));
      gw = widen(load(g + c, a.H - c));
      if (a.w) {
        const F8 w = load_any(a.w, a.w_f32, c, a.H - c);
#pragma unroll
        for (int j = 0; j < 8; ++j) gw.v[j] *= w.v[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) nv.v[j] = kCenter ? (nv.v[j] - mu) * r : nv.v[j] * r;
    };
    float s[kVals] = {};
    for (int c = 8 * threadIdx.x; c < a.H; c += 8 * R) {
      F8 nv, gw;
      values(c, nv, gw);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        s[0] = __builtin_fmaf(gw.v[j], nv.v[j], s[0]);
        if constexpr (kCenter) s[1] += gw.v[j];
      }
    }
    RowSum<R>::run(s, red[turn]);
    const float c1 = s[0] / fH;
    float c2 = 0.f;
    if constexpr (kCenter) c2 = s[1] / fH;
    X* gx = static_cast<X*>(a.grad_x) + row * a.H;
    for (int c = 8 * threadIdx.x; c < a.H; c += 8 * R) {
      F8 nv, gw;
      values(c, nv, gw);
#pragma unroll
      for (int j = 0; j < 8; ++j) gw.v[j] = r * ((kCenter ? gw.v[j] - c2 : gw.v[j]) - nv.v[j] * c1);
      store(gx + c, gw, a.H - c);
    }
  }
}

// The sums of such rows: 2048 columns a block, rows p, p + P, ...
template <class X, class G, bool kCenter>
__global__ __launch_bounds__(256) void norm_sums_wide(NormBwdArgs a) {
  const int c = 8 * (blockIdx.x * 256 + threadIdx.x);
  if (c >= a.H) return;
  F8 dw{}, db{};
  for (int64_t row = blockIdx.y; row < a.T; row += gridDim.y) {
    const F8 x = widen(load(static_cast<const X*>(a.x) + row * a.ldx + c, a.H - c));
    const F8 g = widen(load(static_cast<const G*>(a.g) + row * a.ldg + c, a.H - c));
    const float mu = kCenter ? a.mean[row] : 0.f, r = a.rstd[row];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float n = kCenter ? (x.v[j] - mu) * r : x.v[j] * r;
      dw.v[j] = __builtin_fmaf(g.v[j], n, dw.v[j]);
      db.v[j] += g.v[j];
    }
  }
  float* part = a.part + (int64_t)blockIdx.y * a.Hp + c;
  store(part, dw, 8);
  if (kCenter) store(part + (int64_t)gridDim.y * a.Hp, db, 8);
}

struct NormSumArgs {
  const float* part;
  int P, H, Hp;
  void* out[2];  // the weight's gradient, the bias's; either may be NULL
  int f32;
};

// The blocks' sums folded: 32 columns a block, 32 groups of parts (p, p + 32,
// ...), then these groups in order.
__global__ __launch_bounds__(256) void norm_grad_sum(NormSumArgs a) {
  __shared__ float4 lds[32][8];
  void* out = a.out[blockIdx.y];
  if (!out) return;
  const int k = threadIdx.x % 8, q = threadIdx.x / 8;
  const int c = 32 * blockIdx.x + 4 * k;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < a.Hp) {
    const float* p = a.part + (int64_t)blockIdx.y * a.P * a.Hp + c;
#pragma unroll 8
    for (int i = q; i < a.P; i += 32) {
      const float4 t = *reinterpret_cast<const float4*>(p + (int64_t)i * a.Hp);
      s.x += t.x;
      s.y += t.y;
      s.z += t.z;
      s.w += t.w;
    }
  }
  lds[q][k] = s;
  __syncthreads();
  if (threadIdx.x >= 32 || 32 * blockIdx.x + threadIdx.x >= (unsigned)a.H) return;
  const float* l = reinterpret_cast<const float*>(lds) + threadIdx.x;
  float v = l[0];
#pragma unroll
  for (int i = 1; i < 32; ++i) v += l[32 * i];
  const int at = 32 * blockIdx.x + threadIdx.x;
  if (a.f32) static_cast<float*>(out)[at] = v;
  else static_cast<uint16_t*>(out)[at] = (uint16_t)pack_bf16x2(v, 0.f);
}

// --- token embeddings ----------------------------------------------------------
struct IdsArg {
  const void* p;
  int64_t ignore;
  int wide;  // int64
};
__device__ __forceinline__ int64_t id_at(const IdsArg& a, int64_t t) {
  return a.wide ? static_cast<const int64_t*>(a.p)[t] : (int64_t)static_cast<const int32_t*>(a.p)[t];
}

struct EmbedArgs {
  IdsArg ids;
  const void* E;
  void* out;
  int T, H, V;
  float scale;
};

// out[t] = scale E[id]: L lanes a row, each vectors lane, lane + L, ...
template <class E, class O, int L>
__global__ __launch_bounds__(256) void embed_rows(EmbedArgs a) {
  const int lane = threadIdx.x % L;
  for (int64_t t = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L; t < a.T; t += (int64_t)gridDim.x * (256 / L)) {
    const int64_t id = id_at(a.ids, t);
    O* out = static_cast<O*>(a.out) + t * a.H;
    const bool ignored = id == a.ids.ignore;
    if (ignored || id < 0 || id >= a.V) {
      const float f = ignored ? 0.f : __builtin_nanf("");
      for (int c = 8 * lane; c < a.H; c += 8 * L) store(out + c, F8{{f, f, f, f, f, f, f, f}}, a.H - c);
      continue;
    }
    const E* row = static_cast<const E*>(a.E) + id * a.H;
#pragma unroll 4
    for (int c = 8 * lane; c < a.H; c += 8 * L) {
      F8 f = widen(load(row + c, a.H - c));
#pragma unroll
      for (int j = 0; j < 8; ++j) f.v[j] *= a.scale;
      store(out + c, f, a.H - c);
    }
  }
}

// The gradient goes by positions of the tokens sorted by (id, t): keys[i] and
// the row perm[i].  Ids that reach no row have the key V and stand last.
__device__ __forceinline__ int key_of(const IdsArg& a, int64_t t, int V) {
  const int64_t id = id_at(a, t);
  return id == a.ignore || id < 0 || id >= V ? V : (int)id;
}

// Up to kRankRows tokens: a token's position is the number of tokens before it
// in that order, counted against all others.  64 tokens a block, one a lane;
// the 16 waves count a sixteenth of the others each.
constexpr int kRankRows = 16384;

__global__ __launch_bounds__(1024) void embed_rank(IdsArg ids, int T, int V, int32_t* keys, int32_t* perm) {
  __shared__ int32_t all[kRankRows];
  __shared__ int32_t count[16][64];
  // padded to whole groups of four per wave with keys that precede nothing
  const int per = (T + 63) / 64 * 4;
  for (int t = threadIdx.x; t < 16 * per; t += 1024) all[t] = t < T ? key_of(ids, t, V) : INT32_MAX;
  __syncthreads();
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int t0 = 64 * blockIdx.x, t = t0 + lane;
  const int key = t < T ? all[t] : INT32_MIN;
  const int lo = wave * per, hi = lo + per;
  int n = 0;
  // tokens before this block's, its own, and those behind (bounds are
  // multiples of four)
  const int a = min(max(t0, lo), hi), b = min(max(t0 + 64, lo), hi);
#pragma unroll 4
  for (int i = lo; i < a; i += 4) {
    const int4 k = *reinterpret_cast<const int4*>(all + i);
    n += (k.x <= key) + (k.y <= key) + (k.z <= key) + (k.w <= key);
  }
  for (int i = a; i < b; ++i) n += all[i] < key || (all[i] == key && i < t);
#pragma unroll 4
  for (int i = b; i < hi; i += 4) {
    const int4 k = *reinterpret_cast<const int4*>(all + i);
    n += (k.x < key) + (k.y < key) + (k.z < key) + (k.w < key);
  }
  count[wave][lane] = n;
  __syncthreads();
  if (wave || t >= T) return;
  int at = 0;
#pragma unroll
  for (int w = 0; w < 16; ++w) at += count[w][lane];
  keys[at] = key;
  perm[at] = t;
}

// More tokens: a radix sort by digits of up to nine bits, the lowest first;
// tiles of 4096 tokens, a wave's 1024 in order.
constexpr int kTile = 4096, kBins = 512;

struct RadixArgs {
  IdsArg ids;  // the first pass's input
  const int32_t* keys_in;
  const int32_t* perm_in;
  int32_t* keys;
  int32_t* perm;
  int32_t* hist;   // [kBins][tiles]
  int32_t* total;  // [kBins]
  int T, V, tiles;
  int shift, bits, first;
};
__device__ __forceinline__ int radix_key(const RadixArgs& a, int t) {
  return a.first ? key_of(a.ids, t, a.V) : a.keys_in[t];
}

__global__ __launch_bounds__(256) void radix_count(RadixArgs a) {
  __shared__ int32_t bin[kBins];
  const int mask = (1 << a.bits) - 1;
  for (int i = threadIdx.x; i < kBins; i += 256) bin[i] = 0;
  __syncthreads();
  const int base = blockIdx.x * kTile;
  for (int i = threadIdx.x; i < kTile && base + i < a.T; i += 256)
    atomicAdd(&bin[(radix_key(a, base + i) >> a.shift) & mask], 1);
  __syncthreads();
  for (int i = threadIdx.x; i <= mask; i += 256) a.hist[(int64_t)i * a.tiles + blockIdx.x] = bin[i];
}

// Exclusive sum over 256 threads, and the total.
__device__ __forceinline__ int block_scan(int v, int* lds, int& total) {
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  int s = v;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(s, d);
    if (lane >= d) s += o;
  }
  if (lane == 63) lds[wave] = s;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if (w < wave) before += lds[w];
    total += lds[w];
  }
  __syncthreads();
  return before + s - v;
}

// A digit's tiles: exclusive sums in place, and the digit's total.
__global__ __launch_bounds__(256) void radix_scan(RadixArgs a) {
  __shared__ int lds[4];
  int32_t* h = a.hist + (int64_t)blockIdx.x * a.tiles;
  int run = 0;
  for (int i = 0; i < a.tiles; i += 256) {
    const int at = i + threadIdx.x;
    int sum;
    const int before = block_scan(at < a.tiles ? h[at] : 0, lds, sum);
    if (at < a.tiles) h[at] = run + before;
    run += sum;
  }
  if (threadIdx.x == 0) a.total[blockIdx.x] = run;
}

__global__ __launch_bounds__(256) void radix_scatter(RadixArgs a) {
  __shared__ int32_t at[4][kBins];
  __shared__ int lds[4];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int bins = 1 << a.bits, mask = bins - 1;
  for (int i = threadIdx.x; i < 4 * kBins; i += 256) (&at[0][0])[i] = 0;
  __syncthreads();
  const int base = blockIdx.x * kTile + wave * (kTile / 4);
  constexpr int kRounds = kTile / 4 / 64;
  int key[kRounds];
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int t = base + 64 * r + lane;
    key[r] = t < a.T ? radix_key(a, t) : -1;
    if (t < a.T) atomicAdd(&at[wave][(key[r] >> a.shift) & mask], 1);
  }
  __syncthreads();
  // a wave's first position of a digit: digits below, tiles before, waves before
  int run = 0;
  for (int i = 0; i < kBins; i += 256) {
    const int d = i + threadIdx.x;
    int sum;
    const int before = block_scan(d < bins ? a.total[d] : 0, lds, sum);
    if (d < bins) {
      int p = run + before + a.hist[(int64_t)d * a.tiles + blockIdx.x];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const int c = at[w][d];
        at[w][d] = p;
        p += c;
      }
    }
    run += sum;
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int t = base + 64 * r + lane;
    const bool live = t < a.T;
    const int d = (key[r] >> a.shift) & mask;
    uint64_t same = __ballot(live);
    for (int b = 0; b < a.bits; ++b) {
      const uint64_t one = __ballot((d >> b) & 1);
      same &= (d >> b) & 1 ? one : ~one;
    }
    const int rank = __builtin_popcountll(same & ((1ull << lane) - 1));
    int p = 0;
    if (live) p = at[wave][d] + rank;
    // the whole wave has read its positions before their first lane moves on
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (live && rank == 0) at[wave][d] += __builtin_popcountll(same);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (live) {
      a.keys[p] = key[r];
      a.perm[p] = a.first ? t : a.perm_in[t];
    }
  }
}

// The first position of keys[0, n) (ascending) that is not below v, found by
// a whole wave, 64 probes a step.
__device__ __forceinline__ int lower_bound(const int32_t* keys, int n, int v) {
  const int lane = threadIdx.x % 64;
  int lo = 0, hi = n;
  while (lo < hi) {
    const int step = (hi - lo + 63) / 64;
    const int p = lo + lane * step;
    const int below = __builtin_popcountll(__ballot(p < hi && keys[p] < v));
    if (!below) break;
    hi = min(hi, lo + below * step);
    lo += (below - 1) * step + 1;
  }
  return lo;
}

// Rows of one token are summed in runs of kRun from its first on, a wave and
// 512 columns each; a token of more rows leaves its runs' sums in parts.
constexpr int kRun = 64;

struct EmbedGradArgs {
  const int32_t* keys;
  const int32_t* perm;
  const void* g;
  int64_t ldg;
  void* grad;
  float* part;  // [2 * runs][H], runs = ceil(T / kRun)
  int T, H, V;
  float scale;
  int accumulate;
  int waves;       // of a block, on one position (1, 2 or 4), by H
  int item_blocks;
  int zero_rows;   // rows of grad a block behind item_blocks looks at
};

// The part of the run that starts at position i: a token's first run, or a
// later one, can each start only once in kRun positions.
__device__ __forceinline__ int64_t part_of(int i, bool first) { return 2 * (int64_t)(i / kRun) + first; }

template <class O>
__device__ __forceinline__ void grad_row(const EmbedGradArgs& a, int key, int c, const F8& sum) {
  O* p = static_cast<O*>(a.grad) + (int64_t)key * a.H + c;
  F8 f;
#pragma unroll
  for (int j = 0; j < 8; ++j) f.v[j] = a.scale * sum.v[j];
  if (a.accumulate) {
    const F8 old = widen(load(p, a.H - c));
#pragma unroll
    for (int j = 0; j < 8; ++j) f.v[j] = old.v[j] + f.v[j];
  }
  store(p, f, a.H - c);
}

template <class G, class O>
__device__ __forceinline__ void embed_item(const EmbedGradArgs& a, int i, int slice, int slices) {
  const int lane = threadIdx.x % 64;
  const int32_t* k = a.keys;
  const int key = __builtin_amdgcn_readfirstlane(k[i]);
  if (key >= a.V) return;
  const int ahead = i + lane < a.T ? k[i + lane] : -1;
  const int back = i - 1 - lane >= 0 ? k[i - 1 - lane] : -1;
  const int my_row = i + lane < a.T ? a.perm[i + lane] : 0;
  const uint64_t differ = __ballot(back != key);
  bool first = true;
  if (!(differ & 1)) {
    // a run starts here only a multiple of kRun behind the token's first row
    if (differ) return;
    if ((i - lower_bound(k, a.T, key)) % kRun) return;
    first = false;
  }
  const uint64_t other = __ballot(ahead != key);
  const int n = other ? __builtin_ctzll(other) : kRun;
  const bool whole = first && (n < kRun || i + kRun >= a.T || k[i + kRun] != key);
  // (whole waves turn the loop: rows' numbers are read from other lanes)
  for (int c0 = 512 * slice; c0 < a.H; c0 += 512 * slices) {
    const int c = c0 + 8 * lane;
    F8 sum{};
    const G* g = static_cast<const G*>(a.g) + c;
    int j = 0;
    for (; j + 4 <= n; j += 4) {
      Raw<G> r[4];
#pragma unroll
      for (int m = 0; m < 4; ++m)
        r[m] = load(g + __builtin_amdgcn_readlane(my_row, j + m) * a.ldg, a.H - c);
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const F8 f = widen(r[m]);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum.v[e] += f.v[e];
      }
    }
    for (; j < n; ++j) {
      const F8 f = widen(load(g + __builtin_amdgcn_readlane(my_row, j) * a.ldg, a.H - c));
#pragma unroll
      for (int e = 0; e < 8; ++e) sum.v[e] += f.v[e];
    }
    if (whole) grad_row<O>(a, key, c, sum);
    else store(a.part + part_of(i, first) * a.H + c, sum, a.H - c);
  }
}

// Zeroes the rows [v0, v1) of the gradient whose token does not occur.
template <class O>
__device__ __forceinline__ void embed_zero(const EmbedGradArgs& a, int v0, int v1) {
  const int lane = threadIdx.x % 64;
  uint64_t there = 0;  // bit v - v0; v1 - v0 <= 64
  for (int p = lower_bound(a.keys, a.T, v0); p < a.T;) {
    const int k = p + lane < a.T ? a.keys[p + lane] : a.V;
    const int last = __builtin_amdgcn_readlane(k, 63);
    for (int v = v0; v < v1; ++v)
      if (__ballot(k == v)) there |= 1ull << (v - v0);
    if (last >= v1) break;
    p = p + 64 < a.T && a.keys[p + 64] != last ? p + 64 : lower_bound(a.keys, a.T, last + 1);
  }
  for (int v = v0; v < v1; ++v) {
    if (there >> (v - v0) & 1) continue;
    O* p = static_cast<O*>(a.grad) + (int64_t)v * a.H;
    for (int c = 8 * threadIdx.x; c < a.H; c += 8 * 256) store(p + c, F8{}, a.H - c);
  }
}

template <class G, class O>
__global__ __launch_bounds__(256) void embed_grad(EmbedGradArgs a) {
  if ((int)blockIdx.x < a.item_blocks) {
    const int wave = threadIdx.x / 64, per = 4 / a.waves;
    for (int64_t i = (int64_t)blockIdx.x * per + wave / a.waves; i < a.T; i += (int64_t)a.item_blocks * per)
      embed_item<G, O>(a, __builtin_amdgcn_readfirstlane((int)i), wave % a.waves, a.waves);
  } else {
    const int64_t zero_blocks = gridDim.x - a.item_blocks;
    for (int64_t v = (int64_t)(blockIdx.x - a.item_blocks) * a.zero_rows; v < a.V; v += zero_blocks * a.zero_rows)
      embed_zero<O>(a, (int)v, (int)min(v + a.zero_rows, (int64_t)a.V));
  }
}

// Tokens of more than kRun rows: their runs' sums, in order.  A block for the
// one such token that can start in kRun positions, 512 columns at a time: 16
// waves sum consecutive sixteenths, and these are summed in order.
template <class O>
__global__ __launch_bounds__(1024) void embed_grad_join(EmbedGradArgs a) {
  __shared__ F8 lds[16][64];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int32_t* k = a.keys;
  const int base = blockIdx.x * kRun, p = base + lane;
  const int key = p < a.T ? k[p] : a.V;
  const bool start = key < a.V && p + kRun < a.T && k[p + kRun] == key && (p == 0 || k[p - 1] != key);
  const uint64_t at = __ballot(start);
  if (!at) return;  // the same for all waves
  const int s = base + __builtin_ctzll(at);
  const int token = __builtin_amdgcn_readlane(key, s - base);
  const int end = lower_bound(k, a.T, token + 1);
  const int runs = (end - s + kRun - 1) / kRun, per = (runs + 15) / 16;
  const int lo = min(wave * per, runs), hi = min(lo + per, runs);
  for (int c0 = blockIdx.y * 512; c0 < a.H; c0 += gridDim.y * 512) {
    const int c = c0 + 8 * lane, n = a.H - c;
    F8 sum{};
    for (int r = lo; r < hi; ++r) {
      const F8 f = widen(load(a.part + part_of(s + r * kRun, r == 0) * a.H + c, n));
#pragma unroll
      for (int e = 0; e < 8; ++e) sum.v[e] += f.v[e];
    }
    lds[wave][lane] = sum;
    __syncthreads();
    if (wave == 0 && n > 0) {
      for (int w = 1; w < 16; ++w) {
        const F8 f = lds[w][lane];
#pragma unroll
        for (int e = 0; e < 8; ++e) sum.v[e] += f.v[e];
      }
      grad_row<O>(a, token, c, sum);
    }
    __syncthreads();
  }
}

// --- gradients of a step ---------------------------------------------------------
constexpr int kTensors = 96;       // of one launch (its arguments stay below 4 KB)
constexpr int kChunkElems = 16384;  // a block's unit of work

struct TensorsArgs {
  const void* in[kTensors];
  void* out[kTensors];
  int64_t n[kTensors];
  int32_t first[kTensors + 1];  // the tensor's first chunk
  uint32_t in_f32[kTensors / 32], out_f32[kTensors / 32];
  int count;
  double* part;
  int parts;       // of all launches (scaling)
  float* norm;
  float max_norm;
};

__device__ __forceinline__ int tensor_of(const TensorsArgs& a, int chunk) {
  int lo = 0, hi = a.count;  // first[lo] <= chunk < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.first[mid] <= chunk) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ double block_sum(double v, double* lds) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
  if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = v;
  __syncthreads();
  return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

template <class T>
__device__ __forceinline__ void square_sum(const T* p, int64_t n, double (&s)[4]) {
#pragma unroll
  for (int h = 0; h < kChunkElems / 2048; h += 4) {
    Raw<T> r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t c = 8 * (int64_t)((h + i) * 256 + threadIdx.x);
      r[i] = load(p + c, (int)min<int64_t>(n - c, 8));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const F8 f = widen(r[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const double d = (double)f.v[j];
        s[j & 3] = __builtin_fma(d, d, s[j & 3]);
      }
    }
  }
}

// part[b] = the sum of squares of chunks b, b + gridDim.x, ..., in fp64: no
// square overflows or is lost, and the sum needs no care for its order.
__global__ __launch_bounds__(256) void grads_square(TensorsArgs a) {
  __shared__ double lds[4];
  double s[4] = {0., 0., 0., 0.};
  const int chunks = a.first[a.count];
  for (int64_t chunk = blockIdx.x; chunk < chunks; chunk += gridDim.x) {
    const int i = tensor_of(a, (int)chunk);
    const int64_t at = (chunk - a.first[i]) * kChunkElems, n = a.n[i] - at;
    if (a.in_f32[i / 32] >> (i % 32) & 1) square_sum(static_cast<const float*>(a.in[i]) + at, n, s);
    else square_sum(static_cast<const uint16_t*>(a.in[i]) + at, n, s);
  }
  const double v = block_sum((s[0] + s[1]) + (s[2] + s[3]), lds);
  if (threadIdx.x == 0) a.part[blockIdx.x] = v;
}

__device__ __forceinline__ double norm_of(const double* part, int parts, double* lds) {
  double s = 0.;
  for (int i = threadIdx.x; i < parts; i += 256) s += part[i];
  return __builtin_sqrt(block_sum(s, lds));
}

__global__ __launch_bounds__(256) void grads_norm(const double* part, int parts, float* norm) {
  __shared__ double lds[4];
  const double v = norm_of(part, parts, lds);
  if (threadIdx.x == 0) *norm = (float)v;
}

template <class T, class O>
__device__ __forceinline__ void scale_chunk(const T* p, O* o, int64_t n, float c) {
#pragma unroll
  for (int h = 0; h < kChunkElems / 2048; h += 4) {
    Raw<T> r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t e = 8 * (int64_t)((h + i) * 256 + threadIdx.x);
      r[i] = load(p + e, (int)min<int64_t>(n - e, 8));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t e = 8 * (int64_t)((h + i) * 256 + threadIdx.x);
      F8 f = widen(r[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) f.v[j] *= c;
      store(o + e, f, (int)min<int64_t>(n - e, 8));
    }
  }
}

// out = c grads; every block finds the norm from the parts for itself.
__global__ __launch_bounds__(256) void grads_scale(TensorsArgs a) {
  __shared__ double lds[4];
  const double norm = norm_of(a.part, a.parts, lds);
  const float c = norm <= (double)a.max_norm ? 1.f : (float)((double)a.max_norm / norm);
  if (a.norm && blockIdx.x == 0 && threadIdx.x == 0) *a.norm = (float)norm;
  const int chunks = a.first[a.count];
  for (int64_t chunk = blockIdx.x; chunk < chunks; chunk += gridDim.x) {
    const int i = tensor_of(a, (int)chunk);
    const int64_t at = (chunk - a.first[i]) * kChunkElems, n = a.n[i] - at;
    const bool f = a.in_f32[i / 32] >> (i % 32) & 1, of = a.out_f32[i / 32] >> (i % 32) & 1;
    const float* p = static_cast<const float*>(a.in[i]) + at;
    const uint16_t* pb = static_cast<const uint16_t*>(a.in[i]) + at;
    float* o = static_cast<float*>(a.out[i]) + at;
    uint16_t* ob = static_cast<uint16_t*>(a.out[i]) + at;
    if (a.in[i] == a.out[i] && c == 1.f) continue;
    if (f && of) scale_chunk(p, o, n, c);
    else if (f) scale_chunk(p, ob, n, c);
    else if (of) scale_chunk(pb, o, n, c);
    else scale_chunk(pb, ob, n, c);
  }
}

}  // namespace step
}  // namespace rlk
