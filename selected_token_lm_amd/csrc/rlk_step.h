// Kernels of include/rlk/step_ops.h: norms, token embeddings, gradient norm
// and clipping.  All of them are bound by HBM (a few operations an element)
// or, for a few rows, by latency; there is no product for the matrix units.
//
// Elements move in vectors of eight (16 bytes of bf16, 32 of fp32), or of four
// where all are fp32.  Rows may start at
// any element (odd widths, strides): the hardware loads and stores 16 bytes
// at any address, so one path serves every alignment and a row's sums keep
// their order; only a row's last, short vector goes by elements.
#pragma once

#include "rlk_device.h"

namespace rlk {
namespace step {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Elements of a vector that moves between arrays of these types.
template <class A, class B = A>
constexpr int width_of() {
  return sizeof(A) == 4 && sizeof(B) == 4 ? 4 : 8;
}

template <int V>
struct FV {
  float v[V];
};

// V elements as they lie in memory.
template <class T, int V>
struct Raw {
  uint32_t q[sizeof(T) * V / 4];
};

template <int V>
__device__ __forceinline__ FV<V> widen(const Raw<uint16_t, V>& r) {
  FV<V> f;
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    f.v[2 * i] = __uint_as_float(r.q[i] << 16);
    f.v[2 * i + 1] = __uint_as_float(r.q[i] & 0xffff0000u);
  }
  return f;
}
template <int V>
__device__ __forceinline__ FV<V> widen(const Raw<float, V>& r) {
  FV<V> f;
#pragma unroll
  for (int i = 0; i < V; ++i) f.v[i] = __uint_as_float(r.q[i]);
  return f;
}

// Elements p[0 .. n), n <= V (the rest zero; nothing is read where n <= 0).
template <int V, class T>
__device__ __forceinline__ Raw<T, V> load(const T* p, int n) {
  Raw<T, V> r;
  if (n >= V) {
    __builtin_memcpy(&r, p, sizeof(r));
    return r;
  }
  r = Raw<T, V>{};
#pragma unroll
  for (int i = 0; i < V - 1; ++i) {
    if (i < n) {
      if constexpr (sizeof(T) == 4) r.q[i] = __float_as_uint(p[i]);
      else r.q[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
    }
  }
  return r;
}

template <int V>
__device__ __forceinline__ void store(uint16_t* p, const FV<V>& f, int n) {
  Raw<uint16_t, V> r;
#pragma unroll
  for (int i = 0; i < V / 2; ++i) r.q[i] = pack_bf16x2(f.v[2 * i], f.v[2 * i + 1]);
  if (n >= V) {
    __builtin_memcpy(p, &r, sizeof(r));
    return;
  }
#pragma unroll
  for (int i = 0; i < V - 1; ++i)
    if (i < n) p[i] = (uint16_t)(r.q[i >> 1] >> (16 * (i & 1)));
}
template <int V>
__device__ __forceinline__ void store(float* p, const FV<V>& f, int n) {
  if (n >= V) {
    __builtin_memcpy(p, &f, sizeof(f));
    return;
  }
#pragma unroll
  for (int i = 0; i < V - 1; ++i)
    if (i < n) p[i] = f.v[i];
}

// A vector that is not read again soon (non-temporal).
template <int V, class T>
__device__ __forceinline__ Raw<T, V> load_once(const T* p, int64_t n) {
  if (n < V) return load<V>(p, (int)n);
  constexpr int kBytes = sizeof(T) * V, kWords = kBytes / 4;
  typedef uint32_t words __attribute__((ext_vector_type(kWords), aligned(sizeof(T))));
  const words w = __builtin_nontemporal_load(reinterpret_cast<const words*>(p));
  Raw<T, V> r;
#pragma unroll
  for (int i = 0; i < kWords; ++i) r.q[i] = w[i];
  return r;
}
template <int V, class T>
__device__ __forceinline__ void store_once(T* p, const FV<V>& f, int64_t n) {
  if (n < V) {
    store(p, f, (int)n);
    return;
  }
  constexpr int kWords = sizeof(T) * V / 4;
  typedef uint32_t words __attribute__((ext_vector_type(kWords), aligned(sizeof(T))));
  words w;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < V; ++i) w[i] = __float_as_uint(f.v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) w[i] = pack_bf16x2(f.v[2 * i], f.v[2 * i + 1]);
  }
  __builtin_nontemporal_store(w, reinterpret_cast<words*>(p));
}

// Elements of an array whose type is known at run time (uniform).
template <int V>
__device__ __forceinline__ FV<V> load_any(const void* p, bool f32, int64_t at, int n) {
  if (f32) return widen(load<V>(static_cast<const float*>(p) + at, n));
  return widen(load<V>(static_cast<const uint16_t*>(p) + at, n));
}

// Sum over groups of R lanes (16, 32 or 64) of a wave, in every lane: pairs 1,
// 2, then mirrored quads and octets (lanes 4 and 8 apart hold sums of four and
// eight), rows of 16, halves.  Groups may sit out as a whole.
template <int kCtrl>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(v), kCtrl, 0xf, 0xf, true));
}
template <int R>
__device__ __forceinline__ float lane_sum(float v) {
  v += dpp<0xb1>(v);   // quad_perm [1, 0, 3, 2]
  v += dpp<0x4e>(v);   // quad_perm [2, 3, 0, 1]
  v += dpp<0x141>(v);  // row_half_mirror
  v += dpp<0x140>(v);  // row_mirror
  if constexpr (R >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if constexpr (R >= 64) {
    float lo, hi;
    lane_halves(v, lo, hi);
    v = lo + hi;
  }
  return v;
}

// --- norms -------------------------------------------------------------------
// Bound by HBM: a few operations an element.  R threads hold a row in registers,
// N vectors of V each: vector i * R + lane.  The split goes by H and the types
// alone, so a row's sums have one order.
template <int R>
struct RowSum {
  static constexpr int kWaves = R > 64 ? R / 64 : 1;
  // red (R > 64): kWaves floats for each of the kVals sums; consecutive calls
  // take different ones (one barrier a call).
  template <int kVals>
  static __device__ __forceinline__ void run(float (&v)[kVals], float* red) {
#pragma unroll
    for (int k = 0; k < kVals; ++k) v[k] = lane_sum<R < 64 ? R : 64>(v[k]);
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

// A mean whose sum left fp32 is taken again from terms scaled by a power of two
// that 65536 of them do not leave it with (rows that hold a NaN or an infinity
// end as they were).
constexpr float kSmall = 1.f / (1 << 17);
__device__ __forceinline__ bool in_range(float f) { return __builtin_fabsf(f) <= 3.402823466e38f; }

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
// variance is taken about the mean (a second sum over registers).  Weights are
// loaded with the row, not after its sums (16384 x 2048, fp32 -> bf16: 48 -> 41
// us, 4.9 TB/s; 4096 x 4096 bf16: 13 us, 5.0 TB/s; one row 2.3 us).  Narrow rows
// share a wave (163840 rows of 128, bf16: 16 us, 100000 of 64: 9,
// where a wave a row takes 30).
template <class X, class Y, bool kCenter, int R, int E>
__global__ __launch_bounds__(norm_block(R)) void norm_fwd(NormFwdArgs a) {
  constexpr int V = width_of<X, Y>(), N = E / V;
  constexpr int kRows = norm_rows(R);
  constexpr int kWaves = RowSum<R>::kWaves;
  __shared__ float red[3 * kWaves];
  const int lane = threadIdx.x % R;
  const float fH = (float)a.H;
  for (int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / R; row < a.T; row += (int64_t)gridDim.x * kRows) {
    const X* x = static_cast<const X*>(a.x) + row * a.ldx;
    Raw<X, V> raw[N];
#pragma unroll
    for (int i = 0; i < N; ++i) raw[i] = load<V>(x + V * (i * R + lane), a.H - V * (i * R + lane));
    FV<V> w[N], b[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = V * (i * R + lane);
      if (a.w) w[i] = load_any<V>(a.w, a.w_f32, c, a.H - c);
      if (kCenter && a.b) b[i] = load_any<V>(a.b, a.w_f32, c, a.H - c);
    }
    FV<V> v[N];
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = widen(raw[i]);
#pragma unroll
      for (int j = 0; j < V; ++j) s[0] += kCenter ? v[i].v[j] : v[i].v[j] * v[i].v[j];
    }
    RowSum<R>::run(s, red);
    float mean = 0.f;
    if constexpr (kCenter) {
      mean = s[0] / fH;
      if (!in_range(mean)) {  // the same for all threads of the row
        s[0] = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int j = 0; j < V; ++j) s[0] += v[i].v[j] * kSmall;
        RowSum<R>::run(s, red + 2 * kWaves);
        mean = s[0] / fH / kSmall;
      }
      s[0] = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int n = a.H - V * (i * R + lane);
#pragma unroll
        for (int j = 0; j < V; ++j) {
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
      const int c = V * (i * R + lane), n = a.H - c;
      if (n <= 0) continue;
      FV<V> o;
#pragma unroll
      for (int j = 0; j < V; ++j) o.v[j] = v[i].v[j] * rstd;
      if (a.w) {
#pragma unroll
        for (int j = 0; j < V; ++j) o.v[j] *= w[i].v[j];
      }
      if (kCenter && a.b) {
#pragma unroll
        for (int j = 0; j < V; ++j) o.v[j] += b[i].v[j];
      }
      store(y + c, o, n);
    }
    if (!kCenter && R > 64) __syncthreads();  // red is free again
  }
}

// Behind the row's end x is 0 and n = -mean rstd, which may be infinite where no
// element's n is (a constant row of 2^121): 0 there, as g is.
template <int V>
__device__ __forceinline__ void zero_past(FV<V>& n, int left) {
  if (left >= V) return;
#pragma unroll
  for (int j = 0; j < V; ++j) n.v[j] = j < left ? n.v[j] : 0.f;
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

// A block takes rows b, b + P, ... (several at a time where they are narrow):
// grad_x of each, and the block's sums for the weight's and bias's gradients in
// registers, so that x and g are read once.  The next row's loads are issued
// before the current row's sums are exchanged.  256 or 512 blocks: more write
// more parts, fewer do not hide the memory (the kernel alone: 16384 x 2048, fp32
// and bf16, 59 us, 5.7 TB/s; 4096 x 4096 bf16 19 us, 5.3 TB/s).
template <class X, class G, bool kCenter, bool kSums, int R, int E>
__global__ __launch_bounds__(norm_block(R)) void norm_bwd(NormBwdArgs a) {
  constexpr int V = width_of<X, G>(), N = E / V;
  constexpr int kRows = norm_rows(R);
  constexpr int kVals = kCenter ? 2 : 1;
  constexpr int kWaves = RowSum<R>::kWaves;
  __shared__ float red[2][kVals * kWaves];
  const int lane = threadIdx.x % R;
  const float fH = (float)a.H;
  FV<V> w[N], dw[N], db[N];
  FV<V> ones;
#pragma unroll
  for (int j = 0; j < V; ++j) ones.v[j] = 1.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = V * (i * R + lane), n = a.H - c;
    if (a.w) w[i] = load_any<V>(a.w, a.w_f32, c, n);
    else w[i] = ones;
    dw[i] = db[i] = FV<V>{};
  }
  Raw<X, V> xr[N];
  Raw<G, V> gr[N];
  float mean = 0.f, rstd = 0.f;
  int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / R;
  const int64_t stride = (int64_t)gridDim.x * kRows;
  auto fetch = [&](int64_t t) {
    const X* x = static_cast<const X*>(a.x) + t * a.ldx;
    const G* g = static_cast<const G*>(a.g) + t * a.ldg;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = V * (i * R + lane);
      xr[i] = load<V>(x + c, a.H - c);
      gr[i] = load<V>(g + c, a.H - c);
    }
    if (kCenter) mean = a.mean[t];
    rstd = a.rstd[t];
  };
  if (row < a.T) fetch(row);
  int turn = 0;
  for (; row < a.T; row += stride, turn ^= 1) {
    FV<V> nv[N], gw[N];
    float s[kVals] = {};
    const float r = rstd, mu = mean;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const FV<V> xv = widen(xr[i]), gv = widen(gr[i]);
#pragma unroll
      for (int j = 0; j < V; ++j) nv[i].v[j] = kCenter ? (xv.v[j] - mu) * r : xv.v[j] * r;
      if constexpr (kCenter) zero_past(nv[i], a.H - V * (i * R + lane));
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float n = nv[i].v[j], g = gv.v[j];
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
      const int c = V * (i * R + lane);
      if (c >= a.H) continue;
      FV<V> o;
#pragma unroll
      for (int j = 0; j < V; ++j) {
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
      __shared__ float4 lds[kRows][R * E / 4];
#pragma unroll
      for (int k = 0; k < kVals; ++k) {
        if (k) __syncthreads();
        const FV<V>* d = k ? db : dw;
        float* mine = reinterpret_cast<float*>(lds[threadIdx.x / R]);
#pragma unroll
        for (int i = 0; i < N; ++i) *reinterpret_cast<FV<V>*>(mine + V * (i * R + lane)) = d[i];
        __syncthreads();
        for (int e = threadIdx.x; e < R * E / 4; e += norm_block(R)) {
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
        const int c = V * (i * R + lane);
        if (c >= a.H) continue;
        store(part + c, dw[i], V);
        if (kCenter) store(part + second + c, db[i], V);
      }
    }
  }
}

// Rows wider than the registers hold: a pass over the row for each sum and one
// for the result.  The rows of all blocks at once fit L2 where they are few (64
// x 65536 bf16 is fetched once: 17 us) or not much wider than the registers (4096
// x 20000 bf16 1.2 times: 89 us, 3.7 TB/s); 512 x 65536 fp32 is fetched three
// times: 91 us, 3.0 TB/s of what has to move.
template <class X, class Y, bool kCenter>
__global__ __launch_bounds__(1024) void norm_fwd_wide(NormFwdArgs a) {
  constexpr int R = 1024, V = width_of<X, Y>();
  __shared__ float red[3][R / 64];
  const float fH = (float)a.H;
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
    const X* x = static_cast<const X*>(a.x) + row * a.ldx;
    float mean = 0.f, s[1] = {0.f};
    if constexpr (kCenter) {
      for (int c = V * threadIdx.x; c < a.H; c += V * R) {
        const FV<V> f = widen(load<V>(x + c, a.H - c));
#pragma unroll
        for (int j = 0; j < V; ++j) s[0] += f.v[j];
      }
      RowSum<R>::run(s, red[0]);
      mean = s[0] / fH;
      if (!in_range(mean)) {
        s[0] = 0.f;
        for (int c = V * threadIdx.x; c < a.H; c += V * R) {
          const FV<V> f = widen(load<V>(x + c, a.H - c));
#pragma unroll
          for (int j = 0; j < V; ++j) s[0] += f.v[j] * kSmall;
        }
        RowSum<R>::run(s, red[2]);
        mean = s[0] / fH / kSmall;
      }
      s[0] = 0.f;
    }
    for (int c = V * threadIdx.x; c < a.H; c += V * R) {
      const FV<V> f = widen(load<V>(x + c, a.H - c));
#pragma unroll
      for (int j = 0; j < V; ++j) {
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
    for (int c = V * threadIdx.x; c < a.H; c += V * R) {
      FV<V> o = widen(load<V>(x + c, a.H - c));
#pragma unroll
      for (int j = 0; j < V; ++j) o.v[j] = (kCenter ? o.v[j] - mean : o.v[j]) * rstd;
      if (a.w) {
        const FV<V> w = load_any<V>(a.w, a.w_f32, c, a.H - c);
#pragma unroll
        for (int j = 0; j < V; ++j) o.v[j] *= w.v[j];
      }
      if (kCenter && a.b) {
        const FV<V> b = load_any<V>(a.b, a.w_f32, c, a.H - c);
#pragma unroll
        for (int j = 0; j < V; ++j) o.v[j] += b.v[j];
      }
      store(y + c, o, a.H - c);
    }
    if (!kCenter) __syncthreads();  // red[1] is free again
  }
}

// The backward of such rows: one pass for its sums, one for grad_x (512 x 65536
// fp32 116 us, x and g fetched twice; 1024 x 16384 bf16 24 us).
template <class X, class G, bool kCenter>
__global__ __launch_bounds__(1024) void norm_bwd_wide(NormBwdArgs a) {
  constexpr int R = 1024, V = width_of<X, G>(), kVals = kCenter ? 2 : 1;
  __shared__ float red[2][kVals * (R / 64)];
  const float fH = (float)a.H;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x, turn ^= 1) {
    const X* x = static_cast<const X*>(a.x) + row * a.ldx;
    const G* g = static_cast<const G*>(a.g) + row * a.ldg;
    const float mu = kCenter ? a.mean[row] : 0.f, r = a.rstd[row];
    auto values = [&](int c, FV<V>& nv, FV<V>& gw) {
      nv = widen(load<V>(x + c, a.H - c));
      gw = widen(load<V>(g + c, a.H - c));
      if (a.w) {
        const FV<V> w = load_any<V>(a.w, a.w_f32, c, a.H - c);
#pragma unroll
        for (int j = 0; j < V; ++j) gw.v[j] *= w.v[j];
      }
#pragma unroll
      for (int j = 0; j < V; ++j) nv.v[j] = kCenter ? (nv.v[j] - mu) * r : nv.v[j] * r;
      if constexpr (kCenter) zero_past(nv, a.H - c);
    };
    float s[kVals] = {};
    for (int c = V * threadIdx.x; c < a.H; c += V * R) {
      FV<V> nv, gw;
      values(c, nv, gw);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        s[0] = __builtin_fmaf(gw.v[j], nv.v[j], s[0]);
        if constexpr (kCenter) s[1] += gw.v[j];
      }
    }
    RowSum<R>::run(s, red[turn]);
    const float c1 = s[0] / fH;
    float c2 = 0.f;
    if constexpr (kCenter) c2 = s[1] / fH;
    X* gx = static_cast<X*>(a.grad_x) + row * a.H;
    for (int c = V * threadIdx.x; c < a.H; c += V * R) {
      FV<V> nv, gw;
      values(c, nv, gw);
#pragma unroll
      for (int j = 0; j < V; ++j) gw.v[j] = r * ((kCenter ? gw.v[j] - c2 : gw.v[j]) - nv.v[j] * c1);
      store(gx + c, gw, a.H - c);
    }
  }
}

// The sums of such rows: 256 vectors a block, rows p, p + P, ... (512 x 65536
// fp32 49 us, 5.5 TB/s; 1024 x 16384 bf16 13 us).
template <class X, class G, bool kCenter>
__global__ __launch_bounds__(256) void norm_sums_wide(NormBwdArgs a) {
  constexpr int V = width_of<X, G>();
  const int c = V * (blockIdx.x * 256 + threadIdx.x);
  if (c >= a.H) return;
  FV<V> dw{}, db{};
  for (int64_t row = blockIdx.y; row < a.T; row += gridDim.y) {
    const FV<V> x = widen(load<V>(static_cast<const X*>(a.x) + row * a.ldx + c, a.H - c));
    const FV<V> g = widen(load<V>(static_cast<const G*>(a.g) + row * a.ldg + c, a.H - c));
    const float mu = kCenter ? a.mean[row] : 0.f, r = a.rstd[row];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float n = kCenter ? (x.v[j] - mu) * r : x.v[j] * r;
      dw.v[j] = __builtin_fmaf(g.v[j], n, dw.v[j]);
      db.v[j] += g.v[j];
    }
  }
  float* part = a.part + (int64_t)blockIdx.y * a.Hp + c;
  store(part, dw, V);
  if (kCenter) store(part + (int64_t)gridDim.y * a.Hp, db, V);
}

struct NormSumArgs {
  const float* part;
  int P, H, Hp;
  void* out[2];  // the weight's gradient, the bias's; either may be NULL
  int f32;
};

// The blocks' sums folded as a tree, nine roundings for 512 parts (one after the
// other, 16 parts and then 32 groups, 46: the sums of a batch were farther from
// 64 bits than a column sum's): 32 columns a block, 32 groups of parts (p,
// p + 32, ...), then these groups.  Latency: 4 us for 512 parts of 4096.
constexpr int kMaxParts = 512;

__global__ __launch_bounds__(256) void norm_grad_sum(NormSumArgs a) {
  constexpr int kGroups = 32, kOfGroup = kMaxParts / kGroups;
  __shared__ float4 lds[kGroups][8];
  void* out = a.out[blockIdx.y];
  if (!out) return;
  const int k = threadIdx.x % 8, q = threadIdx.x / 8;
  const int c = 32 * blockIdx.x + 4 * k;
  float4 s[kOfGroup];
  const float* p = a.part + (int64_t)blockIdx.y * a.P * a.Hp + c;
#pragma unroll
  for (int i = 0; i < kOfGroup; ++i) {
    const int at = q + kGroups * i;
    s[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < a.Hp && at < a.P) s[i] = *reinterpret_cast<const float4*>(p + (int64_t)at * a.Hp);
  }
#pragma unroll
  for (int d = 1; d < kOfGroup; d *= 2) {
#pragma unroll
    for (int i = 0; i < kOfGroup; i += 2 * d) {
      s[i].x += s[i + d].x;
      s[i].y += s[i + d].y;
      s[i].z += s[i + d].z;
      s[i].w += s[i + d].w;
    }
  }
  lds[q][k] = s[0];
  __syncthreads();
  const int at = 32 * blockIdx.x + threadIdx.x;
  if (threadIdx.x >= 32 || at >= a.H) return;
  const float* l = reinterpret_cast<const float*>(lds) + threadIdx.x;
  float v[kGroups];
#pragma unroll
  for (int i = 0; i < kGroups; ++i) v[i] = l[32 * i];
#pragma unroll
  for (int d = 1; d < kGroups; d *= 2)
#pragma unroll
    for (int i = 0; i < kGroups; i += 2 * d) v[i] += v[i + d];
  if (a.f32) static_cast<float*>(out)[at] = v[0];
  else static_cast<uint16_t*>(out)[at] = (uint16_t)pack_bf16x2(v[0], 0.f);
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
  int slices;  // of a row, a wave each
  float scale;
};

// out[t] = scale E[id]: a wave for kRowVecs vectors a lane of a row, all loaded
// before the first is stored.  Four, or one where the rows are so few that
// all waves are there at once (48 rows of H = 2048: 3.6 -> 3.0 us).  Bound by
// HBM's random rows: 16384 of H = 2048 20 us, 4.7 TB/s.
template <class E, class O, int kRowVecs>
__global__ __launch_bounds__(256) void embed_rows(EmbedArgs a) {
  constexpr int V = width_of<E, O>();
  const int lane = threadIdx.x % 64;
  const int64_t items = (int64_t)a.T * a.slices;
  for (int64_t w = (int64_t)blockIdx.x * 4 + threadIdx.x / 64; w < items; w += (int64_t)gridDim.x * 4) {
    const int64_t t = w / a.slices;
    const int c = V * (64 * kRowVecs * (int)(w - t * a.slices) + lane);
    const int64_t id = id_at(a.ids, t);
    O* out = static_cast<O*>(a.out) + t * a.H;
    const bool ignored = id == a.ids.ignore, bad = id < 0 || id >= a.V;
    Raw<E, V> r[kRowVecs] = {};
    if (!ignored && !bad) {
      const E* row = static_cast<const E*>(a.E) + id * a.H;
#pragma unroll
      for (int i = 0; i < kRowVecs; ++i) r[i] = load<V>(row + c + 64 * V * i, a.H - c - 64 * V * i);
    }
    const float nan = __builtin_nanf("");
#pragma unroll
    for (int i = 0; i < kRowVecs; ++i) {
      FV<V> f = widen(r[i]);
#pragma unroll
      for (int j = 0; j < V; ++j) f.v[j] = ignored ? 0.f : bad ? nan : f.v[j] * a.scale;
      store(out + c + 64 * V * i, f, a.H - c - 64 * V * i);
    }
  }
}

// The gradient goes by positions of the tokens sorted by (key, t): keys[i] and
// the row perm[i].  A key is the token with its `low` lowest bits moved to the
// top (frequent tokens have low ids: these bits spread them); ids that reach
// no row have the key `none`, above all others.
struct KeyMap {
  int low, high;  // bits; low + high cover the vocabulary
  int none;
  int V;
};
__device__ __forceinline__ int key_of(const IdsArg& a, const KeyMap& m, int64_t t) {
  const int64_t id = id_at(a, t);
  if (id == a.ignore || id < 0 || id >= m.V) return m.none;
  return ((int)id & ((1 << m.low) - 1)) << m.high | (int)id >> m.low;
}
__device__ __forceinline__ int token_of(const KeyMap& m, int key) {
  return (key & ((1 << m.high) - 1)) << m.low | key >> m.high;
}

// Zeroes of the dense gradient, by the blocks of a sort's launch that do not
// sort: the sort is bound by latency and leaves the memory idle.  Rows of
// tokens that occur are written again afterwards.
struct ZeroArgs {
  char* p;        // NULL: nothing to zero
  int64_t bytes;  // even
};
__device__ __forceinline__ void zero_share(const ZeroArgs& z, int64_t block, int64_t blocks, int threads) {
  const int64_t n16 = z.bytes / 16;
  for (int64_t i = block * threads + threadIdx.x; i < n16; i += blocks * threads) {
    const u32x4 zero = {0u, 0u, 0u, 0u};
    __builtin_memcpy(z.p + 16 * i, &zero, 16);
  }
  if (block == 0 && threadIdx.x < (z.bytes - 16 * n16) / 2)
    reinterpret_cast<uint16_t*>(z.p + 16 * n16)[threadIdx.x] = 0;
}

// Up to kRankRows tokens, one launch: every block sorts all keys into buckets by
// their first ten bits in LDS (in any order), and finds the places of kTok
// tokens: the buckets before, and the tokens before it in its own, which 16
// threads count.  Up to 4096 tokens small blocks with little LDS leave the
// units to the blocks that zero; beyond, fewer blocks read all ids.
// Bound by LDS latency: 16384 tokens of text 13 us (25 for counting against all
// others), of one token 60, which all add to one counter.
constexpr int kRankRows = 16384, kBucketBits = 10, kBuckets = 1 << kBucketBits;

struct RankArgs {
  IdsArg ids;
  KeyMap map;
  int32_t* keys;
  int32_t* perm;
  int T;
  int blocks;  // that rank
  ZeroArgs zero;
};

template <int kTok>
__global__ __launch_bounds__(16 * kTok) void embed_rank(RankArgs a) {
  constexpr int kThreads = 16 * kTok, kMost = 256 * kTok, kKeys = 16;
  __shared__ uint32_t entry[kMost];      // by bucket: the key's other bits and t
  __shared__ int32_t bucket[kBuckets];   // its entries, then its first one, then its end
  __shared__ int32_t waves[kThreads / 64];
  __shared__ int32_t count[kThreads / 64][64];
  if ((int)blockIdx.x >= a.blocks) {
    zero_share(a.zero, blockIdx.x - a.blocks, gridDim.x - a.blocks, kThreads);
    return;
  }
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int keys = (a.T + kThreads - 1) / kThreads;  // of a thread
  constexpr int kTBits = 14;
  static_assert(kRankRows <= 1 << kTBits && kMost <= kRankRows, "t in an entry");
  for (int i = threadIdx.x; i < kBuckets; i += kThreads) bucket[i] = 0;
  __syncthreads();
  int key[kKeys];
#pragma unroll
  for (int i = 0; i < kKeys; ++i) {
    const int t = i * kThreads + threadIdx.x;
    key[i] = i < keys && t < a.T ? key_of(a.ids, a.map, t) : a.map.none;
  }
#pragma unroll
  for (int i = 0; i < kKeys; ++i)
    if (key[i] != a.map.none) atomicAdd(&bucket[key[i] >> a.map.high], 1);
  __syncthreads();
  // exclusive sums: kBuckets / kThreads buckets a thread
  constexpr int kPer = kBuckets / kThreads;
  int own[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    own[i] = sum;
    sum += bucket[threadIdx.x * kPer + i];
  }
  int upto = sum;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(upto, d);
    if (lane >= d) upto += o;
  }
  if (lane == 63) waves[wave] = upto;
  __syncthreads();
  int before = upto - sum;
  for (int w = 0; w < wave; ++w) before += waves[w];
#pragma unroll
  for (int i = 0; i < kPer; ++i) bucket[threadIdx.x * kPer + i] = before + own[i];
  __syncthreads();
  const int rest = (1 << a.map.high) - 1;
#pragma unroll
  for (int i = 0; i < kKeys; ++i) {
    if (key[i] == a.map.none) continue;
    const int at = atomicAdd(&bucket[key[i] >> a.map.high], 1);
    entry[at] = (uint32_t)(key[i] & rest) << kTBits | (uint32_t)(i * kThreads + threadIdx.x);
  }
  __syncthreads();
  const int tok = threadIdx.x % kTok, set = threadIdx.x / kTok;
  const int t = kTok * blockIdx.x + tok;
  const int mine = t < a.T ? key_of(a.ids, a.map, t) : a.map.none;
  int n = 0, first = 0;
  if (mine != a.map.none) {
    const int b = mine >> a.map.high;
    const uint32_t e = (uint32_t)(mine & rest) << kTBits | (uint32_t)t;
    first = b ? bucket[b - 1] : 0;
    const int end = bucket[b];
#pragma unroll 4
    for (int i = first + set; i < end; i += 16) n += entry[i] < e;
  }
  // a token's sets: lanes kTok apart, then the waves
#pragma unroll
  for (int d = kTok; d < 64; d *= 2) n += __shfl_xor(n, d);
  count[wave][lane] = n;
  __syncthreads();
  if (threadIdx.x >= kTok || t >= a.T) return;
  // places behind the tokens that reach a row
  if (t >= bucket[kBuckets - 1]) a.keys[t] = a.map.none;
  if (mine == a.map.none) return;
  int at = first;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) at += count[w][tok];
  a.keys[at] = mine;
  a.perm[at] = t;
}

// More tokens: a radix sort by digits of up to nine bits, the lowest first,
// three launches each; tiles of 4096 tokens, a wave's 1024 in order.  Bound by
// latency: 131072 tokens, two digits, 60 us in six launches (the rows after them
// take 110).
constexpr int kTile = 4096, kBins = 512;

// The lanes of a wave whose digit is this lane's.
__device__ __forceinline__ uint64_t same_digit(int d, int bits) {
  uint64_t same = ~0ull;
  for (int b = 0; b < bits; ++b) {
    const uint64_t one = __ballot((d >> b) & 1);
    same &= (d >> b) & 1 ? one : ~one;
  }
  return same;
}

struct RadixArgs {
  IdsArg ids;  // the first pass's input
  KeyMap map;
  const int32_t* keys_in;
  const int32_t* perm_in;
  int32_t* keys;
  int32_t* perm;
  int32_t* hist;   // [kBins][tiles]
  int32_t* total;  // [kBins]
  int T, tiles;
  int shift, bits, first;
  ZeroArgs zero;  // for blocks behind the tiles of the first pass's counts
};
__device__ __forceinline__ int radix_key(const RadixArgs& a, int t) {
  return a.first ? key_of(a.ids, a.map, t) : a.keys_in[t];
}

__global__ __launch_bounds__(256) void radix_count(RadixArgs a) {
  __shared__ int32_t bin[kBins];
  if ((int)blockIdx.x >= a.tiles) {
    zero_share(a.zero, blockIdx.x - a.tiles, gridDim.x - a.tiles, 256);
    return;
  }
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
    const uint64_t same = same_digit(d, a.bits) & __ballot(live);
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

// Rows of one token are summed in runs of kRun from its first on; a token of
// more rows leaves its runs' sums in parts.
constexpr int kRun = 16;

struct EmbedGradArgs {
  const int32_t* keys;
  const int32_t* perm;
  const void* g;
  int64_t ldg;
  void* grad;
  float* part;  // [2][runs][H]
  int runs;     // ceil(T / kRun)
  KeyMap map;
  int T, H;
  float scale;
  int accumulate;
  int slices;  // of the columns, a wave each
  int window;  // positions of a wave
};

// The part of the run that starts at position i: a token's first run, or a
// later one, can each start only once in kRun positions.
__device__ __forceinline__ float* part_of(const EmbedGradArgs& a, int i, bool first) {
  return a.part + ((first ? a.runs : 0) + (int64_t)(i / kRun)) * a.H;
}

// grad = old + scale * sum, or scale * sum; stored non-temporally (16384 rows of
// H = 2048 added to fp32 34 -> 30 us, else the same).
template <int V, class O>
__device__ __forceinline__ void grad_row(const EmbedGradArgs& a, O* p, const Raw<O, V>& old, const FV<V>& sum, int n) {
  FV<V> f;
#pragma unroll
  for (int j = 0; j < V; ++j) f.v[j] = a.scale * sum.v[j];
  if (a.accumulate) {
    const FV<V> o = widen(old);
#pragma unroll
    for (int j = 0; j < V; ++j) f.v[j] = o.v[j] + f.v[j];
  }
  store_once(p, f, n);
}

// Vectors by the gradient's type: an fp32 row that is read and written goes by
// 16 bytes a lane (16384 rows of H = 2048 added to fp32: 32 us, 42 by 32 bytes).
template <class O>
constexpr int grad_width() {
  return sizeof(O) == 4 ? 4 : 8;
}

// A wave takes the runs that start in a window of a.window (<= 16) positions,
// for 64 vectors of the columns: their rows follow each other in the sorted
// order, up to 15 past the window, and are loaded kBatch at a time.
template <class G, class O>
__device__ __forceinline__ void embed_window(const EmbedGradArgs& a, int p0, int slice) {
  constexpr int V = grad_width<O>(), kBatch = 8;
  const int lane = threadIdx.x % 64;
  const int32_t* k = a.keys;
  // lane l: position q = p0 + l - 16
  const int q = p0 + lane - kRun;
  const bool in = q >= 0 && q < a.T;
  const int key = in ? k[q] : -1;
  const int row = in ? a.perm[q] : 0;
  const int prev = __shfl_up(key, 1), next = __shfl_down(key, 1);
  const int key0 = __builtin_amdgcn_readlane(key, kRun);
  if (key0 == a.map.none) return;
  // the first position of a lane's token: the last one at or before it whose
  // predecessor differs (found outside where 16 rows before p0 are the same)
  const uint64_t starts = __ballot(lane > 0 && key != prev);
  const uint64_t upto = starts & (~0ull >> (63 - lane));
  int start0 = 0;
  if (!(starts & (~0ull >> (63 - kRun)))) start0 = lower_bound(k, a.T, key0);
  const int start = upto ? p0 - kRun + 63 - __builtin_clzll(upto) : start0;
  const int behind = q - start, head = lane - (behind & (kRun - 1));
  const bool mine = in && key != a.map.none && lane >= kRun && head >= kRun && head < kRun + a.window;
  const uint64_t own = __ballot(mine);
  const int token = token_of(a.map, key);
  if (!own) return;
  const bool leaves = lane == 63 || next != key;  // the token's last row (lane 63 owns nothing)
  const uint64_t ends = __ballot(mine && ((behind & (kRun - 1)) == kRun - 1 || leaves));
  const uint64_t whole = __ballot(mine && behind < kRun && leaves);  // at a run's end: the token's only run
  const int c = V * (64 * slice + lane), left = a.H - c;
  const G* g = static_cast<const G*>(a.g) + c;
  FV<V> sum{};
  const int first = __builtin_ctzll(own), last = 63 - __builtin_clzll(own);
  for (int j = first; j <= last; j += kBatch) {
    Raw<G, V> r[kBatch];
    Raw<O, V> old[kBatch];
#pragma unroll
    for (int m = 0; m < kBatch; ++m) {
      if (j + m > last) continue;
      r[m] = load<V>(g + __builtin_amdgcn_readlane(row, j + m) * a.ldg, left);
      if (a.accumulate && (whole >> (j + m) & 1))
        old[m] = load<V>(static_cast<const O*>(a.grad) + (int64_t)__builtin_amdgcn_readlane(token, j + m) * a.H + c, left);
    }
#pragma unroll
    for (int m = 0; m < kBatch; ++m) {
      if (j + m > last) continue;
      const FV<V> f = widen(r[m]);
#pragma unroll
      for (int e = 0; e < V; ++e) sum.v[e] += f.v[e];
      if (!(ends >> (j + m) & 1)) continue;
      if (whole >> (j + m) & 1) {
        O* p = static_cast<O*>(a.grad) + (int64_t)__builtin_amdgcn_readlane(token, j + m) * a.H + c;
        grad_row(a, p, old[m], sum, left);
      } else {
        const int b = __builtin_amdgcn_readlane(behind, j + m);
        const int h = __builtin_amdgcn_readlane(head, j + m) + p0 - kRun;
        store(part_of(a, h, b < kRun) + c, sum, left);
      }
      sum = FV<V>{};
    }
  }
}

// Bound by HBM's random rows and their latency: 16384 tokens of H = 2048 (6200
// distinct) added to fp32 38 us, 4.2 TB/s; 4096 of H = 4096 into bf16 19 us.
template <class G, class O>
__global__ __launch_bounds__(256) void embed_grad(EmbedGradArgs a) {
  const int64_t items = (int64_t)((a.T + a.window - 1) / a.window) * a.slices;
  for (int64_t w = (int64_t)blockIdx.x * 4 + threadIdx.x / 64; w < items; w += (int64_t)gridDim.x * 4) {
    const int i = __builtin_amdgcn_readfirstlane((int)(w / a.slices));
    embed_window<G, O>(a, i * a.window, (int)(w - (int64_t)i * a.slices));
  }
}

// Tokens of more than kRun rows: their runs' sums, in order.  A block looks for
// the first rows of such tokens in 128 positions and takes each in turn, 256
// columns at a time: eight waves sum consecutive eighths, eight parts in flight
// each, and these are summed in order.  Bound by latency: 5 to 7 us where few
// tokens have more than a few runs, 45 us for one token of 16384 rows.
template <class O>
__global__ __launch_bounds__(512) void embed_grad_join(EmbedGradArgs a) {
  constexpr int V = 4, kWaves = 8, kSpan = 128, kStarts = kSpan / kRun;
  __shared__ FV<V> lds[kWaves][64];
  __shared__ int32_t found[kStarts];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int32_t* k = a.keys;
  if (threadIdx.x < kStarts) found[threadIdx.x] = -1;
  __syncthreads();
  if (threadIdx.x < kSpan) {
    const int p = blockIdx.x * kSpan + threadIdx.x;
    const int key = p < a.T ? k[p] : a.map.none;
    const int before = p > 0 && p < a.T ? k[p - 1] : -1;
    const int behind = p + kRun < a.T ? k[p + kRun] : -1;
    // (one at most in kRun positions)
    if (key != a.map.none && behind == key && before != key) found[threadIdx.x / kRun] = p;
  }
  __syncthreads();
  for (int f = 0; f < kStarts; ++f) {
    const int s = found[f];
    if (s < 0) continue;  // the same for all waves
    const int same = k[s], token = token_of(a.map, same);
    // up to 64 runs are counted by one probe of their starts
    const int64_t q = s + (int64_t)kRun * lane;
    const uint64_t other = __ballot(q >= a.T || k[q] != same);
    const int runs = other ? __builtin_ctzll(other) : (lower_bound(k, a.T, same + 1) - s + kRun - 1) / kRun;
    const int per = (runs + kWaves - 1) / kWaves;
    const int lo = min(wave * per, runs), hi = min(lo + per, runs);
    for (int c0 = blockIdx.y * 64 * V; c0 < a.H; c0 += gridDim.y * 64 * V) {
      const int c = c0 + V * lane, n = a.H - c;
      O* grad = static_cast<O*>(a.grad) + (int64_t)token * a.H + c;
      Raw<O, V> old{};
      if (a.accumulate && wave == 0) old = load<V>(grad, n);
      FV<V> sum{};
      int r = lo;
      for (; r + 8 <= hi; r += 8) {
        Raw<float, V> raw[8];
#pragma unroll
        for (int m = 0; m < 8; ++m) raw[m] = load<V>(part_of(a, s + (r + m) * kRun, r + m == 0) + c, n);
#pragma unroll
        for (int m = 0; m < 8; ++m) {
          const FV<V> v = widen(raw[m]);
#pragma unroll
          for (int e = 0; e < V; ++e) sum.v[e] += v.v[e];
        }
      }
      for (; r < hi; ++r) {
        const FV<V> v = widen(load<V>(part_of(a, s + r * kRun, r == 0) + c, n));
#pragma unroll
        for (int e = 0; e < V; ++e) sum.v[e] += v.v[e];
      }
      lds[wave][lane] = sum;
      __syncthreads();
      if (wave == 0 && n > 0) {
#pragma unroll
        for (int w = 1; w < kWaves; ++w) {
          const FV<V> v = lds[w][lane];
#pragma unroll
          for (int e = 0; e < V; ++e) sum.v[e] += v.v[e];
        }
        grad_row(a, grad, old, sum, n);
      }
      __syncthreads();
    }
  }
}

// --- gradients of a step ---------------------------------------------------------
// Both kernels move all data once and keep none for later (non-temporal, with
// which reads reach 7.0 TB/s instead of 6.3).  The scaling takes a block for
// every few KB: a grid that strides over larger chunks moves 10 to 25 % less.
constexpr int kTensors = 96;        // of one launch (its arguments stay below 4 KB)
constexpr int kSquareElems = 8192;  // a block's unit of work, squares
constexpr int kScaleElems = 4096;   // ..., scaling

struct TensorsArgs {
  const void* in[kTensors];
  void* out[kTensors];
  int64_t n[kTensors];
  int32_t first[kTensors + 1];  // the tensor's first chunk
  uint32_t in_f32[kTensors / 32], out_f32[kTensors / 32];
  int count;
  double* part;   // sums of squares
  int parts;      // of all launches; 0: `c` holds the factor
  float* norm;
  float* c;
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

// Vectors of a chunk are dealt to the block's threads, all in flight.
template <class T>
__device__ __forceinline__ void square_sum(const T* p, int64_t n, double (&s)[4]) {
  constexpr int V = width_of<T>(), kTurns = kSquareElems / (256 * V);
  Raw<T, V> r[kTurns];
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const int c = V * (i * 256 + threadIdx.x);
    r[i] = load_once<V>(p + c, n - c);
  }
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const FV<V> f = widen(r[i]);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const double d = (double)f.v[j];
      s[j & 3] = __builtin_fma(d, d, s[j & 3]);
    }
  }
}

// part[b] = the sum of squares of chunks b, b + gridDim.x, ..., in fp64: no
// square overflows or is lost, and the sum needs no care for its order.  Bound
// by HBM: 622 M fp32 in 350 us, 7.1 TB/s (the fp64 operations hide behind it).
__global__ __launch_bounds__(256) void grads_square(TensorsArgs a) {
  __shared__ double lds[4];
  double s[4] = {0., 0., 0., 0.};
  const int chunks = a.first[a.count];
  for (int64_t chunk = blockIdx.x; chunk < chunks; chunk += gridDim.x) {
    const int i = tensor_of(a, (int)chunk);
    const int64_t at = (chunk - a.first[i]) * kSquareElems, n = a.n[i] - at;
    if (a.in_f32[i / 32] >> (i % 32) & 1) square_sum(static_cast<const float*>(a.in[i]) + at, n, s);
    else square_sum(static_cast<const uint16_t*>(a.in[i]) + at, n, s);
  }
  const double v = block_sum((s[0] + s[1]) + (s[2] + s[3]), lds);
  if (threadIdx.x == 0) a.part[blockIdx.x] = v;
}

__device__ __forceinline__ double norm_of(const double* part, int parts, double* lds) {
  double s = 0.;
#pragma unroll 4
  for (int i = threadIdx.x; i < parts; i += 256) s += part[i];
  return __builtin_sqrt(block_sum(s, lds));
}
__device__ __forceinline__ float factor_of(double norm, float max_norm) {
  return norm <= (double)max_norm ? 1.f : (float)((double)max_norm / norm);
}

// The norm, and the factor of a clipping (c not NULL).
__global__ __launch_bounds__(256) void grads_norm(const double* part, int parts, float* norm, float* c,
                                                  float max_norm) {
  __shared__ double lds[4];
  const double v = norm_of(part, parts, lds);
  if (threadIdx.x) return;
  *norm = (float)v;
  if (c) *c = factor_of(v, max_norm);
}

template <class T, class O>
__device__ __forceinline__ void scale_chunk(const T* p, O* o, int64_t n, float c) {
  constexpr int V = sizeof(T) == 2 && sizeof(O) == 2 ? 8 : 4, kTurns = kScaleElems / (256 * V);
  Raw<T, V> r[kTurns];
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const int e = V * (i * 256 + threadIdx.x);
    r[i] = load_once<V>(p + e, n - e);
  }
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const int e = V * (i * 256 + threadIdx.x);
    FV<V> f = widen(r[i]);
#pragma unroll
    for (int j = 0; j < V; ++j) f.v[j] *= c;
    store_once(o + e, f, n - e);
  }
}

// out = c grads.  A few blocks find c from the parts for themselves (one
// launch less); many read it.  Bound by HBM: 412 M fp32 -> bf16 in 396 us, 6.2
// TB/s.
__global__ __launch_bounds__(256) void grads_scale(TensorsArgs a) {
  float c;
  if (a.parts) {
    __shared__ double lds[4];
    const double norm = norm_of(a.part, a.parts, lds);
    c = factor_of(norm, a.max_norm);
    if (a.norm && blockIdx.x == 0 && threadIdx.x == 0) *a.norm = (float)norm;
  } else {
    c = *a.c;
  }
  const int chunks = a.first[a.count];
  for (int64_t chunk = blockIdx.x; chunk < chunks; chunk += gridDim.x) {
    const int i = tensor_of(a, (int)chunk);
    if (a.in[i] == a.out[i] && c == 1.f) continue;
    const int64_t at = (chunk - a.first[i]) * kScaleElems, n = a.n[i] - at;
    const bool f = a.in_f32[i / 32] >> (i % 32) & 1, of = a.out_f32[i / 32] >> (i % 32) & 1;
    const float* p = static_cast<const float*>(a.in[i]) + at;
    const uint16_t* pb = static_cast<const uint16_t*>(a.in[i]) + at;
    float* o = static_cast<float*>(a.out[i]) + at;
    uint16_t* ob = static_cast<uint16_t*>(a.out[i]) + at;
    if (f && of) scale_chunk(p, o, n, c);
    else if (f) scale_chunk(p, ob, n, c);
    else if (of) scale_chunk(pb, o, n, c);
    else scale_chunk(pb, ob, n, c);
  }
}

}  // namespace step
}  // namespace rlk
