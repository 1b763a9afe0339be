// gq_gnorm.cu -- group normalization of segments of rows (the graphs of a batch,
// channels last) with the activation behind it, forward and backward.
//
//   over the rows r of segment s and the channels c of group g (N cells):
//     mean = sum x / N,  rstd = 1 / sqrt(sum (x - mean)^2 / N + eps)
//     z = (x - mean) rstd gamma + beta,  y = act(z)
//   dz = dy act'(z),  h = dz gamma
//     dx = rstd (h - mean(h) - xhat mean(h xhat)),  dgamma = sum dz xhat,  dbeta = sum dz
//
// Everything is bound by memory.  Two forms:
//
//   short segments  one block (or, for the smallest, one warp) a segment reads its
//                   rows, makes the statistics and reads the rows again, from L1
//                   or L2: DRAM sees x once.  The backward pass's take several
//                   segments and keep their sums of dgamma and dbeta.
//   long segments   three launches: statistics of pieces (a chunk of rows cut at
//                   segment borders), their combination, and the rows again.  A piece's
//                   number is chunk + segment: neither falls along the rows and
//                   one of them grows from piece to piece, so the numbers are
//                   distinct and every kernel finds them without a table.
//
// A thread owns four channels (one where rows are not aligned for that) and walks
// rows, so groups of any width are met only when channels' sums are put together.
// Variances are sums of squares around the mean of the first eight values that
// a thread meets, then around the mean of the parts: no difference of large
// squares.  Eight values are added up by themselves before the running sum takes
// them.  All sums run in fp32 in a fixed order; those that join the pieces of
// long segments in 64 bits, and the parts of dgamma and dbeta with what each
// addition loses.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <type_traits>

#include "gq_common.cuh"
#include "gq_internal.cuh"
#include "gq_sm100.cuh"
#include "gq_train.h"

namespace gq {
namespace {

constexpr int kThreads = 256;

struct Args {
  const void* X;
  const void* dY;
  void* Y;               // or dX
  int64_t n, ldx, lddy, ldy;
  int d, groups, cg;
  const int64_t* ptr;    // s + 1 offsets, or null: one segment of n rows
  int64_t s;
  const float* gamma;
  const float* beta;
  float eps;
  float* mean;
  float* rstd;
  int vpr, tx, ry;       // vectors of a row, of a slab's row; rows at a time
  int lpg;               // lanes that put a group's channels together: a power of two
  // long segments
  int64_t rows_per, chunks;
  float2* part;          // [chunks + s][d]
  float2* hsum;          // backward: [s][groups] means of h and h xhat, negated
  float2* tot;           // backward: [chunks or blocks][d] sums of dz xhat and dz
  int64_t parts;
  float* dgamma;
  float* dbeta;
};

// Rows of a segment, kept inside [0, n] whatever ptr holds.
__device__ __forceinline__ void segment(const Args& p, int64_t j, int64_t& r0, int64_t& r1) {
  if (p.ptr == nullptr) {
    r0 = 0;
    r1 = p.n;
    return;
  }
  r0 = min(max(p.ptr[j], (int64_t)0), p.n);
  r1 = min(max(p.ptr[j + 1], r0), p.n);
}
// The first segment that ends behind row r.
__device__ __forceinline__ int64_t first_segment(const Args& p, int64_t r) {
  if (p.ptr == nullptr) return 0;
  int64_t lo = 0, hi = p.s;
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (p.ptr[mid + 1] > r)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

// ------------------------------------------------------------------- types --
// V = 4 or 1 values, two at a time where there are four
template <int V>
struct Pk {
  alignas(4 * V) float e[V];
};
template <int V>
__device__ __forceinline__ float2& two(Pk<V>& a, int k) { return reinterpret_cast<float2*>(a.e)[k]; }
template <int V>
__device__ __forceinline__ const float2& two(const Pk<V>& a, int k) { return reinterpret_cast<const float2*>(a.e)[k]; }
template <int V>
__device__ __forceinline__ Pk<V> add(const Pk<V>& a, const Pk<V>& b) {
  Pk<V> r;
  if constexpr (V == 1) {
    r.e[0] = a.e[0] + b.e[0];
  } else {
#pragma unroll
    for (int k = 0; k < V / 2; ++k) two(r, k) = add2(two(a, k), two(b, k));
  }
  return r;
}
template <int V>
__device__ __forceinline__ Pk<V> mul(const Pk<V>& a, const Pk<V>& b) {
  Pk<V> r;
  if constexpr (V == 1) {
    r.e[0] = a.e[0] * b.e[0];
  } else {
#pragma unroll
    for (int k = 0; k < V / 2; ++k) two(r, k) = mul2(two(a, k), two(b, k));
  }
  return r;
}
template <int V>
__device__ __forceinline__ Pk<V> fma(const Pk<V>& a, const Pk<V>& b, const Pk<V>& c) {
  Pk<V> r;
  if constexpr (V == 1) {
    r.e[0] = fmaf(a.e[0], b.e[0], c.e[0]);
  } else {
#pragma unroll
    for (int k = 0; k < V / 2; ++k) two(r, k) = fma2(two(a, k), two(b, k), two(c, k));
  }
  return r;
}
template <int V>
__device__ __forceinline__ Pk<V> all(float x) {
  Pk<V> r;
#pragma unroll
  for (int k = 0; k < V; ++k) r.e[k] = x;
  return r;
}
template <int V>
__device__ __forceinline__ Pk<V> neg(const Pk<V>& a) {
  Pk<V> r;
#pragma unroll
  for (int k = 0; k < V; ++k) r.e[k] = -a.e[k];
  return r;
}

// raw values of a row, as loaded
template <typename T, int V>
struct Raw {
  alignas(sizeof(T) * V) T e[V];
};
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> load(const void* base, int64_t i) {
  Raw<T, V> r;
  const T* a = static_cast<const T*>(base) + i;
  if constexpr (V == 1)
    r.e[0] = *a;
  else if constexpr (sizeof(T) == 4)
    *reinterpret_cast<uint4*>(r.e) = *reinterpret_cast<const uint4*>(a);
  else
    *reinterpret_cast<uint2*>(r.e) = *reinterpret_cast<const uint2*>(a);
  return r;
}
template <typename T, int V>
__device__ __forceinline__ Pk<V> value(const Raw<T, V>& r) {
  Pk<V> x;
  if constexpr (V == 1 || sizeof(T) == 4) {
#pragma unroll
    for (int k = 0; k < V; ++k) x.e[k] = (float)r.e[k];
  } else {
    const uint2 w = *reinterpret_cast<const uint2*>(r.e);
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {  // its bits are fp32's upper half
      x.e[0] = __uint_as_float(w.x << 16);
      x.e[1] = __uint_as_float(w.x & 0xffff0000u);
      x.e[2] = __uint_as_float(w.y << 16);
      x.e[3] = __uint_as_float(w.y & 0xffff0000u);
    } else {
      two(x, 0) = __half22float2(*reinterpret_cast<const __half2*>(&w.x));
      two(x, 1) = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
    }
  }
  return x;
}
__device__ __forceinline__ void put(float& o, float x) { o = x; }
__device__ __forceinline__ void put(__nv_bfloat16& o, float x) { o = __float2bfloat16_rn(x); }
__device__ __forceinline__ void put(__half& o, float x) { o = __float2half_rn(x); }
template <typename T, int V>
__device__ __forceinline__ void store(void* base, int64_t i, const Pk<V>& x) {
  T* a = static_cast<T*>(base) + i;
  if constexpr (V == 4 && sizeof(T) == 2) {
    uint2 w;
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
      w.x = pack_bf16x2(x.e[0], x.e[1]);
      w.y = pack_bf16x2(x.e[2], x.e[3]);
    } else {
      const __half2 p = __floats2half2_rn(x.e[0], x.e[1]), q = __floats2half2_rn(x.e[2], x.e[3]);
      w.x = *reinterpret_cast<const uint32_t*>(&p);
      w.y = *reinterpret_cast<const uint32_t*>(&q);
    }
    *reinterpret_cast<uint2*>(a) = w;
  } else {
    Raw<T, V> r;
#pragma unroll
    for (int k = 0; k < V; ++k) put(r.e[k], x.e[k]);
    if constexpr (V == 1)
      *a = r.e[0];
    else
      *reinterpret_cast<uint4*>(a) = *reinterpret_cast<const uint4*>(r.e);
  }
}

// 1 / (1 + e^-z) by the special function unit's 2^x and 1 / x (each within two
// steps): off by u (8 + 2 |z|) of itself at most.  0 and 1 where e^-z leaves
// fp32's range.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <int V>
__device__ __forceinline__ Pk<V> sigmoid(const Pk<V>& z) {
  Pk<V> t = mul(z, all<V>(-1.4426950408889634f));
#pragma unroll
  for (int k = 0; k < V; ++k) t.e[k] = ex2(t.e[k]);
  t = add(t, all<V>(1.0f));
#pragma unroll
  for (int k = 0; k < V; ++k) t.e[k] = rcp(t.e[k]);
  return t;
}
template <int ACT, int V>
__device__ __forceinline__ Pk<V> activate(const Pk<V>& z) {
  if constexpr (ACT == GQ_ACT_SILU) return mul(z, sigmoid(z));
  Pk<V> y = z;
  if constexpr (ACT == GQ_ACT_RELU) {
#pragma unroll
    for (int k = 0; k < V; ++k) y.e[k] = z.e[k] > 0.0f ? z.e[k] : 0.0f;
  }
  return y;
}
// dy act'(z)
template <int ACT, int V>
__device__ __forceinline__ Pk<V> slope(const Pk<V>& dy, const Pk<V>& z) {
  if constexpr (ACT == GQ_ACT_SILU) {
    const Pk<V> g = sigmoid(z);
    return mul(mul(dy, g), fma(z, fma(g, all<V>(-1.0f), all<V>(1.0f)), all<V>(1.0f)));
  }
  Pk<V> d = dy;
  if constexpr (ACT == GQ_ACT_RELU) {
#pragma unroll
    for (int k = 0; k < V; ++k) d.e[k] = z.e[k] > 0.0f ? dy.e[k] : 0.0f;
  }
  return d;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) x += __shfl_xor_sync(FULL, x, k);
  return x;
}
// over groups of `lanes` lanes
__device__ __forceinline__ float lane_sum(float x, int lanes) {
  for (int k = lanes >> 1; k > 0; k >>= 1) x += __shfl_xor_sync(FULL, x, k);
  return x;
}

// ---------------------------------------------------------- sums of a piece --
// Several rows are read before the first is used (and, where the output may be
// an input, before the first is written: the compiler cannot move a read ahead
// of a write by itself).
template <int V>
struct Ahead {
  static constexpr int sums = 8, sums_bwd = 4, fwd = V == 1 ? 8 : 4, bwd = V == 1 ? 8 : 4;
};

// Rows [r0, r1) of one thread's channels: mean and sum of squares around it.
template <typename T, int V>
__device__ __forceinline__ void spread(const Args& p, int64_t r0, int64_t r1, int ry, int c, Pk<V>& mean, Pk<V>& m2) {
  constexpr int U = Ahead<V>::sums;
  Pk<V> k = all<V>(0.0f), s = k, q = k;
  const int64_t first = r0 + ry;
  const int rows = first < r1 ? (int)((r1 - first + p.ry - 1) / p.ry) : 0;
  const T* x = static_cast<const T*>(p.X) + first * p.ldx + c;
  const int64_t step = (int64_t)p.ry * p.ldx;
  auto total = [](const Pk<V>(&y)[U]) {
    return add(add(add(y[0], y[1]), add(y[2], y[3])), add(add(y[4], y[5]), add(y[6], y[7])));
  };
  static_assert(U == 8, "total");
  int i = 0;
  for (; i + U <= rows; i += U) {
    Raw<T, V> w[U];
    Pk<V> y[U];
#pragma unroll
    for (int u = 0; u < U; ++u) w[u] = load<T, V>(x, u * step);
    x += U * step;
#pragma unroll
    for (int u = 0; u < U; ++u) y[u] = value(w[u]);
    if (i == 0) k = mul(total(y), all<V>(-1.0f / U));
#pragma unroll
    for (int u = 0; u < U; ++u) y[u] = add(y[u], k);
    s = add(s, total(y));
#pragma unroll
    for (int u = 0; u < U; ++u) y[u] = mul(y[u], y[u]);
    q = add(q, total(y));
  }
  if (i == 0 && rows > 0) k = neg(value(load<T, V>(x, 0)));
  for (; i < rows; ++i, x += step) {
    const Pk<V> y = add(value(load<T, V>(x, 0)), k);
    s = add(s, y);
    q = fma(y, y, q);
  }
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const float m = rows > 0 ? __fdiv_rn(s.e[e], (float)rows) : 0.0f;  // the reciprocal would err the same way everywhere
    mean.e[e] = m - k.e[e];
    m2.e[e] = fmaxf(fmaf(-s.e[e], m, q.e[e]), 0.0f);
    if (!(q.e[e] == q.e[e])) m2.e[e] = q.e[e];  // fmaxf would drop a NaN
  }
}

// What the backward pass needs of a thread's channels (mean negated).
template <int V>
struct Chan {
  Pk<V> mu, rs, ga, sc, be;
};
template <int V>
__device__ __forceinline__ void channels(const Args& p, int64_t j, int c, Chan<V>& h) {
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const int64_t g = j * p.groups + (c + e) / p.cg;
    h.mu.e[e] = -p.mean[g];
    h.rs.e[e] = p.rstd[g];
    h.ga.e[e] = p.gamma != nullptr ? p.gamma[c + e] : 1.0f;
    h.sc.e[e] = __fmul_rn(h.rs.e[e], h.ga.e[e]);
    h.be.e[e] = p.beta != nullptr ? p.beta[c + e] : 0.0f;
  }
}

// z once more.  ReLU's from sc = rstd gamma, by forward's own operations: next to 0
// another order of them has another sign, and ReLU would stop gradients of
// values that it let through.  SiLU's slope is smooth, and xhat is there.
template <int ACT, int V>
__device__ __forceinline__ Pk<V> again(const Pk<V>& xc, const Pk<V>& xh, const Chan<V>& h) {
  return ACT == GQ_ACT_RELU ? fma(xc, h.sc, h.be) : fma(xh, h.ga, h.be);
}

// sums of dz xhat and of dz
template <typename T, int V, int ACT>
__device__ __forceinline__ void slopes(const Args& p, int64_t r0, int64_t r1, int ry, int c, const Chan<V>& h, Pk<V>& a,
                                       Pk<V>& b) {
  constexpr int U = Ahead<V>::sums_bwd;
  a = b = all<V>(0.0f);
  const int64_t first = r0 + ry;
  const int rows = first < r1 ? (int)((r1 - first + p.ry - 1) / p.ry) : 0;
  const T* x = static_cast<const T*>(p.X) + first * p.ldx + c;
  const T* y = static_cast<const T*>(p.dY) + first * p.lddy + c;
  const int64_t sx = (int64_t)p.ry * p.ldx, sy = (int64_t)p.ry * p.lddy;
  auto use = [&](const Raw<T, V>& wx, const Raw<T, V>& wy) {
    const Pk<V> xc = add(value(wx), h.mu), xh = mul(xc, h.rs);
    const Pk<V> dz = ACT == GQ_ACT_NONE ? value(wy) : slope<ACT>(value(wy), again<ACT>(xc, xh, h));
    a = fma(dz, xh, a);
    b = add(b, dz);
  };
  int i = 0;
  for (; i + U <= rows; i += U) {
    Raw<T, V> wx[U], wy[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      wx[u] = load<T, V>(x, u * sx);
      wy[u] = load<T, V>(y, u * sy);
    }
    x += U * sx;
    y += U * sy;
#pragma unroll
    for (int u = 0; u < U; ++u) use(wx[u], wy[u]);
  }
  for (; i < rows; ++i, x += sx, y += sy) use(load<T, V>(x, 0), load<T, V>(y, 0));
}

template <typename T, int V, int ACT>
__device__ __forceinline__ void apply(const Args& p, int64_t r0, int64_t r1, int ry, int c, const Pk<V>& mu, const Pk<V>& sc,
                                      const Pk<V>& be) {
  constexpr int U = Ahead<V>::fwd;
  const int64_t first = r0 + ry;
  const int rows = first < r1 ? (int)((r1 - first + p.ry - 1) / p.ry) : 0;
  const T* x = static_cast<const T*>(p.X) + first * p.ldx + c;
  T* o = static_cast<T*>(p.Y) + first * p.ldy + c;
  const int64_t sx = (int64_t)p.ry * p.ldx, so = (int64_t)p.ry * p.ldy;
  int i = 0;
  for (; i + U <= rows; i += U) {
    Raw<T, V> w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) w[u] = load<T, V>(x, u * sx);
    x += U * sx;
#pragma unroll
    for (int u = 0; u < U; ++u) store<T, V>(o, u * so, activate<ACT>(fma(add(value(w[u]), mu), sc, be)));
    o += U * so;
  }
  for (; i < rows; ++i, x += sx, o += so) store<T, V>(o, 0, activate<ACT>(fma(add(value(load<T, V>(x, 0)), mu), sc, be)));
}

template <typename T, int V, int ACT>
__device__ __forceinline__ void apply_bwd(const Args& p, int64_t r0, int64_t r1, int ry, int c, const Chan<V>& h,
                                          const Pk<V>& h1, const Pk<V>& h2) {  // the means of h and h xhat, negated
  constexpr int U = Ahead<V>::bwd;
  Pk<V> k1, k2;  // ReLU has sc: with rstd in the means too, it holds no gamma beside it
  if constexpr (ACT == GQ_ACT_RELU) {
    k1 = mul(h.rs, h1);
    k2 = mul(h.rs, h2);
  }
  const int64_t first = r0 + ry;
  const int rows = first < r1 ? (int)((r1 - first + p.ry - 1) / p.ry) : 0;
  const T* x = static_cast<const T*>(p.X) + first * p.ldx + c;
  const T* y = static_cast<const T*>(p.dY) + first * p.lddy + c;
  T* o = static_cast<T*>(p.Y) + first * p.ldy + c;
  const int64_t sx = (int64_t)p.ry * p.ldx, sy = (int64_t)p.ry * p.lddy, so = (int64_t)p.ry * p.ldy;
  auto use = [&](const Raw<T, V>& wx, const Raw<T, V>& wy) {
    const Pk<V> xc = add(value(wx), h.mu), xh = mul(xc, h.rs);
    const Pk<V> dz = ACT == GQ_ACT_NONE ? value(wy) : slope<ACT>(value(wy), again<ACT>(xc, xh, h));
    if constexpr (ACT == GQ_ACT_RELU) return fma(dz, h.sc, fma(xh, k2, k1));
    return mul(h.rs, fma(xh, h2, fma(dz, h.ga, h1)));
  };
  int i = 0;
  for (; i + U <= rows; i += U) {
    Raw<T, V> wx[U], wy[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      wx[u] = load<T, V>(x, u * sx);
      wy[u] = load<T, V>(y, u * sy);
    }
    x += U * sx;
    y += U * sy;
#pragma unroll
    for (int u = 0; u < U; ++u) store<T, V>(o, u * so, use(wx[u], wy[u]));
    o += U * so;
  }
  for (; i < rows; ++i, x += sx, y += sy, o += so) store<T, V>(o, 0, use(load<T, V>(x, 0), load<T, V>(y, 0)));
}

// Rows of thread `ry` among `rows`.
__device__ __forceinline__ int rows_of(int64_t rows, int ry, int step) {
  return ry < rows ? (int)((rows - ry + step - 1) / step) : 0;
}

// Channel `k` of the slab from its threads' means and squares in red.
template <int V>
__device__ __forceinline__ float2 merge(const float2* red, const Args& p, int k, int64_t rows) {
  const int tv = k / V, e = k - tv * V;
  float s = 0.0f;
  for (int y = 0; y < p.ry; ++y) s = fmaf((float)rows_of(rows, y, p.ry), red[(y * p.tx + tv) * V + e].x, s);
  const float mean = s / (float)rows;
  float q = 0.0f;
  for (int y = 0; y < p.ry; ++y) {
    const float2 w = red[(y * p.tx + tv) * V + e];
    const float dev = w.x - mean;
    q += fmaf((float)rows_of(rows, y, p.ry) * dev, dev, w.y);
  }
  return make_float2(mean, q);
}

// (mean, squares around it) of na rows and of nb more.
__device__ __forceinline__ float2 join(const float2& a, int na, const float2& b, int nb) {
  const float f = (float)nb / (float)(na + nb), dev = b.x - a.x;
  return make_float2(fmaf(dev, f, a.x), a.y + fmaf((float)na * f * dev, dev, b.y));
}

template <int V>
__device__ __forceinline__ float2 add_up(const float2* red, const Args& p, int k) {
  const int tv = k / V, e = k - tv * V;
  float2 s = make_float2(0.0f, 0.0f);
  for (int y = 0; y < p.ry; ++y) {
    const float2 w = red[(y * p.tx + tv) * V + e];
    s.x += w.x;
    s.y += w.y;
  }
  return s;
}

// ---------------------------------------------------------- short segments --
// GROUP threads, a warp or the whole block, take a segment, kPieceRows rows of a
// thread at a time: none has more where the longest segment is what the caller
// said, and where it is far longer the sums stay as short as long segments'.
constexpr int kPieceRows = 1024;
// Shared memory of each
// of them: [d] channel values, the backward kernel's [d] sums over its segments,
// [GROUP x V] of the threads'.
template <int GROUP>
__device__ __forceinline__ void group_sync() {
  if constexpr (GROUP == 32)
    __syncwarp();
  else
    __syncthreads();
}

template <typename T, int V, int ACT, int GROUP>
__global__ void __launch_bounds__(kThreads, 4) short_fwd_kernel(const Args p) {
  extern __shared__ float2 sm[];
  constexpr int per_block = kThreads / GROUP, warps = GROUP / 32;
  const int t = threadIdx.x % GROUP, unit = threadIdx.x / GROUP;
  float2* ch = sm + unit * (p.d + GROUP * V);
  float2* red = ch + p.d;
  grid_wait();
  const int tx = t % p.tx, ry = t / p.tx;
  const int piece = kPieceRows * p.ry;
  const int warp = t >> 5, lane = t & 31;
  for (int64_t j = (int64_t)blockIdx.x * per_block + unit; j < p.s; j += (int64_t)gridDim.x * per_block) {
    int64_t r0, r1;
    segment(p, j, r0, r1);
    const int64_t rows = r1 - r0;
    if (rows == 0) {
      for (int g = t; g < p.groups; g += GROUP) {
        p.mean[j * p.groups + g] = 0.0f;
        p.rstd[j * p.groups + g] = __frcp_rn(__fsqrt_rn(p.eps));
      }
      continue;
    }
    for (int v0 = 0; v0 < p.vpr; v0 += p.tx) {
      const int c = (v0 + tx) * V;
      int done = 0;
      do {
        const int more = min((int)rows - done, piece);
        if (ry < p.ry && v0 + tx < p.vpr) {
          Pk<V> mean, m2;
          spread<T, V>(p, r0 + done, r0 + done + more, ry, c, mean, m2);
#pragma unroll
          for (int e = 0; e < V; ++e) red[(ry * p.tx + tx) * V + e] = make_float2(mean.e[e], m2.e[e]);
        }
        group_sync<GROUP>();
        for (int k = t; k < min(p.tx, p.vpr - v0) * V; k += GROUP) {
          float2 w = merge<V>(red, p, k, more);
          if (done > 0) w = join(ch[v0 * V + k], done, w, more);
          ch[v0 * V + k] = w;
        }
        group_sync<GROUP>();
        done += more;
      } while (done < (int)rows);
    }
    const int at_once = 32 / p.lpg, sub = lane % p.lpg;
    for (int g0 = warp * at_once; g0 < p.groups; g0 += warps * at_once) {
      const int g = g0 + lane / p.lpg, end = g < p.groups ? p.cg : 0;
      float2* w = ch + (g < p.groups ? g * p.cg : 0);
      float s = 0.0f, q = 0.0f;
      for (int k = sub; k < end; k += p.lpg) s += w[k].x;
      const float mean = lane_sum(s, p.lpg) / (float)p.cg;
      for (int k = sub; k < end; k += p.lpg) {
        const float dev = w[k].x - mean;
        q += fmaf((float)rows * dev, dev, w[k].y);
      }
      const float var = lane_sum(q, p.lpg) / ((float)rows * (float)p.cg);
      const float rstd = __frcp_rn(__fsqrt_rn(var + p.eps));
      for (int k = sub; k < end; k += p.lpg) w[k] = make_float2(mean, rstd);
      if (sub == 0 && g < p.groups) {
        p.mean[j * p.groups + g] = mean;
        p.rstd[j * p.groups + g] = rstd;
      }
    }
    group_sync<GROUP>();
    for (int v0 = 0; v0 < p.vpr; v0 += p.tx) {
      const int c = (v0 + tx) * V;
      if (ry < p.ry && v0 + tx < p.vpr) {
        Pk<V> mu, sc, be;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float2 w = ch[c + e];
          mu.e[e] = -w.x;
          sc.e[e] = __fmul_rn(w.y, p.gamma != nullptr ? p.gamma[c + e] : 1.0f);
          be.e[e] = p.beta != nullptr ? p.beta[c + e] : 0.0f;
        }
        apply<T, V, ACT>(p, r0, r1, ry, c, mu, sc, be);
      }
    }
    group_sync<GROUP>();
  }
}

template <typename T, int V, int ACT, int GROUP>
__global__ void __launch_bounds__(kThreads, 3) short_bwd_kernel(const Args p) {
  extern __shared__ float2 sm[];
  constexpr int per_block = kThreads / GROUP, warps = GROUP / 32;
  const int t = threadIdx.x % GROUP, unit = threadIdx.x / GROUP;
  float2* ch = sm + unit * (2 * p.d + GROUP * V);
  float2* tot = ch + p.d;
  float2* red = tot + p.d;
  grid_wait();
  const int tx = t % p.tx, ry = t / p.tx;
  const int piece = kPieceRows * p.ry;
  const int warp = t >> 5, lane = t & 31;
  for (int k = t; k < p.d; k += GROUP) tot[k] = make_float2(0.0f, 0.0f);
  group_sync<GROUP>();
  for (int64_t j = (int64_t)blockIdx.x * per_block + unit; j < p.s; j += (int64_t)gridDim.x * per_block) {
    int64_t r0, r1;
    segment(p, j, r0, r1);
    const int64_t rows = r1 - r0;
    if (rows == 0) continue;
    for (int v0 = 0; v0 < p.vpr; v0 += p.tx) {
      const int c = (v0 + tx) * V;
      for (int64_t r = r0; r < r1; r += piece) {
        if (ry < p.ry && v0 + tx < p.vpr) {
          Chan<V> h;
          Pk<V> a, b;
          channels<V>(p, j, c, h);
          slopes<T, V, ACT>(p, r, min(r1, r + piece), ry, c, h, a, b);
#pragma unroll
          for (int e = 0; e < V; ++e) red[(ry * p.tx + tx) * V + e] = make_float2(a.e[e], b.e[e]);
        }
        group_sync<GROUP>();
        for (int k = t; k < min(p.tx, p.vpr - v0) * V; k += GROUP) {
          const float2 w = add_up<V>(red, p, k), o = r == r0 ? make_float2(0.0f, 0.0f) : ch[v0 * V + k];
          ch[v0 * V + k] = make_float2(o.x + w.x, o.y + w.y);
          tot[v0 * V + k].x += w.x;
          tot[v0 * V + k].y += w.y;
        }
        group_sync<GROUP>();
      }
    }
    const int at_once = 32 / p.lpg, sub = lane % p.lpg;
    for (int g0 = warp * at_once; g0 < p.groups; g0 += warps * at_once) {
      const int g = g0 + lane / p.lpg, end = g < p.groups ? p.cg : 0, c0 = g < p.groups ? g * p.cg : 0;
      float2* w = ch + c0;
      float s1 = 0.0f, s2 = 0.0f;
      for (int k = sub; k < end; k += p.lpg) {
        const float ga = p.gamma != nullptr ? p.gamma[c0 + k] : 1.0f;
        s1 = fmaf(ga, w[k].y, s1);
        s2 = fmaf(ga, w[k].x, s2);
      }
      const float inv = -1.0f / ((float)rows * (float)p.cg);
      s1 = lane_sum(s1, p.lpg) * inv;
      s2 = lane_sum(s2, p.lpg) * inv;
      for (int k = sub; k < end; k += p.lpg) w[k] = make_float2(s1, s2);
    }
    group_sync<GROUP>();
    for (int v0 = 0; v0 < p.vpr; v0 += p.tx) {
      const int c = (v0 + tx) * V;
      if (ry < p.ry && v0 + tx < p.vpr) {
        Chan<V> h;
        Pk<V> h1, h2;
        channels<V>(p, j, c, h);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float2 w = ch[c + e];
          h1.e[e] = w.x;
          h2.e[e] = w.y;
        }
        apply_bwd<T, V, ACT>(p, r0, r1, ry, c, h, h1, h2);
      }
    }
    group_sync<GROUP>();
  }
  for (int k = t; k < p.d; k += GROUP) p.tot[((int64_t)blockIdx.x * per_block + unit) * p.d + k] = tot[k];
}

// ----------------------------------------------------------- long segments --
// block: chunk blockIdx.x of rows, slab blockIdx.y of channels
template <typename T, int V>
__global__ void __launch_bounds__(kThreads, 4) stats_kernel(const Args p) {
  extern __shared__ float2 red[];
  grid_wait();
  const int t = threadIdx.x, tx = t % p.tx, ry = t / p.tx;
  const int v0 = blockIdx.y * p.tx, c = (v0 + tx) * V;
  const bool live = ry < p.ry && v0 + tx < p.vpr;
  const int64_t chunk = blockIdx.x, a = chunk * p.rows_per, b = min(p.n, a + p.rows_per);
  for (int64_t j = first_segment(p, a); j < p.s; ++j) {
    int64_t r0, r1;
    segment(p, j, r0, r1);
    if (r0 >= b) break;
    r0 = max(r0, a);
    r1 = min(r1, b);
    if (r1 <= r0) continue;
    if (live) {
      Pk<V> mean, m2;
      spread<T, V>(p, r0, r1, ry, c, mean, m2);
#pragma unroll
      for (int e = 0; e < V; ++e) red[(ry * p.tx + tx) * V + e] = make_float2(mean.e[e], m2.e[e]);
    }
    __syncthreads();
    for (int k = t; k < min(p.tx, p.vpr - v0) * V; k += blockDim.x)
      p.part[(chunk + j) * p.d + v0 * V + k] = merge<V>(red, p, k, r1 - r0);
    __syncthreads();
  }
}

// A block (BLOCK) or a warp a segment and group: its pieces' channels together,
// in 64 bits: a mean over millions of cells can be thousands of times smaller
// than they are (2,449,029 x 16 of them: off by 2e-6 of itself in fp32, 5e-8 so).
constexpr int kCombine = 512;
template <bool BLOCK>
__device__ __forceinline__ double unit_sum(double x, double* sh) {
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) x += __shfl_xor_sync(FULL, x, k);
  if (!BLOCK) return x;
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = x;
  __syncthreads();
  double s = 0.0;
  for (int w = 0; w < kCombine / 32; ++w) s += sh[w];
  return s;
}
template <bool BWD, bool BLOCK>
__global__ void __launch_bounds__(kCombine) combine_kernel(const Args p) {
  __shared__ double sh[kCombine / 32];
  grid_wait();
  constexpr int per = BLOCK ? 1 : kCombine / 32, step = BLOCK ? kCombine : 32;
  const int64_t unit = (int64_t)blockIdx.x * per + (BLOCK ? 0 : threadIdx.x >> 5);
  const int lane = BLOCK ? threadIdx.x : threadIdx.x & 31;
  if (unit >= p.s * p.groups) return;
  const int64_t j = unit / p.groups;
  const int g = (int)(unit - j * p.groups);
  int64_t r0, r1;
  segment(p, j, r0, r1);
  const int64_t rows = r1 - r0;
  if (rows == 0) {
    if (!BWD && lane == 0) {
      p.mean[unit] = 0.0f;
      p.rstd[unit] = __frcp_rn(__fsqrt_rn(p.eps));
    }
    return;
  }
  const int64_t c0 = r0 / p.rows_per, c1 = (r1 - 1) / p.rows_per;
  const int64_t cells = (c1 - c0 + 1) * p.cg;
  auto count = [&](int64_t k) {  // rows of the segment's piece in its k-th chunk
    return (float)(min(r1, (c0 + k + 1) * p.rows_per) - max(r0, (c0 + k) * p.rows_per));
  };
  double s1 = 0.0, s2 = 0.0;
  for (int64_t i = lane; i < cells; i += step) {
    const int64_t k = i / p.cg;
    const int c = g * p.cg + (int)(i - k * p.cg);
    const float2 w = p.part[(c0 + k + j) * p.d + c];
    if (BWD) {
      const float ga = p.gamma != nullptr ? p.gamma[c] : 1.0f;
      s1 += (double)ga * w.y;
      s2 += (double)ga * w.x;
    } else {
      s1 += (double)count(k) * w.x;
    }
  }
  const double inv = 1.0 / ((double)rows * p.cg);
  s1 = unit_sum<BLOCK>(s1, sh) * inv;
  if constexpr (BWD) {
    s2 = unit_sum<BLOCK>(s2, sh) * inv;
    if (lane == 0) p.hsum[unit] = make_float2(-(float)s1, -(float)s2);
  } else {
    const float mean = (float)s1;
    for (int64_t i = lane; i < cells; i += step) {
      const int64_t k = i / p.cg;
      const float2 w = p.part[(c0 + k + j) * p.d + g * p.cg + (int)(i - k * p.cg)];
      const float dev = w.x - mean;
      s2 += (double)fmaf(count(k) * dev, dev, w.y);
    }
    s2 = unit_sum<BLOCK>(s2, sh) * inv;
    if (lane == 0) {
      p.mean[unit] = mean;
      p.rstd[unit] = __frcp_rn(__fsqrt_rn((float)s2 + p.eps));
    }
  }
}

template <typename T, int V, int ACT>
__global__ void __launch_bounds__(kThreads, 4) apply_kernel(const Args p) {
  grid_wait();
  const int t = threadIdx.x, tx = t % p.tx, ry = t / p.tx;
  const int v0 = blockIdx.y * p.tx, c = (v0 + tx) * V;
  if (ry >= p.ry || v0 + tx >= p.vpr) return;
  const int64_t a = (int64_t)blockIdx.x * p.rows_per, b = min(p.n, a + p.rows_per);
  for (int64_t j = first_segment(p, a); j < p.s; ++j) {
    int64_t r0, r1;
    segment(p, j, r0, r1);
    if (r0 >= b) break;
    r0 = max(r0, a);
    r1 = min(r1, b);
    if (r1 <= r0) continue;
    Pk<V> mu, sc, be;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int64_t g = j * p.groups + (c + e) / p.cg;
      mu.e[e] = -p.mean[g];
      sc.e[e] = __fmul_rn(p.rstd[g], p.gamma != nullptr ? p.gamma[c + e] : 1.0f);
      be.e[e] = p.beta != nullptr ? p.beta[c + e] : 0.0f;
    }
    apply<T, V, ACT>(p, r0, r1, ry, c, mu, sc, be);
  }
}

template <typename T, int V, int ACT>
__global__ void __launch_bounds__(kThreads, 4) slopes_kernel(const Args p) {
  extern __shared__ float2 red[];
  grid_wait();
  const int t = threadIdx.x, tx = t % p.tx, ry = t / p.tx;
  const int v0 = blockIdx.y * p.tx, c = (v0 + tx) * V;
  const bool live = ry < p.ry && v0 + tx < p.vpr;
  const int64_t chunk = blockIdx.x, a = chunk * p.rows_per, b = min(p.n, a + p.rows_per);
  Pk<V> ta = all<V>(0.0f), tb = ta;
  for (int64_t j = first_segment(p, a); j < p.s; ++j) {
    int64_t r0, r1;
    segment(p, j, r0, r1);
    if (r0 >= b) break;
    r0 = max(r0, a);
    r1 = min(r1, b);
    if (r1 <= r0) continue;
    if (live) {
      Chan<V> h;
      Pk<V> sa, sb;
      channels<V>(p, j, c, h);
      slopes<T, V, ACT>(p, r0, r1, ry, c, h, sa, sb);
      ta = add(ta, sa);
      tb = add(tb, sb);
#pragma unroll
      for (int e = 0; e < V; ++e) red[(ry * p.tx + tx) * V + e] = make_float2(sa.e[e], sb.e[e]);
    }
    __syncthreads();
    for (int k = t; k < min(p.tx, p.vpr - v0) * V; k += blockDim.x)
      p.part[(chunk + j) * p.d + v0 * V + k] = add_up<V>(red, p, k);
    __syncthreads();
  }
  if (live) {
#pragma unroll
    for (int e = 0; e < V; ++e) red[(ry * p.tx + tx) * V + e] = make_float2(ta.e[e], tb.e[e]);
  }
  __syncthreads();
  for (int k = t; k < min(p.tx, p.vpr - v0) * V; k += blockDim.x)
    p.tot[chunk * p.d + v0 * V + k] = add_up<V>(red, p, k);
}

template <typename T, int V, int ACT>
__global__ void __launch_bounds__(kThreads, 4) apply_bwd_kernel(const Args p) {
  grid_wait();
  const int t = threadIdx.x, tx = t % p.tx, ry = t / p.tx;
  const int v0 = blockIdx.y * p.tx, c = (v0 + tx) * V;
  if (ry >= p.ry || v0 + tx >= p.vpr) return;
  const int64_t a = (int64_t)blockIdx.x * p.rows_per, b = min(p.n, a + p.rows_per);
  for (int64_t j = first_segment(p, a); j < p.s; ++j) {
    int64_t r0, r1;
    segment(p, j, r0, r1);
    if (r0 >= b) break;
    r0 = max(r0, a);
    r1 = min(r1, b);
    if (r1 <= r0) continue;
    Chan<V> h;
    Pk<V> h1, h2;
    channels<V>(p, j, c, h);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float2 w = p.hsum[j * p.groups + (c + e) / p.cg];
      h1.e[e] = w.x;
      h2.e[e] = w.y;
    }
    apply_bwd<T, V, ACT>(p, r0, r1, ry, c, h, h1, h2);
  }
}

// dgamma, dbeta from the parts' sums: a block takes kSumC channels, 128 parts at a time.
constexpr int kSumC = 8, kSumThreads = 1024;
__global__ void __launch_bounds__(kSumThreads) columns_kernel(const Args p) {
  __shared__ Sum2 sh[kSumThreads / 32][2][kSumC];
  grid_wait();
  const int x = threadIdx.x % kSumC, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * kSumC + x;
  Sum2 ga{}, be{};
  if (c < p.d)
    for (int64_t k = threadIdx.x / kSumC; k < p.parts; k += kSumThreads / kSumC) {
      const float2 w = p.tot[k * p.d + c];
      ga.add(w.x);
      be.add(w.y);
    }
  auto lanes = [&] {
    for (int o = kSumC; o < 32; o *= 2) {
      ga.add(ga.from_lane(o));
      be.add(be.from_lane(o));
    }
  };
  lanes();
  if (lane < kSumC) {
    sh[warp][0][x] = ga;
    sh[warp][1][x] = be;
  }
  __syncthreads();
  if (warp > 0) return;
  ga = sh[lane / kSumC][0][x];
  be = sh[lane / kSumC][1][x];
  for (int w = lane / kSumC + 32 / kSumC; w < kSumThreads / 32; w += 32 / kSumC) {
    ga.add(sh[w][0][x]);
    be.add(sh[w][1][x]);
  }
  lanes();
  if (lane < kSumC && c < p.d) {
    if (p.dgamma != nullptr) p.dgamma[c] = ga.value();
    if (p.dbeta != nullptr) p.dbeta[c] = be.value();
  }
}

// -------------------------------------------------------------------- host --
bool valid_type(int type) { return type == GQ_F32 || type == GQ_BF16 || type == GQ_F16; }
int type_bytes(int type) { return type == GQ_F32 ? 4 : 2; }

struct Plan {
  bool brief;            // a block or a warp a segment
  int group;             // threads of a segment
  int tx, ry, vpr, slabs;
  int64_t rows_per, chunks, blocks, parts;
};

// Short segments have one launch and read DRAM once, but a block reads alone: 10
// us and 10 more for every 100 KB (forward; backward 17).  Long ones have three
// launches and every SM.  Measured, 256 bf16 channels, short | long, forward and
// backward: 1 segment of 64 KB 15, 21 | as a long one of 1 MB 22, 22; 4 of 256 KB 35, 56
// | 26, 26; 32 of 256 KB 35, 57 | 39, 43; 128 of 512 KB 87, 136 | 94, 133; 512 of
// 512 KB 150, 265 | 215, 338 us.
int64_t short_bytes(int64_t s) {
  const int64_t sms = sm_count();
  return s < sms / 8 ? 128 << 10 : s < sms / 2 ? 256 << 10 : 512 << 10;
}
// A warp instead of a block takes a segment where it has at most kWarpVectors for
// each lane and there are enough of them: 20,000 segments of 512 vectors forward 72 us
// with warps, 412 with blocks, of 1,024 vectors 156 and 316, of 1,600 279 and 285,
// of 3,840 596 and 453.
constexpr int kShortMaxD = 8192, kWarpMaxD = 512, kWarpVectors = 48;

Plan make_plan(int64_t n, int d, int64_t s, int64_t max_rows, int bytes, int v, bool bwd) {
  Plan z{};
  z.vpr = d / v;
  const int64_t longest = max_rows > 0 && max_rows < n ? max_rows : s <= 1 || max_rows > 0 ? n : 4 * (n / s + 1);
  z.brief = longest * d * bytes <= short_bytes(s) && d <= kShortMaxD;
  const int64_t mean = n / (s > 0 ? s : 1) + 1;
  z.group = z.brief && d <= kWarpMaxD && mean * z.vpr <= 32 * kWarpVectors && s > 4 * (int64_t)sm_count() ? 32 : kThreads;
  z.tx = z.vpr < z.group ? z.vpr : z.group;
  z.ry = z.group / z.tx;
  z.slabs = (z.vpr + z.tx - 1) / z.tx;
  const int64_t sms = sm_count();
  if (z.brief) {
    const int64_t per_block = kThreads / z.group;
    // the backward blocks' sums are written and read once a block
    const int64_t most = bwd ? 3 * sms : 0x7fffffff, want = (s + per_block - 1) / per_block;
    z.blocks = want < most ? want : most;
    z.parts = z.blocks * per_block;
    return z;
  }
  // 16 chunks an SM, of at least 4 rows a thread
  int64_t chunks = 16 * sms / z.slabs;
  const int64_t rows = 4 * (int64_t)z.ry;
  if (chunks > (n + rows - 1) / rows) chunks = (n + rows - 1) / rows;
  if (chunks < 1) chunks = 1;
  z.rows_per = (n + chunks - 1) / chunks;
  z.chunks = (n + z.rows_per - 1) / z.rows_per;
  z.parts = z.chunks;
  return z;
}

constexpr int kVec = 4;

// The workspace does not depend on the matrices' alignment: the larger of both vector widths'.
size_t workspace(int64_t n, int d, int groups, int type, int64_t s, int64_t max_rows, bool bwd) {
  size_t most = 0;
  for (int v : {1, kVec}) {
    if (d % v) continue;
    const Plan z = make_plan(n, d, s, max_rows, type_bytes(type), v, bwd);
    size_t b = 0;
    if (z.brief)
      b = bwd ? (size_t)z.parts * d * 8 : 0;
    else
      b = ((size_t)(z.chunks + s) * d * 8 + 255) / 256 * 256 +
          (bwd ? ((size_t)s * groups * 8 + 255) / 256 * 256 + (size_t)z.chunks * d * 8 : 0);
    if (b > most) most = b;
  }
  return most;
}

// A block for each segment and group where that has more than 1,024 values to
// put together on average, else a warp.  The whole pass forward, SiLU, fp32 x 256,
// block | warp, us: one segment of 2,449,029 in 1, 16, 256 groups 2,379 | 18,257, 1,204 |
// 2,431, 1,135 | 1,208; 16 in one group 1,204 | 2,379; 200 of 3,000 in one 330 | 426, in 8
// 374 | 323; 2,000 in one 1,218 | 1,153, in 16 2,280 | 1,194.  With one segment and few
// groups a single SM puts everything together: half of the time at one group.
template <bool BWD>
int combine(const Args& a, cudaStream_t s) {
  const int64_t units = a.s * a.groups;
  if ((a.chunks + a.s) * a.cg > 1024 * a.s) {
    if (units > 0x7fffffff) return GQ_ERR_UNSUPPORTED;
    return launch_after(combine_kernel<BWD, true>, dim3((unsigned)units), dim3(kCombine), 0, s, a);
  }
  return launch_after(combine_kernel<BWD, false>, dim3((unsigned)((units + kCombine / 32 - 1) / (kCombine / 32))),
                      dim3(kCombine), 0, s, a);
}

template <typename T, int V, int ACT, int GROUP>
int run_short(bool bwd, const Args& a, const Plan& z, cudaStream_t s) {
  auto bytes = [bwd](int d) { return (kThreads / GROUP) * ((bwd ? 2 : 1) * d + GROUP * V) * 8; };
  auto* kernel = bwd ? short_bwd_kernel<T, V, ACT, GROUP> : short_fwd_kernel<T, V, ACT, GROUP>;
  // the most that any call asks for: the limit is the kernel's, and another host
  // thread may set it between this call's setting and its launch
  GQ_TRY_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   bytes(GROUP == 32 ? kWarpMaxD : kShortMaxD)));
  return launch_after(kernel, dim3((unsigned)z.blocks), dim3(kThreads), bytes(a.d), s, a);
}

template <typename T, int V, int ACT>
int run_fwd(const Args& a, const Plan& z, cudaStream_t s) {
  if (z.brief) return z.group == 32 ? run_short<T, V, ACT, 32>(false, a, z, s) : run_short<T, V, ACT, kThreads>(false, a, z, s);
  const dim3 g((unsigned)z.chunks, z.slabs);
  GQ_TRY(launch_after(stats_kernel<T, V>, g, dim3(kThreads), kThreads * V * 8, s, a));
  GQ_TRY(combine<false>(a, s));
  return launch_after(apply_kernel<T, V, ACT>, g, dim3(kThreads), 0, s, a);
}

template <typename T, int V, int ACT>
int run_bwd(const Args& a, const Plan& z, cudaStream_t s) {
  if (z.brief) {
    GQ_TRY((z.group == 32 ? run_short<T, V, ACT, 32>(true, a, z, s) : run_short<T, V, ACT, kThreads>(true, a, z, s)));
  } else {
    const dim3 g((unsigned)z.chunks, z.slabs);
    GQ_TRY(launch_after(slopes_kernel<T, V, ACT>, g, dim3(kThreads), kThreads * V * 8, s, a));
    GQ_TRY(combine<true>(a, s));
    GQ_TRY(launch_after(apply_bwd_kernel<T, V, ACT>, g, dim3(kThreads), 0, s, a));
  }
  if (a.dgamma == nullptr && a.dbeta == nullptr) return GQ_OK;
  return launch_after(columns_kernel, dim3((a.d + kSumC - 1) / kSumC), dim3(kSumThreads), 0, s, a);
}

template <typename T, int V>
int run_act(bool bwd, int act, const Args& a, const Plan& z, cudaStream_t s) {
  switch (act) {
    case GQ_ACT_NONE: return bwd ? run_bwd<T, V, GQ_ACT_NONE>(a, z, s) : run_fwd<T, V, GQ_ACT_NONE>(a, z, s);
    case GQ_ACT_RELU: return bwd ? run_bwd<T, V, GQ_ACT_RELU>(a, z, s) : run_fwd<T, V, GQ_ACT_RELU>(a, z, s);
    default: return bwd ? run_bwd<T, V, GQ_ACT_SILU>(a, z, s) : run_fwd<T, V, GQ_ACT_SILU>(a, z, s);
  }
}

int run(bool bwd, int type, int act, int v, const Args& a, const Plan& z, cudaStream_t s) {
  switch (type) {
    case GQ_F32: return v == 1 ? run_act<float, 1>(bwd, act, a, z, s) : run_act<float, kVec>(bwd, act, a, z, s);
    case GQ_BF16:
      return v == 1 ? run_act<__nv_bfloat16, 1>(bwd, act, a, z, s) : run_act<__nv_bfloat16, kVec>(bwd, act, a, z, s);
    default: return v == 1 ? run_act<__half, 1>(bwd, act, a, z, s) : run_act<__half, kVec>(bwd, act, a, z, s);
  }
}

// rows that start aligned for four values
bool rows4(const void* p, int64_t ld, int type) { return aligned(p, 4 * type_bytes(type)) && ld % kVec == 0; }

// The largest power of two of lanes that each have a channel of a group.
int lanes_of(int cg) {
  int l = 1;
  while (l < 32 && 2 * l <= cg) l *= 2;
  return l;
}

int check(int type, int64_t n, int d, int groups, int64_t s, int64_t max_rows, int act, const int64_t* ptr) {
  if (!valid_type(type) || n < 0 || d < 1 || groups < 1 || d % groups || s < 0 || max_rows < 0 ||
      (act != GQ_ACT_NONE && act != GQ_ACT_RELU && act != GQ_ACT_SILU) || !aligned(ptr, 8) || (ptr == nullptr && s != 1))
    return GQ_ERR_INVALID_ARG;
  if (d > 16384 || n >= (int64_t)1 << 31 || s > (int64_t)1 << 30 || s * groups > 0x7fffffff) return GQ_ERR_UNSUPPORTED;
  return GQ_OK;
}

}  // namespace
}  // namespace gq

extern "C" size_t gq_group_norm_workspace_bytes(int64_t n, int d, int groups, int type, int64_t segments,
                                                int64_t max_rows, int backward) {
  using namespace gq;
  if (!valid_type(type) || n < 1 || d < 1 || d > 16384 || groups < 1 || d % groups || segments < 1 || max_rows < 0) return 0;
  return workspace(n, d, groups, type, segments, max_rows, backward != 0);
}

extern "C" int gq_group_norm_fwd(const void* X, int type, int64_t n, int d, int64_t ldx, int groups, const int64_t* ptr,
                                 int64_t segments, int64_t max_rows, const float* gamma, const float* beta, float eps,
                                 int act, void* Y, int64_t ldy, float* mean, float* rstd, void* ws, size_t ws_bytes,
                                 gq_stream stream) {
  using namespace gq;
  GQ_TRY(check(type, n, d, groups, segments, max_rows, act, ptr));
  if (ldx < d || ldy < d || !(eps >= 0.0f) || std::isinf(eps)) return GQ_ERR_INVALID_ARG;
  if (segments == 0) return GQ_OK;
  const int e = type_bytes(type);
  if (mean == nullptr || rstd == nullptr || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(gamma, 4) ||
      !aligned(beta, 4) || (n > 0 && (X == nullptr || Y == nullptr)) || !aligned(X, e) || !aligned(Y, e))
    return GQ_ERR_INVALID_ARG;
  const int64_t rows = n > 0 ? n : 1;  // without rows: the statistics of empty segments
  const int v = d % kVec == 0 && rows4(X, ldx, type) && rows4(Y, ldy, type) ? kVec : 1;
  const Plan z = make_plan(rows, d, segments, max_rows, e, v, false);
  const size_t need = workspace(rows, d, groups, type, segments, max_rows, false);
  if (need > 0 && (ws == nullptr || !aligned(ws, 256) || ws_bytes < need)) return GQ_ERR_WORKSPACE;
  Args a{};
  a.X = X;
  a.Y = Y;
  a.n = n;
  a.ldx = ldx;
  a.ldy = ldy;
  a.d = d;
  a.groups = groups;
  a.cg = d / groups;
  a.ptr = ptr;
  a.s = segments;
  a.gamma = gamma;
  a.beta = beta;
  a.eps = eps;
  a.mean = mean;
  a.rstd = rstd;
  a.vpr = z.vpr;
  a.tx = z.tx;
  a.ry = z.ry;
  a.lpg = lanes_of(a.cg);
  a.rows_per = z.rows_per;
  a.chunks = z.chunks;
  a.part = static_cast<float2*>(ws);
  return run(false, type, act, v, a, z, (cudaStream_t)stream);
}

extern "C" int gq_group_norm_bwd(const void* dY, int64_t lddy, const void* X, int64_t ldx, int type, int64_t n, int d,
                                 int groups, const int64_t* ptr, int64_t segments, int64_t max_rows, const float* mean,
                                 const float* rstd, const float* gamma, const float* beta, int act, void* dX,
                                 int64_t lddx, float* dgamma, float* dbeta, void* ws, size_t ws_bytes,
                                 gq_stream stream) {
  using namespace gq;
  GQ_TRY(check(type, n, d, groups, segments, max_rows, act, ptr));
  if (ldx < d || lddy < d || lddx < d || !aligned(dgamma, 4) || !aligned(dbeta, 4)) return GQ_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  if (segments == 0 || n == 0) {
    if (dgamma != nullptr) GQ_TRY_CUDA(cudaMemsetAsync(dgamma, 0, (size_t)d * 4, s));
    if (dbeta != nullptr) GQ_TRY_CUDA(cudaMemsetAsync(dbeta, 0, (size_t)d * 4, s));
    return GQ_OK;
  }
  const int e = type_bytes(type);
  if (mean == nullptr || rstd == nullptr || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(gamma, 4) ||
      !aligned(beta, 4) || X == nullptr || dY == nullptr || dX == nullptr || !aligned(X, e) || !aligned(dY, e) ||
      !aligned(dX, e))
    return GQ_ERR_INVALID_ARG;
  const int v = d % kVec == 0 && rows4(X, ldx, type) && rows4(dY, lddy, type) && rows4(dX, lddx, type) ? kVec : 1;
  const Plan z = make_plan(n, d, segments, max_rows, e, v, true);
  const size_t need = workspace(n, d, groups, type, segments, max_rows, true);
  if (ws == nullptr || !aligned(ws, 256) || ws_bytes < need) return GQ_ERR_WORKSPACE;
  Args a{};
  a.X = X;
  a.dY = dY;
  a.Y = dX;
  a.n = n;
  a.ldx = ldx;
  a.lddy = lddy;
  a.ldy = lddx;
  a.d = d;
  a.groups = groups;
  a.cg = d / groups;
  a.ptr = ptr;
  a.s = segments;
  a.gamma = gamma;
  a.beta = beta;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.vpr = z.vpr;
  a.tx = z.tx;
  a.ry = z.ry;
  a.lpg = lanes_of(a.cg);
  a.rows_per = z.rows_per;
  a.chunks = z.chunks;
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  a.parts = z.parts;
  if (z.brief) {
    a.tot = static_cast<float2*>(ws);
  } else {
    char* w = static_cast<char*>(ws);
    a.part = reinterpret_cast<float2*>(w);
    w += ((size_t)(z.chunks + segments) * d * 8 + 255) / 256 * 256;
    a.hsum = reinterpret_cast<float2*>(w);
    w += ((size_t)segments * groups * 8 + 255) / 256 * 256;
    a.tot = reinterpret_cast<float2*>(w);
  }
  return run(true, type, act, v, a, z, s);
}
