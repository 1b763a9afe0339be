// gq_adamw.cu -- one AdamW step over many tensors in one launch, with the two
// moments in fp32 or in 8-bit floats that share an exponent in blocks of 256.
//
//   m' = b1 m + (1 - b1) g,  v' = b2 v + (1 - b2) g^2
//   p' = p (1 - lr wd) - (lr / (1 - b1^t)) m' / (sqrt(v') / sqrt(1 - b2^t) + eps)
//
// It is bound by DRAM: every value of p, m, v is read and written once and g
// read once, 28 bytes an element with fp32 throughout, 16 with 8-bit moments.
//
// 8-bit moments.  A block holds an exponent byte e, that of its largest
// value's fp32 exponent field, and a code per value: the first moment as sign,
// 4 exponent bits, 3 of mantissa (E4M3), the second, which has no sign, as 4
// and 4.  The exponent is a power of two and no scale, so encoding is two exact
// products and an integer addition: scaled so that the codes' exponent field
// lines up with fp32's, a value's bits shifted right are its code, the codes
// without an exponent (subnormal) falling out of fp32's own subnormals.
// Rounding is stochastic, by the library's counter hash: a moving average
// with b2 = 0.999 changes by less than half a step of any 8-bit code, and
// rounded to the nearest it would stand still (a constant gradient's second
// moment stops at about 1/30 of its value); rounded at random it is right in
// the mean, its noise averaged over the 1 / (1 - b) steps that it remembers.  A second moment
// that is not 0 never becomes 0: it is the divisor of its first.
// Not right in the mean are a block's largest second moments: its codes end at 31/16 of
// a power of two, and what would be rounded up beyond it is not.  With b2 = 0.999
// the largest of 256 is half of its 32-bit value after 5,000 steps, and its parameter
// moves up to 1.4 times as far; those below a quarter of it are right to 1 in 10,000.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "gq_common.cuh"
#include "gq_internal.cuh"
#include "gq_sm100.cuh"
#include "gq_train.h"

namespace gq {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kBlockValues = 256;                   // values that share an exponent: a warp's, 8 a lane
constexpr int kMinExp = 16, kMaxExp = 254;          // so that every scale below is a normal fp32 number

// What a step multiplies by; made on the host, or by begin_kernel from the
// step number in device memory.
struct Coef {
  float b1, o1, b2, o2;   // beta and 1 - beta
  float keep;             // 1 - lr wd
  float lr1;              // lr / (1 - b1^t)
  float rs2;              // 1 / sqrt(1 - b2^t)
  float eps;
  float one;              // 1, which the compiler does not know
  uint32_t key;           // of the rounding noise
};

struct Tensor {
  void* p;
  const void* g;
  void* m;
  void* v;
  uint8_t* me;
  uint8_t* ve;
  int64_t n;
  int64_t tile0;          // tiles of the tensors before it in this launch
  int64_t cols, ldp, ldg; // rows of `cols` values; cols = n: dense
  uint32_t block0;        // the first block's number in the noise
  uint32_t vec;           // dense and 16-byte aligned
};

template <int CAP>
struct Batch {
  Tensor t[CAP];
  int count;
};

struct DevRecord {        // gq_adamw_dev_bytes() of them
  int64_t step;
  double lr;
  Coef coef;
};

Coef make_coef(const gq_adamw_args& a, int64_t step) {
  Coef c;
  c.b1 = (float)a.beta1;
  c.o1 = (float)(1.0 - a.beta1);
  c.b2 = (float)a.beta2;
  c.o2 = (float)(1.0 - a.beta2);
  c.keep = (float)(1.0 - a.lr * a.weight_decay);
  c.lr1 = (float)(a.lr / (1.0 - std::pow(a.beta1, (double)step)));
  c.rs2 = (float)(1.0 / std::sqrt(1.0 - std::pow(a.beta2, (double)step)));
  c.eps = (float)a.eps;
  c.one = 1.0f;
  c.key = seed_key_host(a.seed + (uint64_t)step * 0x9E3779B97F4A7C15ULL);
  return c;
}

__global__ void begin_kernel(DevRecord* rec, const gq_adamw_args a, const float* gscale) {
  grid_wait();
  if (gscale != nullptr && !isfinite(*gscale)) return;  // the step is skipped: it does not count
  const int64_t step = ++rec->step;
  const double lr = rec->lr;
  Coef c;
  c.b1 = (float)a.beta1;
  c.o1 = (float)(1.0 - a.beta1);
  c.b2 = (float)a.beta2;
  c.o2 = (float)(1.0 - a.beta2);
  c.keep = (float)(1.0 - lr * a.weight_decay);
  c.lr1 = (float)(lr / (1.0 - pow(a.beta1, (double)step)));
  c.rs2 = (float)(1.0 / sqrt(1.0 - pow(a.beta2, (double)step)));
  c.eps = (float)a.eps;
  c.one = 1.0f;
  c.key = fmix32(seed_fold(a.seed + (uint64_t)step * 0x9E3779B97F4A7C15ULL));
  rec->coef = c;
}

// ------------------------------------------------------------------- types --
template <typename T>
__device__ __forceinline__ float to_f(T x) {
  return (float)x;
}
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }

// A lane's eight values of a block: 4 l .. 4 l + 3 and 128 further, so that a
// warp's loads and stores are contiguous whatever the type.
__device__ __forceinline__ int place(int lane, int j) { return 4 * lane + (j & 3) + (j & 4) * 32; }
template <typename T>
struct Raw {
  uint4 w[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw<T> load8(const void* base, int64_t block, int lane) {
  Raw<T> r;
  const T* a = static_cast<const T*>(base) + block * 256 + 4 * lane;
  if constexpr (sizeof(T) == 4) {
    r.w[0] = *reinterpret_cast<const uint4*>(a);
    r.w[1] = *reinterpret_cast<const uint4*>(a + 128);
  } else {
    const uint2 x = *reinterpret_cast<const uint2*>(a), y = *reinterpret_cast<const uint2*>(a + 128);
    r.w[0] = make_uint4(x.x, x.y, y.x, y.y);
  }
  return r;
}
template <typename T>
__device__ __forceinline__ void unpack8(const Raw<T>& r, float (&x)[8]) {
  const T* e = reinterpret_cast<const T*>(&r);
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = to_f(e[j]);
}
template <typename T>
__device__ __forceinline__ void store8(void* base, int64_t block, int lane, const float (&x)[8]) {
  Raw<T> r;
  T* e = reinterpret_cast<T*>(&r);
#pragma unroll
  for (int j = 0; j < 8; ++j) e[j] = from_f<T>(x[j]);
  T* a = static_cast<T*>(base) + block * 256 + 4 * lane;
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<uint4*>(a) = r.w[0];
    *reinterpret_cast<uint4*>(a + 128) = r.w[1];
  } else {
    *reinterpret_cast<uint2*>(a) = make_uint2(r.w[0].x, r.w[0].y);
    *reinterpret_cast<uint2*>(a + 128) = make_uint2(r.w[0].z, r.w[0].w);
  }
}
__device__ __forceinline__ uint2 load8c(const void* base, int64_t block, int lane) {
  const uint32_t* a = reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(base) + block * 256) + lane;
  return make_uint2(a[0], a[32]);
}
__device__ __forceinline__ void store8c(void* base, int64_t block, int lane, uint2 w) {
  uint32_t* a = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(base) + block * 256) + lane;
  a[0] = w.x;
  a[32] = w.y;
}

// ------------------------------------------------------------ 8-bit floats --
__device__ __forceinline__ float pow2f(int field) { return __uint_as_float((uint32_t)field << 23); }

// SECOND = false: sign, 4, 3;  true: 4, 4 without a sign.  The block's largest
// value, of exponent field e, comes to [2^7, 2^8) or [2^8, 2^9): all but the
// last octave of the codes' range below it, room for one rounding up.
template <bool SECOND>
struct Code {
  static constexpr int kept = SECOND ? 4 : 3;
  static constexpr int shift = 23 - kept;
  static constexpr int top = SECOND ? 8 : 7;
  static constexpr float far = 1.329227995784916e36f;   // 2^120: fp32's exponent bias less the codes'
  static constexpr float near = 7.52316384526264e-37f;  // 2^-120
  // scale of decode, its reciprocal for encode
  static __device__ __forceinline__ float down(int e) { return pow2f(e - top); }
  static __device__ __forceinline__ float up(int e) { return pow2f(254 - (e - top)); }
  // a code, byte K of w, as the bits of its value times 2^-120
  template <int K>
  static __device__ __forceinline__ uint32_t bits(uint32_t w) {
    if (SECOND) return K < 3 ? ((w >> (8 * K)) & 255u) << shift : w >> 24 << shift;
    const int at_top = (int)__byte_perm(w, 0, 0x0444 | K << 12);  // bit 31 is the sign
    return (uint32_t)(at_top >> 4) & 0x87F00000u;
  }
};
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// codes w (4 values) -> values
template <bool SECOND>
__device__ __forceinline__ void decode4(uint32_t w, float scale, float2& lo, float2& hi) {
  using F = Code<SECOND>;
  const float2 far = both(F::far), s = both(scale);
  lo = make_float2(__uint_as_float(F::template bits<0>(w)), __uint_as_float(F::template bits<1>(w)));
  hi = make_float2(__uint_as_float(F::template bits<2>(w)), __uint_as_float(F::template bits<3>(w)));
  lo = mul2(mul2(lo, far), s);
  hi = mul2(mul2(hi, far), s);
}
// values -> codes, byte k from noise word h[k].  Codes end at 120, the 2^8 that a
// block's largest value may be rounded up to, and 255, the 2^9 less a step; what is
// not finite gets these.  A second moment that is not 0 gets at least 1.
template <bool SECOND>
__device__ __forceinline__ uint32_t encode4(float2 lo, float2 hi, float scale, const uint32_t (&h)[4]) {
  using F = Code<SECOND>;
  const float2 near = both(F::near), s = both(scale);
  const float2 a = mul2(mul2(lo, s), near), b = mul2(mul2(hi, s), near);
  const uint32_t x[4] = {__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y)};
  const uint32_t v[4] = {__float_as_uint(lo.x), __float_as_uint(lo.y), __float_as_uint(hi.x), __float_as_uint(hi.y)};
  uint32_t c[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (SECOND)
      c[k] = min(max((x[k] + (h[k] & 0x7FFFFu)) >> F::shift, min(v[k], 1u)), 255u);
    else
      c[k] = min(((x[k] & 0x7FFFFFFFu) + (h[k] >> 12)) >> F::shift, 120u);
  }
  const uint32_t w = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
  if (SECOND) return w;
  const uint32_t sign = __byte_perm(__byte_perm(v[0], v[1], 0x0073), __byte_perm(v[2], v[3], 0x0073), 0x5410);
  return w | (sign & 0x80808080u);
}

// A magnitude's rank: twice its bits, which drops the sign, and one exponent more,
// which takes infinities and NaN past the end, below all finite values.  The
// block's exponent is that of its largest finite value, so that one that is not
// finite takes the greatest code and the other 255 keep theirs.
__device__ __forceinline__ uint32_t rank_of(float x) { return __float_as_uint(x) * 2u + (1u << 24); }
__device__ __forceinline__ int block_exp(uint32_t largest_rank) {
  return min(max((int)(__reduce_max_sync(FULL, largest_rank) >> 24) - 1, kMinExp), kMaxExp);
}
__device__ __forceinline__ float sqrt_fast(float x) {
  float y;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// a + b rounded by itself, as a one + b: a packed sum of packed products is
// fused with them, also where the 1 is a constant
__device__ __forceinline__ float2 sum2(float2 a, float2 b, float one) { return fma2(a, both(one), b); }

// Two values.  The moments' update is products and a sum, each rounded: the codes
// can be reproduced from elementary operations.  The root and the reciprocal are
// the special function unit's (a step off each): their quotient is lr times smaller than p.
__device__ __forceinline__ void update(float2& p, float2 g, float2& m, float2& v, const Coef& c) {
  m = sum2(mul2(m, both(c.b1)), mul2(g, both(c.o1)), c.one);
  v = sum2(mul2(v, both(c.b2)), mul2(mul2(g, g), both(c.o2)), c.one);
  const float2 den = fma2(make_float2(sqrt_fast(v.x), sqrt_fast(v.y)), both(c.rs2), both(c.eps));
  const float2 step = mul2(mul2(m, both(-c.lr1)), make_float2(rcp_fast(den.x), rcp_fast(den.y)));
  p = fma2(p, both(c.keep), step);
}

// What a lane holds of a block, as loaded.
template <typename TP, typename TG, bool SMALL>
struct Held {
  Raw<TP> p;
  Raw<TG> g;
  Raw<float> m, v;       // 32-bit moments
  uint2 mc, vc;          // 8-bit ones
  int em, ev;
};

// The arithmetic of a lane's eight values; mc, vc, em, ev are replaced by the new ones.
template <bool SMALL>
__device__ __forceinline__ void step8(float (&p)[8], float (&g)[8], float (&m)[8], float (&v)[8], uint2& mc, uint2& vc,
                                      int& em, int& ev, uint32_t block, int lane, const Coef& c, float gs) {
  float2* p2 = reinterpret_cast<float2*>(p);
  float2* g2 = reinterpret_cast<float2*>(g);
  float2* m2 = reinterpret_cast<float2*>(m);
  float2* v2 = reinterpret_cast<float2*>(v);
  if (SMALL) {
    const float dm = Code<false>::down(min(max(em, kMinExp), kMaxExp));
    const float dv = Code<true>::down(min(max(ev, kMinExp), kMaxExp));
    decode4<false>(mc.x, dm, m2[0], m2[1]);
    decode4<false>(mc.y, dm, m2[2], m2[3]);
    decode4<true>(vc.x, dv, v2[0], v2[1]);
    decode4<true>(vc.y, dv, v2[2], v2[3]);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) update(p2[j], mul2(g2[j], both(gs)), m2[j], v2[j], c);
  if (SMALL) {
    uint32_t bm = 0, bv = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      bm = max(bm, rank_of(m[j]));
      bv = max(bv, rank_of(v[j]));
    }
    em = block_exp(bm);
    ev = block_exp(bv);
    const float um = Code<false>::up(em), uv = Code<true>::up(ev);
    const uint32_t kr = row_key(c.key, block) + (uint32_t)lane * (4u * 0x9E3779B9u);
    uint32_t h[2][4];
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j >> 2][j & 3] = fmix32(kr + (uint32_t)place(0, j) * 0x9E3779B9u);
    mc = make_uint2(encode4<false>(m2[0], m2[1], um, h[0]), encode4<false>(m2[2], m2[3], um, h[1]));
    vc = make_uint2(encode4<true>(v2[0], v2[1], uv, h[0]), encode4<true>(v2[2], v2[3], uv, h[1]));
  }
}

template <typename TP, typename TG, bool SMALL>
__device__ __forceinline__ void take(const Tensor& t, int64_t b, int lane, Held<TP, TG, SMALL>& w) {
  w.p = load8<TP>(t.p, b, lane);
  w.g = load8<TG>(t.g, b, lane);
  if constexpr (SMALL) {
    w.mc = load8c(t.m, b, lane);
    w.vc = load8c(t.v, b, lane);
    w.em = t.me[b];
    w.ev = t.ve[b];
  } else {
    w.m = load8<float>(t.m, b, lane);
    w.v = load8<float>(t.v, b, lane);
  }
}

template <typename TP, typename TG, bool SMALL>
__device__ __forceinline__ void work(const Tensor& t, int64_t b, int lane, Held<TP, TG, SMALL>& w, const Coef& c, float gs) {
  alignas(16) float p[8], g[8], m[8], v[8];
  unpack8<TP>(w.p, p);
  unpack8<TG>(w.g, g);
  if constexpr (!SMALL) {
    unpack8<float>(w.m, m);
    unpack8<float>(w.v, v);
  }
  step8<SMALL>(p, g, m, v, w.mc, w.vc, w.em, w.ev, t.block0 + (uint32_t)b, lane, c, gs);
  store8<TP>(t.p, b, lane, p);
  if constexpr (SMALL) {
    store8c(t.m, b, lane, w.mc);
    store8c(t.v, b, lane, w.vc);
    if (lane == 0) {
      t.me[b] = (uint8_t)w.em;
      t.ve[b] = (uint8_t)w.ev;
    }
  } else {
    store8<float>(t.m, b, lane, m);
    store8<float>(t.v, b, lane, v);
  }
}

// A block that is not whole, not aligned or not dense, value by value.
template <typename TP, typename TG, bool SMALL>
__device__ __forceinline__ void ragged(const Tensor& t, int64_t b, int lane, const Coef& c, float gs) {
  const int64_t i0 = b * kBlockValues;
  alignas(16) float p[8], g[8], m[8], v[8];
  uint32_t w[4] = {0, 0, 0, 0};
  const bool dense = t.cols == t.n;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    p[j] = g[j] = m[j] = v[j] = 0.0f;
    const int64_t i = i0 + place(lane, j);
    if (i < t.n) {
      const int64_t r = dense ? 0 : i / t.cols, col = i - r * t.cols;
      p[j] = to_f(static_cast<const TP*>(t.p)[r * t.ldp + col]);
      g[j] = to_f(static_cast<const TG*>(t.g)[r * t.ldg + col]);
      if (SMALL) {
        w[j >> 2] |= (uint32_t) static_cast<const uint8_t*>(t.m)[i] << (8 * (j & 3));
        w[2 + (j >> 2)] |= (uint32_t) static_cast<const uint8_t*>(t.v)[i] << (8 * (j & 3));
      } else {
        m[j] = static_cast<const float*>(t.m)[i];
        v[j] = static_cast<const float*>(t.v)[i];
      }
    }
  }
  uint2 mc = make_uint2(w[0], w[1]), vc = make_uint2(w[2], w[3]);
  int em = SMALL ? t.me[b] : 0, ev = SMALL ? t.ve[b] : 0;
  step8<SMALL>(p, g, m, v, mc, vc, em, ev, t.block0 + (uint32_t)b, lane, c, gs);
  if (SMALL && lane == 0) {
    t.me[b] = (uint8_t)em;
    t.ve[b] = (uint8_t)ev;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int64_t i = i0 + place(lane, j);
    if (i < t.n) {
      const int64_t r = dense ? 0 : i / t.cols, col = i - r * t.cols;
      static_cast<TP*>(t.p)[r * t.ldp + col] = from_f<TP>(p[j]);
      if (SMALL) {
        static_cast<uint8_t*>(t.m)[i] = (uint8_t)((j < 4 ? mc.x : mc.y) >> (8 * (j & 3)));
        static_cast<uint8_t*>(t.v)[i] = (uint8_t)((j < 4 ? vc.x : vc.y) >> (8 * (j & 3)));
      } else {
        static_cast<float*>(t.m)[i] = m[j];
        static_cast<float*>(t.v)[i] = v[j];
      }
    }
  }
}

// A block a warp, and as many warps as 48 registers a thread allow: what hides the
// reads is other warps.  With 8-bit moments 152 M fp32 values take 424 us, 5.7 TB/s,
// and 67 M bf16 ones 165 (their arithmetic, 74 instructions a value, is three
// quarters of the issue slots) with 40 warps an SM; 411 and 175 with 32; 655 and 300 with 24
// that each read their next block while they work on one.  With fp32 moments
// 67 M values take 247 us, 7.0 TB/s.
template <typename TP, typename TG, bool SMALL, int CAP>
__global__ void __launch_bounds__(kThreads, 10)
    adamw_kernel(const __grid_constant__ Batch<CAP> batch, const Coef host, const DevRecord* rec, const float* gscale) {
  grid_wait();
  float gs = 1.0f;
  if (gscale != nullptr) {
    gs = *gscale;
    if (!isfinite(gs)) return;
  }
  const Coef c = rec != nullptr ? rec->coef : host;
  const int64_t tile = blockIdx.x;
  int lo = 0, hi = batch.count - 1;  // the last tensor whose first tile is not behind this one
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (batch.t[mid].tile0 <= tile)
      lo = mid;
    else
      hi = mid - 1;
  }
  const Tensor& t = batch.t[lo];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t b = (tile - t.tile0) * kWarps + warp;
  if (t.vec && (b + 1) * kBlockValues <= t.n) {
    Held<TP, TG, SMALL> w;
    take(t, b, lane, w);
    work(t, b, lane, w, c, gs);
  } else if (b * kBlockValues < t.n) {
    ragged<TP, TG, SMALL>(t, b, lane, c, gs);
  }
}

// ------------------------------------------------------------------ values --
template <typename T, bool SECOND>
__global__ void __launch_bounds__(kThreads)
    moment_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ exps, int64_t n, T* __restrict__ out,
                  int vec) {
  const int lane = threadIdx.x & 31;
  const int64_t blocks = (n + kBlockValues - 1) / kBlockValues;
  for (int64_t b = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); b < blocks; b += (int64_t)gridDim.x * kWarps) {
    const float s = Code<SECOND>::down(min(max((int)exps[b], kMinExp), kMaxExp));
    alignas(16) float x[8];
    float2* x2 = reinterpret_cast<float2*>(x);
    if (vec && (b + 1) * kBlockValues <= n) {
      const uint2 c = load8c(codes, b, lane);
      decode4<SECOND>(c.x, s, x2[0], x2[1]);
      decode4<SECOND>(c.y, s, x2[2], x2[3]);
      store8<T>(out, b, lane, x);
    } else {
      for (int j = lane; j < kBlockValues && b * kBlockValues + j < n; j += 32) {
        decode4<SECOND>(codes[b * kBlockValues + j], s, x2[0], x2[1]);
        out[b * kBlockValues + j] = from_f<T>(x[0]);
      }
    }
  }
}

int type_bytes(int type) { return type == GQ_F32 ? 4 : 2; }
bool valid_type(int type) { return type == GQ_F32 || type == GQ_BF16 || type == GQ_F16; }

template <typename TP, typename TG, bool SMALL, int CAP>
int launch(const Batch<CAP>& b, int64_t tiles, const Coef& c, const DevRecord* rec, const float* gs, cudaStream_t s) {
  return launch_after(adamw_kernel<TP, TG, SMALL, CAP>, dim3((unsigned)tiles), dim3(kThreads), 0, s, b, c, rec, gs);
}

template <typename TP, typename TG, int CAP>
int launch_bits(int bits, const Batch<CAP>& b, int64_t tiles, const Coef& c, const DevRecord* rec, const float* gs,
                cudaStream_t s) {
  return bits == 8 ? launch<TP, TG, true, CAP>(b, tiles, c, rec, gs, s)
                   : launch<TP, TG, false, CAP>(b, tiles, c, rec, gs, s);
}

template <typename TP, int CAP>
int launch_g(int gt, int bits, const Batch<CAP>& b, int64_t tiles, const Coef& c, const DevRecord* rec, const float* gs,
             cudaStream_t s) {
  switch (gt) {
    case GQ_F32: return launch_bits<TP, float, CAP>(bits, b, tiles, c, rec, gs, s);
    case GQ_BF16: return launch_bits<TP, __nv_bfloat16, CAP>(bits, b, tiles, c, rec, gs, s);
    default: return launch_bits<TP, __half, CAP>(bits, b, tiles, c, rec, gs, s);
  }
}

template <int CAP>
int launch_p(int pt, int gt, int bits, const Batch<CAP>& b, int64_t tiles, const Coef& c, const DevRecord* rec,
             const float* gs, cudaStream_t s) {
  switch (pt) {
    case GQ_F32: return launch_g<float, CAP>(gt, bits, b, tiles, c, rec, gs, s);
    case GQ_BF16: return launch_g<__nv_bfloat16, CAP>(gt, bits, b, tiles, c, rec, gs, s);
    default: return launch_g<__half, CAP>(gt, bits, b, tiles, c, rec, gs, s);
  }
}

// The tensors travel as kernel parameters (no table in device memory that a
// captured graph and an eager call would share): 16 of them for the usual
// small model, so that its launch carries 2 KB, up to 256 otherwise (25 KB of
// the 32,764 bytes that a kernel may take).
template <int CAP>
int run(const gq_adamw_tensor* ts, int count, int pt, int gt, int bits, const Coef& c, const DevRecord* rec,
        const float* gs, cudaStream_t s) {
  Batch<CAP> b;
  int64_t tiles = 0;
  b.count = 0;
  for (int i = 0; i < count; ++i) {
    const gq_adamw_tensor& t = ts[i];
    if (t.n > 0) {
      const int64_t per = (int64_t)kWarps * kBlockValues, add = (t.n + per - 1) / per;
      if (tiles + add > 0x7fffffff && b.count > 0) {
        GQ_TRY(launch_p<CAP>(pt, gt, bits, b, tiles, c, rec, gs, s));
        b.count = 0;
        tiles = 0;
      }
      Tensor& o = b.t[b.count++];
      o.p = t.p;
      o.g = t.g;
      o.m = t.m;
      o.v = t.v;
      o.me = t.m_exp;
      o.ve = t.v_exp;
      o.n = t.n;
      o.tile0 = tiles;
      const bool dense = t.cols == 0 || (t.ldp == t.cols && t.ldg == t.cols);
      o.cols = dense ? t.n : t.cols;
      o.ldp = dense ? t.n : t.ldp;
      o.ldg = dense ? t.n : t.ldg;
      o.block0 = (uint32_t)t.block0;
      o.vec = dense && aligned(t.p, 16) && aligned(t.g, 16) && aligned(t.m, bits == 8 ? 8 : 16) &&
              aligned(t.v, bits == 8 ? 8 : 16);
      tiles += add;
    }
    if (b.count == CAP || (i == count - 1 && b.count > 0)) {
      GQ_TRY(launch_p<CAP>(pt, gt, bits, b, tiles, c, rec, gs, s));
      b.count = 0;
      tiles = 0;
    }
  }
  return GQ_OK;
}

int check(const gq_adamw_tensor* ts, int count, int pt, int gt, int bits, const gq_adamw_args* a) {
  if (count < 0 || (count > 0 && ts == nullptr) || a == nullptr || !valid_type(pt) || !valid_type(gt))
    return GQ_ERR_INVALID_ARG;
  if (bits != 8 && bits != 32) return GQ_ERR_INVALID_ARG;
  if (!(a->beta1 >= 0.0 && a->beta1 < 1.0) || !(a->beta2 >= 0.0 && a->beta2 < 1.0) || !(a->eps >= 0.0) ||
      !std::isfinite(a->eps) || !std::isfinite(a->lr) || !std::isfinite(a->weight_decay))
    return GQ_ERR_INVALID_ARG;
  if (a->dev == nullptr && a->step < 1) return GQ_ERR_INVALID_ARG;
  if (!aligned(a->dev, 8) || !aligned(a->grad_scale, 4)) return GQ_ERR_INVALID_ARG;
  for (int i = 0; i < count; ++i) {
    const gq_adamw_tensor& t = ts[i];
    if (t.n < 0 || t.cols < 0) return GQ_ERR_INVALID_ARG;
    if (t.n == 0) continue;
    if (t.n > (int64_t)1 << 40) return GQ_ERR_UNSUPPORTED;
    if (t.p == nullptr || t.g == nullptr || t.m == nullptr || t.v == nullptr) return GQ_ERR_INVALID_ARG;
    if (!aligned(t.p, type_bytes(pt)) || !aligned(t.g, type_bytes(gt))) return GQ_ERR_INVALID_ARG;
    if (bits == 32 && (!aligned(t.m, 4) || !aligned(t.v, 4))) return GQ_ERR_INVALID_ARG;
    if (bits == 8 && (t.m_exp == nullptr || t.v_exp == nullptr)) return GQ_ERR_INVALID_ARG;
    if (t.cols > 0 && (t.n % t.cols || t.ldp < t.cols || t.ldg < t.cols)) return GQ_ERR_INVALID_ARG;
    if (t.block0 < 0 || t.block0 > 0xffffffffLL) return GQ_ERR_INVALID_ARG;
  }
  return GQ_OK;
}

template <typename T>
int moment(const uint8_t* codes, const uint8_t* exps, int64_t n, int second, T* out, cudaStream_t s) {
  const int64_t tiles = (n + kWarps * kBlockValues - 1) / (kWarps * kBlockValues), most = 16 * (int64_t)sm_count();
  const int64_t blocks = tiles < most ? tiles : most;
  const int vec = aligned(codes, 8) && aligned(out, 16);
  if (second)
    moment_kernel<T, true><<<(unsigned)blocks, kThreads, 0, s>>>(codes, exps, n, out, vec);
  else
    moment_kernel<T, false><<<(unsigned)blocks, kThreads, 0, s>>>(codes, exps, n, out, vec);
  return launch_status();
}

}  // namespace
}  // namespace gq

extern "C" size_t gq_adamw_dev_bytes(void) { return sizeof(gq::DevRecord); }

extern "C" int gq_adamw_step(const gq_adamw_tensor* tensors, int count, int p_type, int g_type, int state_bits,
                             const gq_adamw_args* args, gq_stream stream) {
  using namespace gq;
  GQ_TRY(check(tensors, count, p_type, g_type, state_bits, args));
  cudaStream_t s = (cudaStream_t)stream;
  const Coef c = args->dev == nullptr ? make_coef(*args, args->step) : Coef{};
  DevRecord* rec = static_cast<DevRecord*>(args->dev);
  if (rec != nullptr && args->advance) GQ_TRY(launch_after(begin_kernel, dim3(1), dim3(1), 0, s, rec, *args, args->grad_scale));
  return count <= 16 ? run<16>(tensors, count, p_type, g_type, state_bits, c, rec, args->grad_scale, s)
                     : run<256>(tensors, count, p_type, g_type, state_bits, c, rec, args->grad_scale, s);
}

extern "C" int gq_adam_moment(const uint8_t* codes, const uint8_t* exps, int64_t n, int second, void* out, int type,
                              gq_stream stream) {
  using namespace gq;
  if (n < 0 || !valid_type(type)) return GQ_ERR_INVALID_ARG;
  if (n == 0) return GQ_OK;
  if (codes == nullptr || exps == nullptr || out == nullptr || !aligned(out, type_bytes(type)))
    return GQ_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  switch (type) {
    case GQ_F32: return moment(codes, exps, n, second, static_cast<float*>(out), s);
    case GQ_BF16: return moment(codes, exps, n, second, static_cast<__nv_bfloat16*>(out), s);
    default: return moment(codes, exps, n, second, static_cast<__half*>(out), s);
  }
}
