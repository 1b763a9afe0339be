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
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "gq_common.cuh"
#include "gq_internal.cuh"
#include "gq_sm100.cuh"
#include "gq_train.h"

namespace gq {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBlockValues = 256;                   // values that share an exponent: a warp's, 8 a lane
constexpr int kTileBlocks = 16;                     // blocks of a thread block's tile
constexpr int kMinExp = 16, kMaxExp = 254;          // so that every scale below is a normal fp32 number

// What a step multiplies by; made on the host, or by begin_kernel from the
// step number in device memory.
struct Coef {
  float b1, o1, b2, o2;   // beta and 1 - beta
  float keep;             // 1 - lr wd
  float lr1;              // lr / (1 - b1^t)
  float rs2;              // 1 / sqrt(1 - b2^t)
  float eps;
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

// 8 consecutive values, 16-byte aligned
template <typename T>
struct Raw {
  uint4 w[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw<T> load8(const void* base, int64_t i) {
  Raw<T> r;
  const uint4* a = reinterpret_cast<const uint4*>(static_cast<const T*>(base) + i);
#pragma unroll
  for (int k = 0; k < (int)(sizeof(T) / 2); ++k) r.w[k] = a[k];
  return r;
}
template <typename T>
__device__ __forceinline__ void unpack8(const Raw<T>& r, float (&x)[8]) {
  const T* e = reinterpret_cast<const T*>(&r);
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = to_f(e[j]);
}
template <typename T>
__device__ __forceinline__ void store8(void* base, int64_t i, const float (&x)[8]) {
  Raw<T> r;
  T* e = reinterpret_cast<T*>(&r);
#pragma unroll
  for (int j = 0; j < 8; ++j) e[j] = from_f<T>(x[j]);
  uint4* a = reinterpret_cast<uint4*>(static_cast<T*>(base) + i);
#pragma unroll
  for (int k = 0; k < (int)(sizeof(T) / 2); ++k) a[k] = r.w[k];
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

  static __device__ __forceinline__ float decode(uint32_t c, float scale) {
    const uint32_t bits = SECOND ? c << shift : ((c & 127u) << shift | (c & 128u) << 24);
    return __fmul_rn(__fmul_rn(__uint_as_float(bits), far), scale);
  }
  // scale of decode, its reciprocal for encode
  static __device__ __forceinline__ float down(int e) { return pow2f(e - top); }
  static __device__ __forceinline__ float up(int e) { return pow2f(254 - (e - top)); }

  static __device__ __forceinline__ uint32_t encode(float x, float scale, uint32_t noise) {
    const uint32_t add = SECOND ? noise & 0x7FFFFu : noise >> 12;
    const float y = __fmul_rn(__fmul_rn(fabsf(x), scale), near);
    uint32_t c = (__float_as_uint(y) + add) >> shift;
    if (SECOND) return x > 0.0f ? min(max(c, 1u), 255u) : x == 0.0f ? 0u : 255u;
    return min(c, 126u) | (__float_as_uint(x) >> 24 & 128u);
  }
};

__device__ __forceinline__ int block_exp(uint32_t largest_bits) {
  return min(max((int)(__reduce_max_sync(FULL, largest_bits) >> 23), kMinExp), kMaxExp);
}

// The moments' update is products and a sum, each rounded: the codes can be
// reproduced from elementary operations.  The quotient is MUFU's (2 steps off at
// most): it is lr times smaller than p.
__device__ __forceinline__ void update(float& p, float g, float& m, float& v, const Coef& c) {
  m = __fadd_rn(__fmul_rn(m, c.b1), __fmul_rn(g, c.o1));
  v = __fadd_rn(__fmul_rn(v, c.b2), __fmul_rn(__fmul_rn(g, g), c.o2));
  p = fmaf(p, c.keep, -__fdividef(c.lr1 * m, fmaf(sqrtf(v), c.rs2, c.eps)));
}

// One warp, one block of 256 values: lane l holds values 8 l .. 8 l + 7.
template <typename TP, typename TG, bool SMALL>
__device__ __forceinline__ void block_step(const Tensor& t, int64_t b, int lane, const Coef& c, float gs) {
  const int64_t i0 = b * kBlockValues + lane * 8;
  float p[8], g[8], m[8], v[8];
  const bool whole = t.vec && (b + 1) * kBlockValues <= t.n;
  const int live = i0 >= t.n ? 0 : (int)min((int64_t)8, t.n - i0);
  uint2 mc = make_uint2(0, 0), vc = make_uint2(0, 0);
  int em = 0, ev = 0;
  if (whole) {
    const Raw<TP> rp = load8<TP>(t.p, i0);
    const Raw<TG> rg = load8<TG>(t.g, i0);
    if (SMALL) {
      mc = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(t.m) + i0);
      vc = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(t.v) + i0);
    } else {
      unpack8<float>(load8<float>(t.m, i0), m);
      unpack8<float>(load8<float>(t.v, i0), v);
    }
    unpack8<TP>(rp, p);
    unpack8<TG>(rg, g);
  } else {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      p[j] = g[j] = m[j] = v[j] = 0.0f;
      if (j < live) {
        const int64_t i = i0 + j;
        const int64_t r = t.cols == t.n ? 0 : i / t.cols, col = i - r * t.cols;
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
    mc = make_uint2(w[0], w[1]);
    vc = make_uint2(w[2], w[3]);
  }
  if (SMALL) {
    em = min(max((int)t.me[b], kMinExp), kMaxExp);
    ev = min(max((int)t.ve[b], kMinExp), kMaxExp);
    const float dm = Code<false>::down(em), dv = Code<true>::down(ev);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m[j] = Code<false>::decode(((j < 4 ? mc.x : mc.y) >> (8 * (j & 3))) & 255u, dm);
      v[j] = Code<true>::decode(((j < 4 ? vc.x : vc.y) >> (8 * (j & 3))) & 255u, dv);
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) update(p[j], g[j] * gs, m[j], v[j], c);
  if (SMALL) {
    uint32_t bm = 0, bv = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      bm = max(bm, __float_as_uint(m[j]) & 0x7FFFFFFFu);
      bv = max(bv, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    }
    em = block_exp(bm);
    ev = block_exp(bv);
    const float um = Code<false>::up(em), uv = Code<true>::up(ev);
    const uint32_t kr = row_key(c.key, t.block0 + (uint32_t)b);
    mc = vc = make_uint2(0, 0);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t h = fmix32(kr + (uint32_t)(lane * 8 + j) * 0x9E3779B9u);
      const uint32_t a = Code<false>::encode(m[j], um, h) << (8 * (j & 3));
      const uint32_t d = Code<true>::encode(v[j], uv, h) << (8 * (j & 3));
      if (j < 4) {
        mc.x |= a;
        vc.x |= d;
      } else {
        mc.y |= a;
        vc.y |= d;
      }
    }
    if (lane == 0) {
      t.me[b] = (uint8_t)em;
      t.ve[b] = (uint8_t)ev;
    }
  }
  if (whole) {
    store8<TP>(t.p, i0, p);
    if (SMALL) {
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.m) + i0) = mc;
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.v) + i0) = vc;
    } else {
      store8<float>(t.m, i0, m);
      store8<float>(t.v, i0, v);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j < live) {
        const int64_t i = i0 + j;
        const int64_t r = t.cols == t.n ? 0 : i / t.cols, col = i - r * t.cols;
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
}

template <typename TP, typename TG, bool SMALL, int CAP>
__global__ void __launch_bounds__(kThreads)
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
  const int64_t first = (tile - t.tile0) * kTileBlocks;
  const int64_t blocks = (t.n + kBlockValues - 1) / kBlockValues;
#pragma unroll 2
  for (int k = 0; k < kTileBlocks; k += kWarps) {
    const int64_t b = first + k + warp;
    if (b < blocks) block_step<TP, TG, SMALL>(t, b, lane, c, gs);
  }
}

// ------------------------------------------------------------------ values --
template <typename T, bool SECOND>
__global__ void __launch_bounds__(kThreads)
    moment_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ exps, int64_t n, T* __restrict__ out,
                  int vec) {
  const int64_t i0 = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 8;
  if (i0 >= n) return;
  const float s = Code<SECOND>::down(min(max((int)exps[i0 / kBlockValues], kMinExp), kMaxExp));
  if (vec && i0 + 8 <= n) {
    const uint2 c = *reinterpret_cast<const uint2*>(codes + i0);
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = Code<SECOND>::decode(((j < 4 ? c.x : c.y) >> (8 * (j & 3))) & 255u, s);
    store8<T>(out, i0, x);
  } else {
    for (int64_t i = i0; i < n && i < i0 + 8; ++i) out[i] = from_f<T>(Code<SECOND>::decode(codes[i], s));
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
// small model, so that its launch carries 2 KB, up to 256 otherwise (29 KB of
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
      const int64_t per = (int64_t)kTileBlocks * kBlockValues, add = (t.n + per - 1) / per;
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
  const int64_t blocks = (n + 8 * kThreads - 1) / (8 * kThreads);
  if (blocks > 0x7fffffff) return GQ_ERR_UNSUPPORTED;
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
