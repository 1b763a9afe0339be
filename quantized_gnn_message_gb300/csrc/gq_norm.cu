// gq_norm.cu -- layer normalization of node rows (forward and backward, with
// the ReLU and the dropout that follow it fused in) and counter-based
// dropout.
//
//   mean = (1/d) sum_j x_j,  var = (1/d) sum_j (x_j - mean)^2,
//   rstd = 1 / sqrt(var + eps),  xhat = (x - mean) rstd,
//   z = xhat gamma + beta,  y = drop(act(z))
//   backward: dz = [z > 0] drop'(dy);  dgamma = sum_i dz xhat,
//   dbeta = sum_i dz;  g = dz gamma;
//   dx = rstd (g - mean_j(g) - xhat mean_j(g xhat))
//
// All arithmetic is fp32 whatever the matrices' type; results are rounded
// once, when they are stored.  The variance is a second pass over the
// centred row, which is still in registers, so a large mean costs no digits.
//
// DRAM bound by its bytes (2 n d e forward, 3 n d e backward), and near it by
// its instructions: the noise hash takes 12 of about 30 per element.  A row is
// read once and kept in registers.  Rows of d <= 512 belong to a group of 8,
// 16 or 32 lanes (16 elements a lane at most, sums by shuffles), wider rows to
// a thread block (16 elements a thread, sums through shared memory).  gamma,
// beta and the gradient sums of a lane's columns stay with the lane over all
// the rows it visits; the backward's column sums are combined per block in a
// fixed order, written as one partial row per block and summed by a second
// kernel, so results do not depend on scheduling.
//
// Rows that start 16-byte aligned take the vector path; others are read and
// written element by element (16-bit ones of wide rows in pairs where rows
// start 4-byte aligned), neighbouring lanes on neighbouring columns.
//
// Measured (GB300, copy rate 6.8 TB/s): dropout of 2,449,029 x 256 fp32 0.71 ms
// (7.1 TB/s); backward of the same with ReLU and dropout 1.31 ms (5.8 TB/s);
// forward of 131,072 x 256 fp32 with ReLU 47 us (5.7 TB/s); 30,001 x 4,099
// bf16 with dropout, forward and backward, 430 us (2.9 TB/s).  Rows of more
// than 8,192 columns keep a backward pass's column sums in shared memory and
// spill registers: 10,000 x 16,384 fp32 610 us (3.2 TB/s), bf16 440 us, off the
// 16-byte grid 1.1 ms.
//
// Dropout draws u(seed, row, column) from the library's counter hash (see
// gq_quantize_pack) and keeps an element when u >= p, so the backward pass
// recomputes the mask from the seed and no mask is stored.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "gq_common.cuh"
#include "gq_internal.cuh"
#include "gq_sm100.cuh"
#include "gq_train.h"

namespace gq {
namespace {

constexpr int kEpt = 16;           // elements of a row per lane or thread
constexpr int kWarpRowMax = 512;   // rows up to here are one warp's (or less)
constexpr int kMaxWidth = 16384;   // 1024 threads x 16 elements
constexpr int kNormThreads = 256;
// dropout's columns are counted in 31 bits; a thread's next ones are up to
// 256 threads x 8 elements further
constexpr int kMaxDropWidth = 0x7fffffff - 4095;

// 1 / sqrt(v): the hardware estimate and one Newton step (2 ulp), a fifth of
// the instructions of a rounded root and quotient.
__device__ __forceinline__ float inv_sqrt(float v) {
  const float y = rsqrtf(v);
  const float e = __fmaf_rn(-v * y, y, 1.0f);
  return v > 0.0f && e == e ? __fmaf_rn(0.5f * e, y, y) : y;  // y itself at 0 and infinity
}

// ---------------------------------------------------------- vector access --
__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ void from_f(float v, float* o) { *o = v; }
__device__ __forceinline__ void from_f(float v, __nv_bfloat16* o) { *o = __float2bfloat16_rn(v); }
__device__ __forceinline__ void from_f(float v, __half* o) { *o = __float2half_rn(v); }

template <typename T>
struct alignas(16) Pack16 {
  T v[16 / sizeof(T)];
};

// V elements at p (columns col .. col + V - 1 of a row of d), zeros past d
template <typename T, int V>
__device__ __forceinline__ void load_vec(const T* p, int col, int d, float (&o)[V]) {
  if (V * sizeof(T) == 16 && col + V <= d) {
    const Pack16<T> q = *reinterpret_cast<const Pack16<T>*>(p + col);
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] = to_f(q.v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] = col + j < d ? to_f(p[col + j]) : 0.0f;
  }
}

// The same elements as they are stored, to be converted later: a row on its
// way while another one is worked on.  A vector stays the four words of its
// load: taking 16-bit elements apart would wait for them.
template <typename T, int V>
struct Raw {
  uint32_t w[V * sizeof(T) >= 4 ? V * sizeof(T) / 4 : 1];
};
template <typename T, int V>
__device__ __forceinline__ void load_raw(const T* p, int col, int d, Raw<T, V>& o) {
  if constexpr (V * sizeof(T) == 16) {
    if (col + V <= d) {
      const uint4 q = *reinterpret_cast<const uint4*>(p + col);
      o.w[0] = q.x, o.w[1] = q.y, o.w[2] = q.z, o.w[3] = q.w;
      return;
    }
  }
  if constexpr (V == 2 && sizeof(T) == 2) {
    if (col + 2 <= d) {
      o.w[0] = *reinterpret_cast<const uint32_t*>(p + col);
      return;
    }
  }
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int j = 0; j < V; ++j) o.w[j] = col + j < d ? reinterpret_cast<const uint32_t*>(p)[col + j] : 0u;
  } else if constexpr (V == 1) {
    o.w[0] = col < d ? reinterpret_cast<const uint16_t*>(p)[col] : 0u;
  } else {
#pragma unroll
    for (int j = 0; j < V; j += 2) {
      const uint32_t lo = col + j < d ? reinterpret_cast<const uint16_t*>(p)[col + j] : 0u;
      const uint32_t hi = col + j + 1 < d ? reinterpret_cast<const uint16_t*>(p)[col + j + 1] : 0u;
      o.w[j / 2] = lo | hi << 16;
    }
  }
}
template <typename T, int V>
__device__ __forceinline__ void unpack(const Raw<T, V>& r, float* o) {
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if constexpr (sizeof(T) == 4) {
      o[j] = __uint_as_float(r.w[j]);
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {  // the upper half of an fp32
      const uint32_t w = V == 1 ? r.w[0] : r.w[j / 2];
      o[j] = __uint_as_float(V > 1 && (j & 1) ? w & 0xffff0000u : w << 16);
    } else {
      const uint16_t u = (uint16_t)(V == 1 ? r.w[0] : r.w[j / 2] >> (16 * (j & 1)));
      T t;
      memcpy(&t, &u, 2);
      o[j] = to_f(t);
    }
  }
}

// Asynchronous 16-byte copies into a thread's own slots of shared memory,
// zeros past the end of the row: rows on their way that need no registers,
// and no barrier, since each thread reads what it copied itself.
template <typename T, int V>
__device__ __forceinline__ void copy_vec(uint4* slot, const T* p, int col, int d) {
  const int bytes = min(max(d - col, 0) * (int)sizeof(T), 16);
  const T* src = bytes > 0 ? p + col : p;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(slot)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
template <typename T, int V>
__device__ __forceinline__ void read_slot(const uint4* slot, float* o) {
  const uint4 q = *slot;
  Raw<T, V> r;
  r.w[0] = q.x, r.w[1] = q.y, r.w[2] = q.z, r.w[3] = q.w;
  unpack<T, V>(r, o);
}

// stores V elements; VEC: p is aligned for one store of the whole vector
template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, int col, int d, const float (&o)[V], bool vec) {
  if (V > 1 && vec && col + V <= d) {
    struct alignas(V * sizeof(T)) P {
      T v[V];
    } q;
#pragma unroll
    for (int j = 0; j < V; ++j) from_f(o[j], &q.v[j]);
    *reinterpret_cast<P*>(p + col) = q;
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (col + j < d) from_f(o[j], p + col + j);
  }
}

// V consecutive floats of shared memory (16-byte aligned for V >= 4)
template <int V>
__device__ __forceinline__ void load_shared(const float* p, float* o) {
  if (V >= 4) {
#pragma unroll
    for (int j = 0; j < V; j += 4) {
      const float4 q = *reinterpret_cast<const float4*>(p + j);
      o[j] = q.x;
      o[j + 1] = q.y;
      o[j + 2] = q.z;
      o[j + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] = p[j];
  }
}
template <int V>
__device__ __forceinline__ void store_shared(float* p, const float* o) {
  if (V >= 4) {
#pragma unroll
    for (int j = 0; j < V; j += 4) *reinterpret_cast<float4*>(p + j) = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) p[j] = o[j];
  }
}

template <int V>
__device__ __forceinline__ void load_param(const float* p, int col, int d, float none, float (&o)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) o[j] = p == nullptr ? none : (col + j < d ? __ldg(p + col + j) : 0.0f);
}

// Dropout: an element is kept when its 23-bit noise code, the upper bits of
// the hash, is at least T = ceil(p 2^23), that is when the whole hash exceeds
// lim = 512 T - 1 (p = 1: T = 2^23 and nothing exceeds lim).
struct Drop {
  uint32_t on;    // 0: p = 0, nothing is dropped and the hash is skipped
  uint32_t lim;
  float scale;    // 1 / (1 - p)
  uint32_t key;   // fmix32(low32(seed) ^ high32(seed))
};

constexpr uint32_t kColMul = 0x9E3779B9u;

// hash of column col0 + j of the row whose key is krow; base = krow + col0 kColMul
__device__ __forceinline__ bool kept(uint32_t base, int j, uint32_t lim) {
  return fmix32(base + (uint32_t)j * kColMul) > lim;
}

// s / d to the nearest: the product with 1 / d, corrected by its remainder
// (exact where the quotient is, as for the sum of a constant row).
struct Div {
  float d, inv;
};
__device__ __forceinline__ float over(float s, const Div& v) {
  const float q = s * v.inv;
  return fabsf(q) < INFINITY ? __fmaf_rn(__fmaf_rn(-q, v.d, s), v.inv, q) : q;
}

// ---------------------------------------------------------------- dropout --
// A block covers rpb rows at a time, tpr threads a row, kDropRows such row
// sets per block, all loaded before the first is used: at 16 bytes a thread
// one load in flight per thread is half of what the memory latency needs.
// 17.8M x 4 fp32 attention values: 86 us (6.7 TB/s).
constexpr int kDropRows = 4;

template <typename T, int V>
__global__ void __launch_bounds__(kNormThreads)
    dropout_kernel(const T* X, int64_t n, int d, int64_t ldx, const Drop dr, T* Y, int64_t ldy, int tpr, int rpb) {
  const int local = (int)threadIdx.x / tpr;
  if (local >= rpb) return;
  constexpr int U = kDropRows;
  const int64_t r0 = (int64_t)blockIdx.x * rpb * U + local;
  for (int col = ((int)threadIdx.x - local * tpr) * V; col < d; col += tpr * V) {
    float v[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = r0 + (int64_t)u * rpb;
      if (r < n) load_vec<T, V>(X + r * ldx, col, d, v[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = r0 + (int64_t)u * rpb;
      if (r >= n) break;
      if (dr.on) {
        const uint32_t base = row_key(dr.key, (uint32_t)r) + (uint32_t)col * kColMul;
#pragma unroll
        for (int j = 0; j < V; ++j) v[u][j] = kept(base, j, dr.lim) ? v[u][j] * dr.scale : 0.0f;
      }
      store_vec<T, V>(Y + r * ldy, col, d, v[u], true);
    }
  }
}

// Rows that start anywhere, d >= 32: a warp per row, eight elements of a lane
// on their way at once.  2,449,029 x 251 bf16 0.50 ms, fp32 0.73 ms; the kernel
// above hashes a row's key again for each element there, 1.26 ms in bf16.
template <typename T>
__global__ void __launch_bounds__(kNormThreads)
    dropout_rows_kernel(const T* X, int64_t n, int d, int64_t ldx, const Drop dr, T* Y, int64_t ldy) {
  constexpr int U = 8;
  const int lane = threadIdx.x & 31;
  const int64_t step = (int64_t)gridDim.x * (kNormThreads / 32);
  for (int64_t r = (int64_t)blockIdx.x * (kNormThreads / 32) + (threadIdx.x >> 5); r < n; r += step) {
    const T* x = X + r * ldx;
    T* y = Y + r * ldy;
    const uint32_t kr = row_key(dr.key, (uint32_t)r);
    for (int c = lane; c < d; c += 32 * U) {
      float v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = c + 32 * u < d ? to_f(x[c + 32 * u]) : 0.0f;
      if (dr.on) {
        const uint32_t base = kr + (uint32_t)c * kColMul;
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = kept(base, 32 * u, dr.lim) ? v[u] * dr.scale : 0.0f;
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (c + 32 * u < d) from_f(v[u], y + c + 32 * u);
    }
  }
}

// ------------------------------------------------------ sums over a group --
// Sum over the G lanes of a group (G <= 32, aligned), the same in each.
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
  return v;
}

// Sums of two values over the block, the same in each thread.  `red` holds
// 2 x 32 floats and alternates between calls, so one barrier is enough.
__device__ __forceinline__ float2 block_sum2(float a, float b, float* red) {
  a = group_sum<32>(a);
  b = group_sum<32>(b);
  const int w = threadIdx.x >> 5, nw = blockDim.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) {
    red[w] = a;
    red[32 + w] = b;
  }
  __syncthreads();
  a = lane < nw ? red[lane] : 0.0f;
  b = lane < nw ? red[32 + lane] : 0.0f;
  return make_float2(group_sum<32>(a), group_sum<32>(b));
}

// OR of the lanes' V bits into 32-column words: word of the lane's columns,
// complete in every lane of the 32 / V lanes that share it.
template <int V>
__device__ __forceinline__ uint32_t gather_bits(uint32_t bits, int col) {
  if (V == 1) return __ballot_sync(FULL, bits);
  uint32_t w = bits << (col & 31);
#pragma unroll
  for (int o = 1; o < 32 / V; o <<= 1) w |= __shfl_xor_sync(FULL, w, o);
  return w;
}

// s plus V values
template <int V>
__device__ __forceinline__ float sum_of(const float* v, float s) {
  if constexpr (V > 1) {
    float2 a = make_float2(s, 0.0f);
#pragma unroll
    for (int j = 0; j < V; j += 2) a = add2(a, make_float2(v[j], v[j + 1]));
    return a.x + a.y;
  }
  return s + v[0];
}

// Centres V values of a row (those past its end become 0) and adds their
// squares to q; `whole`: all V columns are in the row.
template <int V>
__device__ __forceinline__ float centre(float* v, float mean, bool whole, int col, int d, float q) {
  if constexpr (V > 1) {
    if (whole) {
      const float2 nm = make_float2(-mean, -mean);
      float2 a = make_float2(q, 0.0f);
#pragma unroll
      for (int j = 0; j < V; j += 2) {
        const float2 e = add2(make_float2(v[j], v[j + 1]), nm);
        a = fma2(e, e, a);
        v[j] = e.x, v[j + 1] = e.y;
      }
      return a.x + a.y;
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    v[j] = col + j < d ? v[j] - mean : 0.0f;
    q = __fmaf_rn(v[j], v[j], q);
  }
  return q;
}

struct NormFwd {
  const void* X;
  int64_t n, ldx;
  int d;
  const float* gamma;
  const float* beta;
  float eps;
  Div dv;
  int relu;
  Drop dr;
  void* Y;
  int64_t ldy;
  float* mean;
  float* rstd;
  uint32_t* bits;
  int64_t ldrb;
};

// V outputs of a row from its centred values xc + off, with shift = off rstd.
// Every lane of the warp
// takes part (the bits are gathered by shuffles); `live` lanes store.
template <typename T, int V>
__device__ __forceinline__ void norm_emit(const NormFwd& p, int64_t r, uint32_t kr, bool live, float rstd, float shift,
                                          int col, const float* xc, const float* ga, const float* be) {
  float y[V];
  uint32_t pos = 0;
  if constexpr (V > 1) {
    const float2 rs = make_float2(rstd, rstd), sh = make_float2(shift, shift);
#pragma unroll
    for (int j = 0; j < V; j += 2) {
      const float2 z = fma2(fma2(make_float2(xc[j], xc[j + 1]), rs, sh), make_float2(ga[j], ga[j + 1]),
                            make_float2(be[j], be[j + 1]));
      y[j] = z.x, y[j + 1] = z.y;
    }
  } else {
    y[0] = __fmaf_rn(__fmaf_rn(xc[0], rstd, shift), ga[0], be[0]);
  }
  if (p.relu) {
    if (p.bits != nullptr) {
#pragma unroll
      for (int j = 0; j < V; ++j) pos |= (uint32_t)(y[j] > 0.0f && col + j < p.d) << j;
    }
#pragma unroll
    for (int j = 0; j < V; ++j) y[j] = fmaxf(y[j], 0.0f);
  }
  if (p.dr.on) {
    const uint32_t base = kr + (uint32_t)col * kColMul;
#pragma unroll
    for (int j = 0; j < V; ++j) y[j] = kept(base, j, p.dr.lim) ? y[j] * p.dr.scale : 0.0f;
  }
  if (live && col < p.d) store_vec<T, V>(static_cast<T*>(p.Y) + r * p.ldy, col, p.d, y, true);
  if (p.bits != nullptr) {
    const uint32_t w = gather_bits<V>(pos, col);
    if (live && (col & 31) == 0 && col < p.d) p.bits[r * p.ldrb + (col >> 5)] = w;
  }
}

// Rows of d <= 512: a group of G lanes per row (V = 1: G = 32, so that a
// word of bits is one vector).  WHOLE: d = G NV V, no column to leave out.
template <typename T, int V, int NV, int G, bool WHOLE>
__global__ void __launch_bounds__(kNormThreads) norm_fwd_warp_kernel(const NormFwd p) {
  constexpr int kGroups = 32 / G;
  const int lane = threadIdx.x & 31, sub = lane / G;
  const int c0 = (lane % G) * V;
  const int64_t warp = ((int64_t)blockIdx.x * kNormThreads + threadIdx.x) >> 5;
  const int64_t step = (int64_t)gridDim.x * (kNormThreads / 32) * kGroups;
  float ga[NV][V], be[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    load_param<V>(p.gamma, c0 + i * G * V, p.d, 1.0f, ga[i]);
    load_param<V>(p.beta, c0 + i * G * V, p.d, 0.0f, be[i]);
  }
  Raw<T, V> nx[NV];  // the next row is on its way while one is worked on
  auto fetch = [&](int64_t rw) {
    const T* x = static_cast<const T*>(p.X) + (rw + sub < p.n ? rw + sub : rw) * p.ldx;
#pragma unroll
    for (int i = 0; i < NV; ++i) load_raw<T, V>(x, c0 + i * G * V, p.d, nx[i]);
  };
  if (warp * kGroups < p.n) fetch(warp * kGroups);
  for (int64_t rw = warp * kGroups; rw < p.n; rw += step) {
    const int64_t r = rw + sub;
    const bool live = r < p.n;
    float v[NV][V];
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      unpack<T, V>(nx[i], v[i]);
      s = sum_of<V>(v[i], s);
    }
    if (rw + step < p.n) fetch(rw + step);
    const float mean = over(group_sum<G>(s), p.dv);
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) q = centre<V>(v[i], mean, WHOLE || c0 + i * G * V + V <= p.d, c0 + i * G * V, p.d, q);
    const float rstd = inv_sqrt(over(group_sum<G>(q), p.dv) + p.eps);
    if (live && lane % G == 0) {
      if (p.mean != nullptr) p.mean[r] = mean;
      if (p.rstd != nullptr) p.rstd[r] = rstd;
    }
    const uint32_t kr = row_key(p.dr.key, (uint32_t)r);
#pragma unroll
    for (int i = 0; i < NV; ++i) norm_emit<T, V>(p, r, kr, live, rstd, 0.0f, c0 + i * G * V, v[i], ga[i], be[i]);
  }
}

// Wider rows: a block per row, thread t holding columns (i blockDim + t) V.
// Each warp forms the mean m_w of its n_w columns and their squared distances
// q_w from it; one barrier later every thread joins the warps' triples:
//   mean = sum n_w m_w / d,  d var = sum q_w + sum n_w (m_w - mean)^2
// (both sums of non-negative terms), so a row costs one barrier.  The next
// row is loaded before the barrier; gamma and beta stay in shared memory.
template <typename T, int V>
__global__ void __launch_bounds__(1024, 1) norm_fwd_block_kernel(const NormFwd p) {
  constexpr int NV = kEpt / V;
  extern __shared__ float par[];  // gamma | beta, each blockDim * kEpt
  __shared__ float red[2][96];
  const int c0 = (int)threadIdx.x * V, cs = (int)blockDim.x * V, W = (int)blockDim.x * kEpt;
  const int w = threadIdx.x >> 5, nw = blockDim.x >> 5, lane = threadIdx.x & 31;
  for (int c = threadIdx.x; c < W; c += blockDim.x) {
    par[c] = c < p.d ? (p.gamma != nullptr ? p.gamma[c] : 1.0f) : 0.0f;
    par[W + c] = c < p.d && p.beta != nullptr ? p.beta[c] : 0.0f;
  }
  float cols = 0.0f;  // columns of this warp
#pragma unroll
  for (int i = 0; i < NV; ++i) cols += (float)min(max(p.d - (c0 + i * cs), 0), V);
  cols = group_sum<32>(cols);
  int flip = 0;
  int64_t r = blockIdx.x;
  Raw<T, V> nx[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) load_raw<T, V>(static_cast<const T*>(p.X) + r * p.ldx, c0 + i * cs, p.d, nx[i]);
  __syncthreads();
  for (; r < p.n; r += gridDim.x) {
    float v[NV][V];
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      unpack<T, V>(nx[i], v[i]);
      s = sum_of<V>(v[i], s);
    }
    if (r + gridDim.x < p.n) {
      const T* x = static_cast<const T*>(p.X) + (r + gridDim.x) * p.ldx;
#pragma unroll
      for (int i = 0; i < NV; ++i) load_raw<T, V>(x, c0 + i * cs, p.d, nx[i]);
    }
    const float mw = cols > 0.0f ? group_sum<32>(s) / cols : 0.0f;
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) q = centre<V>(v[i], mw, (i + 1) * cs <= p.d, c0 + i * cs, p.d, q);
    q = group_sum<32>(q);
    float* rd = red[flip];
    flip ^= 1;
    if (lane == 0) {
      rd[w] = cols;
      rd[32 + w] = mw;
      rd[64 + w] = q;
    }
    __syncthreads();
    const float n1 = lane < nw ? rd[lane] : 0.0f, m1 = lane < nw ? rd[32 + lane] : 0.0f;
    const float mean = over(group_sum<32>(n1 * m1), p.dv);
    const float e1 = m1 - mean;
    const float var = over(group_sum<32>(__fmaf_rn(n1 * e1, e1, lane < nw ? rd[64 + lane] : 0.0f)), p.dv);
    const float rstd = inv_sqrt(var + p.eps);
    if (threadIdx.x == 0) {
      if (p.mean != nullptr) p.mean[r] = mean;
      if (p.rstd != nullptr) p.rstd[r] = rstd;
    }
    const float shift = (mw - mean) * rstd;  // from the warp's mean to the row's
    const uint32_t kr = row_key(p.dr.key, (uint32_t)r);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (i * cs >= p.d) break;
      float ga[V], be[V];
      load_shared<V>(par + c0 + i * cs, ga);
      load_shared<V>(par + W + c0 + i * cs, be);
      norm_emit<T, V>(p, r, kr, true, rstd, shift, c0 + i * cs, v[i], ga, be);
    }
  }
}

// --------------------------------------------------------------- backward --
struct NormBwd {
  const void* dY;
  const void* X;
  int64_t n, lddy, ldx;
  int d;
  Div dv;
  const float* mean;
  const float* rstd;
  const float* gamma;
  int relu;
  Drop dr;
  const uint32_t* bits;
  int64_t ldrb;
  void* dX;
  int64_t lddx;
  int vec_out;      // dX rows are aligned for whole-vector stores
  float* partial;   // [block][2][d]: dgamma | dbeta
};

// the ReLU bits of the columns from col on (bit 0: col)
__device__ __forceinline__ uint32_t gate_bits(const NormBwd& p, int64_t r, int col) {
  return p.relu && col < p.d ? __ldg(p.bits + r * p.ldrb + (col >> 5)) >> (col & 31) : 0u;
}

// dz of V columns: the dropout of the forward pass and its ReLU gate w.
// Where dY was past the row it is 0 and stays 0.
template <int V>
__device__ __forceinline__ void gate_dz(const NormBwd& p, uint32_t w, uint32_t kr, int col, float* dz) {
  const uint32_t base = kr + (uint32_t)col * kColMul;
  if (p.relu) {
    if (p.dr.on) {
#pragma unroll
      for (int j = 0; j < V; ++j) dz[j] = (w >> j & 1u) && kept(base, j, p.dr.lim) ? dz[j] * p.dr.scale : 0.0f;
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) dz[j] = (w >> j & 1u) ? dz[j] : 0.0f;
    }
  } else if (p.dr.on) {
#pragma unroll
    for (int j = 0; j < V; ++j) dz[j] = kept(base, j, p.dr.lim) ? dz[j] * p.dr.scale : 0.0f;
  }
}

// The factor of x - mean in xhat: rstd, or 0 for a constant row whose
// mean rstd is beyond fp32 (a row that varies at all has mean rstd below
// 2^24 sqrt(d)).  Its x are the mean, xhat 0; but past the row's end x = 0, and
// an infinite xhat there would make the sums' 0 xhat NaN.
__device__ __forceinline__ float xhat_scale(float mean, float rstd) {
  return rstd < INFINITY && !(fabsf(mean * rstd) < INFINITY) ? 0.0f : rstd;
}

// The backward arithmetic of E (even) elements of a row, two at a time:
// xh = (x - mean) xs over x; g = dz gamma over dz; column sums; s1, s2 the
// row's sums of g and g xh.  Elements past the row have dz = 0 and add
// nothing.
template <int E>
__device__ __forceinline__ void bwd_terms(float* x, float* dz, const float* ga, float* sg, float* sb, float mean,
                                          float xs, float& s1, float& s2) {
  const float2 nm = make_float2(-mean, -mean), rs = make_float2(xs, xs);
  float2 a = make_float2(0.0f, 0.0f), b = a;
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    const float2 xh = mul2(add2(make_float2(x[e], x[e + 1]), nm), rs);
    const float2 z = make_float2(dz[e], dz[e + 1]);
    const float2 ng = fma2(z, xh, make_float2(sg[e], sg[e + 1])), nb = add2(make_float2(sb[e], sb[e + 1]), z);
    const float2 g = mul2(z, make_float2(ga[e], ga[e + 1]));
    a = add2(a, g);
    b = fma2(g, xh, b);
    sg[e] = ng.x, sg[e + 1] = ng.y, sb[e] = nb.x, sb[e + 1] = nb.y;
    x[e] = xh.x, x[e + 1] = xh.y, dz[e] = g.x, dz[e + 1] = g.y;
  }
  s1 += a.x + a.y;
  s2 += b.x + b.y;
}

// rstd (g - m1 - xh m2) of E elements, over g
template <int E>
__device__ __forceinline__ void bwd_out(float* g, const float* xh, float m1, float m2, float rstd) {
  const float2 n1 = make_float2(-m1, -m1), n2 = make_float2(-m2, -m2), rs = make_float2(rstd, rstd);
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    const float2 o =
        mul2(fma2(make_float2(xh[e], xh[e + 1]), n2, add2(make_float2(g[e], g[e + 1]), n1)), rs);
    g[e] = o.x, g[e + 1] = o.y;
  }
}

// The block's column sums from its lanes' (acc: [warp][2][G NV V] floats).
template <int V, int NV, int G>
__device__ __forceinline__ void warp_sums(const NormBwd& p, float* acc, const float* sg, const float* sb) {
  constexpr int kWarps = kNormThreads / 32;
  const int lane = threadIdx.x & 31, sub = lane / G, w = threadIdx.x >> 5;
  const int c0 = (lane % G) * V;
  if (p.partial == nullptr) return;
  constexpr int W = G * NV * V;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float a = sg[i * V + j], b = sb[i * V + j];
#pragma unroll
      for (int o = G; o < 32; o <<= 1) {  // groups of the warp
        a += __shfl_xor_sync(FULL, a, o);
        b += __shfl_xor_sync(FULL, b, o);
      }
      if (sub == 0) {
        acc[(w * 2) * W + c0 + i * G * V + j] = a;
        acc[(w * 2 + 1) * W + c0 + i * G * V + j] = b;
      }
    }
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * p.d; c += kNormThreads) {
    const int k = c >= p.d, col = c - k * p.d;
    float s = 0.0f;
#pragma unroll
    for (int u = 0; u < kWarps; ++u) s += acc[(u * 2 + k) * W + col];
    p.partial[(int64_t)blockIdx.x * 2 * p.d + c] = s;
  }
}

// Rows of d <= 512 that start 16-byte aligned: S - 1 rows of each warp on
// their way through shared memory.  With the next row in registers instead
// (80 to 122 of them a lane, 16 warps per SM) the 2,449,029 x 256 fp32 pass
// waited for its loads: 1.61 ms against 1.31 ms here.
template <typename T, typename TO, int V, int NV, int G, int S>
__global__ void __launch_bounds__(kNormThreads) norm_bwd_ring_kernel(const NormBwd p) {
  constexpr int kGroups = 32 / G;
  constexpr int kWarps = kNormThreads / 32;
  constexpr int E = NV * V;
  extern __shared__ uint4 ring[];  // [warp][S][2 NV][lane]; afterwards the block's sums
  const int lane = threadIdx.x & 31, sub = lane / G, w = threadIdx.x >> 5;
  const int c0 = (lane % G) * V;
  const int64_t step = (int64_t)gridDim.x * kWarps * kGroups;
  uint4* mine = ring + (size_t)w * S * 2 * NV * 32 + lane;
  float ga[E], sg[E], sb[E];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float q[V];
    load_param<V>(p.gamma, c0 + i * G * V, p.d, 1.0f, q);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      ga[i * V + j] = q[j];
      sg[i * V + j] = sb[i * V + j] = 0.0f;
    }
  }
  auto issue = [&](int64_t rw, int slot) {
    if (rw < p.n) {
      const int64_t r = rw + sub < p.n ? rw + sub : rw;
      const int dd = rw + sub < p.n ? p.d : 0;
      uint4* to = mine + slot * 2 * NV * 32;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        copy_vec<T, V>(to + i * 32, static_cast<const T*>(p.X) + r * p.ldx, c0 + i * G * V, p.d);
        copy_vec<T, V>(to + (NV + i) * 32, static_cast<const T*>(p.dY) + r * p.lddy, c0 + i * G * V, dd);
      }
    }
    copy_commit();
  };
  int64_t rw = ((int64_t)blockIdx.x * kWarps + w) * kGroups;
  float nm = 0.0f, nr = 0.0f;
  uint32_t nb[NV] = {};
  auto fetch = [&](int64_t rn) {  // a row's statistics and ReLU bits
    if (rn >= p.n) return;
    const int64_t r = rn + sub < p.n ? rn + sub : rn;
    nm = __ldg(p.mean + r);
    nr = __ldg(p.rstd + r);
#pragma unroll
    for (int i = 0; i < NV; ++i) nb[i] = gate_bits(p, r, c0 + i * G * V);
  };
#pragma unroll
  for (int s = 0; s < S - 1; ++s) issue(rw + s * step, s);
  fetch(rw);
  int slot = 0;
  for (; rw < p.n; rw += step) {
    const int64_t r = rw + sub;
    const bool live = r < p.n;
    const float mean = nm, rstd = nr;
    float xv[E], dz[E];
    uint32_t wb[NV];
    copy_wait<S - 2>();
    const uint4* from = mine + slot * 2 * NV * 32;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      wb[i] = nb[i];
      read_slot<T, V>(from + i * 32, xv + i * V);
      read_slot<T, V>(from + (NV + i) * 32, dz + i * V);
    }
    issue(rw + (S - 1) * step, slot == 0 ? S - 1 : slot - 1);
    fetch(rw + step);
    if (++slot == S) slot = 0;
    const uint32_t kr = row_key(p.dr.key, (uint32_t)(live ? r : rw));
#pragma unroll
    for (int i = 0; i < NV; ++i) gate_dz<V>(p, wb[i], kr, c0 + i * G * V, dz + i * V);
    float s1 = 0.0f, s2 = 0.0f;
    bwd_terms<E>(xv, dz, ga, sg, sb, mean, xhat_scale(mean, rstd), s1, s2);
    const float m1 = over(group_sum<G>(s1), p.dv), m2 = over(group_sum<G>(s2), p.dv);
    bwd_out<E>(dz, xv, m1, m2, rstd);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = c0 + i * G * V;
      if (live && col < p.d)
        store_vec<TO, V>(static_cast<TO*>(p.dX) + r * p.lddx, col, p.d,
                         *reinterpret_cast<const float(*)[V]>(dz + i * V), p.vec_out);
    }
  }
  copy_wait<0>();
  __syncthreads();
  warp_sums<V, NV, G>(p, reinterpret_cast<float*>(ring), sg, sb);
}

template <typename T, typename TO, int V, int NV, int G>
__global__ void __launch_bounds__(kNormThreads) norm_bwd_warp_kernel(const NormBwd p) {
  constexpr int kGroups = 32 / G;
  constexpr int kWarps = kNormThreads / 32;
  constexpr int E = NV * V;
  extern __shared__ float acc[];  // [warp][2][G * NV * V]
  const int lane = threadIdx.x & 31, sub = lane / G, w = threadIdx.x >> 5;
  const int c0 = (lane % G) * V;
  const int64_t warp = (int64_t)blockIdx.x * kWarps + w;
  const int64_t step = (int64_t)gridDim.x * kWarps * kGroups;
  float ga[E], sg[E], sb[E];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float q[V];
    load_param<V>(p.gamma, c0 + i * G * V, p.d, 1.0f, q);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      ga[i * V + j] = q[j];
      sg[i * V + j] = sb[i * V + j] = 0.0f;
    }
  }
  // the next row is on its way while one is worked on
  Raw<T, V> nx[NV], ny[NV];
  float nm = 0.0f, nr = 0.0f;
  uint32_t nb[NV];
  auto fetch = [&](int64_t rw) {
    const int64_t r = rw + sub;
    const int64_t rr = r < p.n ? r : rw;
    const T* x = static_cast<const T*>(p.X) + rr * p.ldx;
    const T* dy = static_cast<const T*>(p.dY) + rr * p.lddy;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      load_raw<T, V>(x, c0 + i * G * V, p.d, nx[i]);
      load_raw<T, V>(dy, c0 + i * G * V, r < p.n ? p.d : 0, ny[i]);
      nb[i] = gate_bits(p, rr, c0 + i * G * V);
    }
    nm = __ldg(p.mean + rr);
    nr = __ldg(p.rstd + rr);
  };
  if (warp * kGroups < p.n) fetch(warp * kGroups);
  for (int64_t rw = warp * kGroups; rw < p.n; rw += step) {
    const int64_t r = rw + sub;
    const bool live = r < p.n;
    const int64_t rr = live ? r : rw;
    const float mean = nm, rstd = nr;
    float xv[E], dz[E];
    uint32_t wb[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      wb[i] = nb[i];
      unpack<T, V>(nx[i], xv + i * V);
      unpack<T, V>(ny[i], dz + i * V);
    }
    if (rw + step < p.n) fetch(rw + step);
    const uint32_t kr = row_key(p.dr.key, (uint32_t)rr);
#pragma unroll
    for (int i = 0; i < NV; ++i) gate_dz<V>(p, wb[i], kr, c0 + i * G * V, dz + i * V);
    float s1 = 0.0f, s2 = 0.0f;
    bwd_terms<E>(xv, dz, ga, sg, sb, mean, xhat_scale(mean, rstd), s1, s2);
    const float m1 = over(group_sum<G>(s1), p.dv), m2 = over(group_sum<G>(s2), p.dv);
    bwd_out<E>(dz, xv, m1, m2, rstd);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = c0 + i * G * V;
      if (live && col < p.d)
        store_vec<TO, V>(static_cast<TO*>(p.dX) + r * p.lddx, col, p.d,
                         *reinterpret_cast<const float(*)[V]>(dz + i * V), p.vec_out);
    }
  }
  warp_sums<V, NV, G>(p, acc, sg, sb);
}

// Wide rows: gamma and the block's column sums live in shared memory, each
// column touched by its one owner thread only; the next row is loaded before
// the current one's barrier.
template <typename T, typename TO, int V, int EPT>
__global__ void __launch_bounds__(1024, 1) norm_bwd_block_kernel(const NormBwd p) {
  constexpr int NV = EPT / V;
  extern __shared__ float acc[];  // dgamma | dbeta | gamma, each blockDim * EPT
  __shared__ float red[2][64];
  const int c0 = (int)threadIdx.x * V, cs = (int)blockDim.x * V;
  const int W = (int)blockDim.x * EPT;
  for (int c = threadIdx.x; c < W; c += blockDim.x) {
    acc[c] = acc[W + c] = 0.0f;
    acc[2 * W + c] = c < p.d ? (p.gamma != nullptr ? p.gamma[c] : 1.0f) : 0.0f;
  }
  int flip = 0;
  int64_t r = blockIdx.x;
  Raw<T, V> nx[NV], ny[NV];
  float nm, nr;
  uint32_t nb[NV];
  auto fetch = [&](int64_t row) {
    const T* x = static_cast<const T*>(p.X) + row * p.ldx;
    const T* dy = static_cast<const T*>(p.dY) + row * p.lddy;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      load_raw<T, V>(x, c0 + i * cs, p.d, nx[i]);
      load_raw<T, V>(dy, c0 + i * cs, p.d, ny[i]);
      nb[i] = gate_bits(p, row, c0 + i * cs);
    }
    nm = __ldg(p.mean + row);
    nr = __ldg(p.rstd + row);
  };
  fetch(r);
  __syncthreads();
  for (; r < p.n; r += gridDim.x) {
    const float mean = nm, rstd = nr, xs = xhat_scale(mean, rstd);
    const uint32_t kr = row_key(p.dr.key, (uint32_t)r);
    float xh[EPT], g[EPT];
    uint32_t wb[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      wb[i] = nb[i];
      unpack<T, V>(nx[i], xh + i * V);
      unpack<T, V>(ny[i], g + i * V);
    }
    if (r + gridDim.x < p.n) fetch(r + gridDim.x);
    float s1 = 0.0f, s2 = 0.0f;
    constexpr int S = V > 1 ? V : 2;  // elements at a time
#pragma unroll
    for (int e = 0; e < EPT; e += S) {
      float sg[S], sb[S], ga[S];
#pragma unroll
      for (int k = 0; k < S; k += V) {
        const int col = c0 + (e + k) / V * cs;
        gate_dz<V>(p, wb[(e + k) / V], kr, col, g + e + k);
        load_shared<V>(acc + col, sg + k);
        load_shared<V>(acc + W + col, sb + k);
        load_shared<V>(acc + 2 * W + col, ga + k);
      }
      bwd_terms<S>(xh + e, g + e, ga, sg, sb, mean, xs, s1, s2);
#pragma unroll
      for (int k = 0; k < S; k += V) {
        const int col = c0 + (e + k) / V * cs;
        store_shared<V>(acc + col, sg + k);
        store_shared<V>(acc + W + col, sb + k);
      }
    }
    const float2 s = block_sum2(s1, s2, red[flip]);
    flip ^= 1;
    bwd_out<EPT>(g, xh, over(s.x, p.dv), over(s.y, p.dv), rstd);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = c0 + i * cs;
      if (col < p.d)
        store_vec<TO, V>(static_cast<TO*>(p.dX) + r * p.lddx, col, p.d,
                         *reinterpret_cast<const float(*)[V]>(g + i * V), p.vec_out);
    }
  }
  if (p.partial == nullptr) return;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int col = c0 + i * cs + j;
      if (col >= p.d) continue;
      p.partial[(int64_t)blockIdx.x * 2 * p.d + col] = acc[col];
      p.partial[(int64_t)blockIdx.x * 2 * p.d + p.d + col] = acc[W + col];
    }
}

// Wide rows up to 8,192 columns that start 16-byte aligned: the column sums
// and the row at work in registers (96 to 128 a thread), S - 1 rows on their
// way through shared memory, gamma there too.  30,001 x 4,099 bf16: 230 us, with
// dropout 260; with the sums in shared memory (norm_bwd_block_kernel) 390 us,
// its shared memory pipe the bound.
template <typename T, typename TO, int V, int S, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) norm_bwd_wide_kernel(const NormBwd p) {
  constexpr int NV = kEpt / V;
  extern __shared__ uint4 ring[];  // [S][2 NV][thread], then gamma [blockDim * kEpt]
  __shared__ float red[2][64];
  const int T0 = (int)blockDim.x;
  float* gam = reinterpret_cast<float*>(ring + (size_t)S * 2 * NV * T0);
  uint4* mine = ring + threadIdx.x;
  const int c0 = (int)threadIdx.x * V, cs = T0 * V;
  for (int c = threadIdx.x; c < T0 * kEpt; c += T0)
    gam[c] = c < p.d ? (p.gamma != nullptr ? p.gamma[c] : 1.0f) : 0.0f;
  float sg[kEpt], sb[kEpt];
#pragma unroll
  for (int e = 0; e < kEpt; ++e) sg[e] = sb[e] = 0.0f;
  auto issue = [&](int64_t r, int slot) {
    if (r < p.n) {
      uint4* to = mine + slot * 2 * NV * T0;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        copy_vec<T, V>(to + i * T0, static_cast<const T*>(p.X) + r * p.ldx, c0 + i * cs, p.d);
        copy_vec<T, V>(to + (NV + i) * T0, static_cast<const T*>(p.dY) + r * p.lddy, c0 + i * cs, p.d);
      }
    }
    copy_commit();
  };
  int64_t r = blockIdx.x;
  float nm = 0.0f, nr = 0.0f;
  uint32_t nb[NV] = {};
  auto fetch = [&](int64_t rn) {
    if (rn >= p.n) return;
    nm = __ldg(p.mean + rn);
    nr = __ldg(p.rstd + rn);
#pragma unroll
    for (int i = 0; i < NV; ++i) nb[i] = gate_bits(p, rn, c0 + i * cs);
  };
#pragma unroll
  for (int s = 0; s < S - 1; ++s) issue(r + (int64_t)s * gridDim.x, s);
  fetch(r);
  __syncthreads();
  int slot = 0, flip = 0;
  for (; r < p.n; r += gridDim.x) {
    const float mean = nm, rstd = nr, xs = xhat_scale(mean, rstd);
    float xv[kEpt], dz[kEpt];
    uint32_t wb[NV];
    copy_wait<S - 2>();
    const uint4* from = mine + slot * 2 * NV * T0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      wb[i] = nb[i];
      read_slot<T, V>(from + i * T0, xv + i * V);
      read_slot<T, V>(from + (NV + i) * T0, dz + i * V);
    }
    issue(r + (int64_t)(S - 1) * gridDim.x, slot == 0 ? S - 1 : slot - 1);
    fetch(r + gridDim.x);
    if (++slot == S) slot = 0;
    const uint32_t kr = row_key(p.dr.key, (uint32_t)r);
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float ga[V];
      gate_dz<V>(p, wb[i], kr, c0 + i * cs, dz + i * V);
      load_shared<V>(gam + c0 + i * cs, ga);
      bwd_terms<V>(xv + i * V, dz + i * V, ga, sg + i * V, sb + i * V, mean, xs, s1, s2);
    }
    const float2 s = block_sum2(s1, s2, red[flip]);
    flip ^= 1;
    bwd_out<kEpt>(dz, xv, over(s.x, p.dv), over(s.y, p.dv), rstd);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = c0 + i * cs;
      if (col < p.d)
        store_vec<TO, V>(static_cast<TO*>(p.dX) + r * p.lddx, col, p.d,
                         *reinterpret_cast<const float(*)[V]>(dz + i * V), p.vec_out);
    }
  }
  copy_wait<0>();
  if (p.partial == nullptr) return;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int col = c0 + i * cs + j;
      if (col >= p.d) continue;
      p.partial[(int64_t)blockIdx.x * 2 * p.d + col] = sg[i * V + j];
      p.partial[(int64_t)blockIdx.x * 2 * p.d + p.d + col] = sb[i * V + j];
    }
}

// out[c] = sum over the blocks' partial rows, 32 columns per block, 32 row
// lanes whose sums are added in lane order.
__global__ void __launch_bounds__(1024) norm_reduce_kernel(const float* partial, int blocks, int d,
                                                           float* dgamma, float* dbeta) {
  grid_wait();
  __shared__ float s[32][33];
  const int c = (int)blockIdx.x * 32 + (int)(threadIdx.x & 31), lane = threadIdx.x >> 5;
  float a = 0.0f;
  if (c < 2 * d)
    for (int b = lane; b < blocks; b += 32) a += partial[(int64_t)b * 2 * d + c];
  s[lane][threadIdx.x & 31] = a;
  __syncthreads();
  if (lane != 0 || c >= 2 * d) return;
  a = 0.0f;
  for (int k = 0; k < 32; ++k) a += s[k][threadIdx.x];
  float* out = c < d ? dgamma : dbeta;
  if (out != nullptr) out[c < d ? c : c - d] = a;
}

// ------------------------------------------------------------------- host --
int type_bytes(int type) { return type == GQ_F32 ? 4 : (type == GQ_BF16 || type == GQ_F16) ? 2 : 0; }

// Elements at a time for rows of two matrices: 16 bytes, or two 16-bit ones,
// where the rows of both start so aligned; else one.
int vec_of(const void* p, int64_t ldp, const void* q, int64_t ldq, int type) {
  const int e = type_bytes(type);
  for (int v = 16 / e; v > 1; v = e == 2 && v > 2 ? 2 : 1)
    if (aligned(p, v * e) && aligned(q, v * e) && ldp % v == 0 && ldq % v == 0) return v;
  return 1;
}

int make_drop(double p, uint64_t seed, Drop* d) {
  if (!(p >= 0.0 && p <= 1.0)) return GQ_ERR_INVALID_ARG;
  const uint32_t t = (uint32_t)std::ceil(p * 8388608.0);
  d->on = t > 0;
  d->lim = t * 512u - 1u;  // p = 1: 2^32 - 1
  d->scale = p < 1.0 ? (float)(1.0 / (1.0 - p)) : 0.0f;
  d->key = seed_key_host(seed);
  return GQ_OK;
}

// Resident blocks of a wide-row kernel per SM: about 1024 threads (64
// registers a thread), within 200 KB of shared memory.
int block_rows_per_sm(int threads, size_t smem) {
  int per = 1024 / threads;
  while (per > 1 && per * smem > 200 * 1024) --per;
  return per < 1 ? 1 : per;
}

// Elements per thread of a wide row's backward pass: 8 keep the two rows in
// flight within 64 registers; beyond 1024 threads, 16.
int bwd_ept(int d) { return d <= 8192 ? 8 : 16; }

// norm_bwd_wide_kernel is built for three sizes of blocks.  Two blocks of up to
// 256 threads share an SM at the 128 registers that a thread can use (96 of
// them, to fit more threads: 120,000 x 1,024 bf16 163 -> 198 us, fp32 249 -> 281,
// 30,000 x 4,096 bf16 164 -> 220).  Above that one block has the SM, but for
// 16-bit rows of up to 288 threads with dropout, whose hash needs the warps
// more than the registers: two blocks, at 96 (with dropout 4,099 bf16 columns
// 285 -> 263 us, 4,608 248 -> 232, from 4,864 on no difference; without it 229
// -> 233 and 200 -> 204).
constexpr int kPairThreads = 256, kPairThreadsDrop = 288;
int wide_threads(int d) { return ((d + kEpt - 1) / kEpt + 31) / 32 * 32; }
// At most so many of its blocks are resident per SM, as far as registers go.
int wide_per_sm(int threads) { return threads <= kPairThreadsDrop ? 2 * kPairThreadsDrop / threads : 1; }

// Upper bound of the backward's blocks, one partial row of sums each.
int bwd_blocks(int64_t n, int d) {
  // enough blocks to fill the SMs (8 x 256 threads, or about 1024 threads of
  // wide rows, each), and no more partial rows than that
  const int sms = sm_count();
  if (d <= kWarpRowMax) {
    const int64_t want = (n + 7) / 8;
    return (int)(want < 8 * sms ? (want < 1 ? 1 : want) : 8 * sms);
  }
  const int ept = bwd_ept(d), threads = ((d + ept - 1) / ept + 31) / 32 * 32;
  int per = block_rows_per_sm(threads, (size_t)3 * threads * ept * sizeof(float));
  if (per < wide_per_sm(wide_threads(d))) per = wide_per_sm(wide_threads(d));
  const int64_t cap = (int64_t)per * sms;
  return (int)(n < cap ? (n < 1 ? 1 : n) : cap);
}

template <typename T>
int launch_dropout(const void* X, int64_t n, int d, int64_t ldx, const Drop& dr, void* Y, int64_t ldy,
                   cudaStream_t s) {
  const int V = vec_of(X, ldx, Y, ldy, sizeof(T) == 4 ? GQ_F32 : GQ_BF16) * (int)sizeof(T) == 16 ? 16 / (int)sizeof(T) : 1;
  if (V == 1 && d >= 32) {
    const int64_t want = (n + kNormThreads / 32 - 1) / (kNormThreads / 32), cap = (int64_t)sm_count() * 64;
    dropout_rows_kernel<T><<<(unsigned)(want < cap ? want : cap), kNormThreads, 0, s>>>(
        static_cast<const T*>(X), n, d, ldx, dr, static_cast<T*>(Y), ldy);
    return launch_status();
  }
  const int vpr = (d + V - 1) / V;
  const int passes = (vpr + kNormThreads - 1) / kNormThreads;
  const int tpr = (vpr + passes - 1) / passes;
  const int rpb = kNormThreads / tpr;
  const int64_t blocks = (n + (int64_t)rpb * kDropRows - 1) / ((int64_t)rpb * kDropRows);
  if (blocks > 0x7fffffff) return GQ_ERR_UNSUPPORTED;
  const int threads = (tpr * rpb + 31) / 32 * 32;
  auto kernel = V > 1 ? dropout_kernel<T, 16 / sizeof(T)> : dropout_kernel<T, 1>;
  kernel<<<(unsigned)blocks, threads, 0, s>>>(static_cast<const T*>(X), n, d, ldx, dr, static_cast<T*>(Y), ldy, tpr,
                                              rpb);
  return launch_status();
}

// Blocks of a persistent kernel: as many as are resident at once (one wave;
// 2.7 waves of 8 blocks per SM cost the 131,072 x 256 forward pass a tenth), at
// most `want`.
template <typename K>
int wave(K kernel, int threads, size_t smem, int64_t want) {
  int per = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, threads, smem) != cudaSuccess || per < 1) per = 1;
  const int64_t cap = (int64_t)per * sm_count();
  return (int)(want < cap ? want : cap);
}

template <typename T, int V, int NV, int G>
int fwd_warp(const NormFwd& p, cudaStream_t s) {
  constexpr int rows = kNormThreads / G;
  const int64_t want = (p.n + rows - 1) / rows;
  auto kernel = V > 2 && p.d == G * NV * V ? norm_fwd_warp_kernel<T, V, NV, G, (V > 2)>
                                           : norm_fwd_warp_kernel<T, V, NV, G, false>;
  kernel<<<wave(kernel, kNormThreads, 0, want), kNormThreads, 0, s>>>(p);
  return launch_status();
}

template <typename T, int V>
int fwd_any(const NormFwd& p, cudaStream_t s) {
  if constexpr (V == 2) {  // wide rows only, see fwd_typed
  } else if constexpr (V == 1) {
    if (p.d <= 64) return fwd_warp<T, 1, 2, 32>(p, s);
    if (p.d <= 128) return fwd_warp<T, 1, 4, 32>(p, s);
    if (p.d <= 256) return fwd_warp<T, 1, 8, 32>(p, s);
    if (p.d <= 384) return fwd_warp<T, 1, 12, 32>(p, s);
    if (p.d <= 512) return fwd_warp<T, 1, 16, 32>(p, s);
  } else {
    if (p.d <= 8 * V) return fwd_warp<T, V, 1, 8>(p, s);
    if (p.d <= 16 * V) return fwd_warp<T, V, 1, 16>(p, s);
    if (p.d <= 32 * V) return fwd_warp<T, V, 1, 32>(p, s);
    if (p.d <= 64 * V) return fwd_warp<T, V, 2, 32>(p, s);
    if constexpr (V == 4)
      if (p.d <= 128 * V) return fwd_warp<T, V, 4, 32>(p, s);
  }
  const int threads = ((p.d + kEpt - 1) / kEpt + 31) / 32 * 32;
  const size_t smem = (size_t)2 * threads * kEpt * sizeof(float);
  const int64_t cap = (int64_t)sm_count() * block_rows_per_sm(threads, smem);
  const int grid = (int)(p.n < cap ? p.n : cap);
  GQ_TRY_CUDA(cudaFuncSetAttribute(norm_fwd_block_kernel<T, V>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   2 * kMaxWidth * (int)sizeof(float)));
  norm_fwd_block_kernel<T, V><<<grid, threads, smem, s>>>(p);
  return launch_status();
}

template <typename T, typename TO, int V, int NV, int G>
int bwd_warp(const NormBwd& p, int& blocks, cudaStream_t s) {
  constexpr int kWarps = kNormThreads / 32;
  const size_t sums = (size_t)kWarps * 2 * G * NV * V * sizeof(float);
  if constexpr (V > 2) {
    constexpr int S = NV > 2 ? 3 : 4;
    const size_t ring = (size_t)kWarps * S * 2 * NV * 32 * 16;
    const size_t smem = ring > sums ? ring : sums;
    auto kernel = norm_bwd_ring_kernel<T, TO, V, NV, G, S>;
    GQ_TRY_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
    blocks = wave(kernel, kNormThreads, smem, blocks);
    kernel<<<blocks, kNormThreads, smem, s>>>(p);
  } else {
    auto kernel = norm_bwd_warp_kernel<T, TO, V, NV, G>;
    blocks = wave(kernel, kNormThreads, sums, blocks);
    kernel<<<blocks, kNormThreads, sums, s>>>(p);
  }
  return launch_status();
}

template <typename T, typename TO, int V, int MAXT, int MINB>
int bwd_wide(const NormBwd& p, int& blocks, int threads, cudaStream_t s) {
  constexpr int S = 3;
  constexpr int kBytes = S * 2 * (kEpt / V) * 16 + kEpt * (int)sizeof(float);  // per thread
  auto kernel = norm_bwd_wide_kernel<T, TO, V, S, MAXT, MINB>;
  GQ_TRY_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, MAXT * kBytes));
  blocks = wave(kernel, threads, threads * kBytes, blocks);
  kernel<<<blocks, threads, threads * kBytes, s>>>(p);
  return launch_status();
}

template <typename T, typename TO, int V, int EPT>
int bwd_block(const NormBwd& p, int& blocks, cudaStream_t s) {
  const int threads = ((p.d + EPT - 1) / EPT + 31) / 32 * 32;
  const size_t smem = (size_t)3 * threads * EPT * sizeof(float);
  auto kernel = norm_bwd_block_kernel<T, TO, V, EPT>;
  GQ_TRY_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   3 * 1024 * EPT * (int)sizeof(float)));
  blocks = wave(kernel, threads, smem, blocks);
  kernel<<<blocks, threads, smem, s>>>(p);
  return launch_status();
}

// `blocks`: at most this many, on return the number launched
template <typename T, typename TO, int V>
int bwd_any(const NormBwd& p, int& blocks, cudaStream_t s) {
  if constexpr (V == 2) {
  } else if constexpr (V == 1) {
    if (p.d <= 64) return bwd_warp<T, TO, 1, 2, 32>(p, blocks, s);
    if (p.d <= 128) return bwd_warp<T, TO, 1, 4, 32>(p, blocks, s);
    if (p.d <= 256) return bwd_warp<T, TO, 1, 8, 32>(p, blocks, s);
    if (p.d <= 384) return bwd_warp<T, TO, 1, 12, 32>(p, blocks, s);
    if (p.d <= 512) return bwd_warp<T, TO, 1, 16, 32>(p, blocks, s);
  } else {
    if (p.d <= 8 * V) return bwd_warp<T, TO, V, 1, 8>(p, blocks, s);
    if (p.d <= 16 * V) return bwd_warp<T, TO, V, 1, 16>(p, blocks, s);
    if (p.d <= 32 * V) return bwd_warp<T, TO, V, 1, 32>(p, blocks, s);
    if (p.d <= 64 * V) return bwd_warp<T, TO, V, 2, 32>(p, blocks, s);
    if constexpr (V == 4)
      if (p.d <= 128 * V) return bwd_warp<T, TO, V, 4, 32>(p, blocks, s);
  }
  if (p.d > 8192) return bwd_block<T, TO, V, 16>(p, blocks, s);
  if constexpr (V > 2) {
    const int threads = wide_threads(p.d);
    if (threads <= kPairThreads) return bwd_wide<T, TO, V, kPairThreads, 2>(p, blocks, threads, s);
    if constexpr (sizeof(T) == 2)
      if (threads <= kPairThreadsDrop && p.dr.on) return bwd_wide<T, TO, V, kPairThreadsDrop, 2>(p, blocks, threads, s);
    return bwd_wide<T, TO, V, 512, 1>(p, blocks, threads, s);
  } else {
    return bwd_block<T, TO, V, 8>(p, blocks, s);
  }
}

template <typename T, typename TO>
int bwd_typed(const NormBwd& p, int& blocks, int vec, cudaStream_t s) {
  if (vec > 2) return bwd_any<T, TO, 16 / sizeof(T)>(p, blocks, s);
  if constexpr (sizeof(T) == 2)
    if (vec == 2 && p.d > kWarpRowMax) return bwd_any<T, TO, 2>(p, blocks, s);
  return bwd_any<T, TO, 1>(p, blocks, s);
}

// Pairs of 16-bit elements only for rows of a block (120,000 x 1,000 bf16, one by
// one at a pitch of 1,001 and in pairs at 1,006: forward 254 and 191 us, backward
// 457 and 276 us); a lane of a warp's row would hold more columns than one by
// one (300,000 x 334: forward 190 -> 273 us, backward 240 -> 963 us).
template <typename T>
int fwd_typed(const NormFwd& p, int vec, cudaStream_t s) {
  if (vec > 2) return fwd_any<T, 16 / sizeof(T)>(p, s);
  if constexpr (sizeof(T) == 2)
    if (vec == 2 && p.d > kWarpRowMax) return fwd_any<T, 2>(p, s);
  return fwd_any<T, 1>(p, s);
}

}  // namespace
}  // namespace gq

using namespace gq;

extern "C" int gq_dropout(const void* X, int type, int64_t n, int d, int64_t ldx, double p, uint64_t seed, void* Y,
                          int64_t ldy, gq_stream stream) {
  Drop dr;
  if (type_bytes(type) == 0 || n < 0 || n > (int64_t)UINT32_MAX || d < 1 || ldx < d || ldy < d)
    return GQ_ERR_INVALID_ARG;
  GQ_TRY(make_drop(p, seed, &dr));
  if (d > kMaxDropWidth) return GQ_ERR_UNSUPPORTED;
  if (n == 0) return GQ_OK;
  if (X == nullptr || Y == nullptr || !aligned(X, type_bytes(type)) || !aligned(Y, type_bytes(type)))
    return GQ_ERR_INVALID_ARG;
  auto s = (cudaStream_t)stream;
  if (type == GQ_F32) return launch_dropout<float>(X, n, d, ldx, dr, Y, ldy, s);
  if (type == GQ_BF16) return launch_dropout<__nv_bfloat16>(X, n, d, ldx, dr, Y, ldy, s);
  return launch_dropout<__half>(X, n, d, ldx, dr, Y, ldy, s);
}

extern "C" int gq_layer_norm_fwd(const void* X, int type, int64_t n, int d, int64_t ldx, const float* gamma,
                                 const float* beta, float eps, int act, double p, uint64_t seed, void* Y, int64_t ldy,
                                 float* mean, float* rstd, uint32_t* relu_bits, int64_t ldrb, gq_stream stream) {
  NormFwd a{};
  if (type_bytes(type) == 0 || n < 0 || n > (int64_t)UINT32_MAX || d < 1 || ldx < d || ldy < d || !(eps >= 0.0f) ||
      std::isinf(eps) || (act != GQ_ACT_NONE && act != GQ_ACT_RELU))
    return GQ_ERR_INVALID_ARG;
  if (relu_bits != nullptr && (act != GQ_ACT_RELU || ldrb < (d + 31) / 32 || !aligned(relu_bits, 4)))
    return GQ_ERR_INVALID_ARG;
  if (!aligned(gamma, 4) || !aligned(beta, 4) || !aligned(mean, 4) || !aligned(rstd, 4)) return GQ_ERR_INVALID_ARG;
  GQ_TRY(make_drop(p, seed, &a.dr));
  if (d > kMaxWidth) return GQ_ERR_UNSUPPORTED;
  if (n == 0) return GQ_OK;
  if (X == nullptr || Y == nullptr || !aligned(X, type_bytes(type)) || !aligned(Y, type_bytes(type)))
    return GQ_ERR_INVALID_ARG;
  a.X = X;
  a.n = n;
  a.ldx = ldx;
  a.d = d;
  a.gamma = gamma;
  a.beta = beta;
  a.eps = eps;
  a.dv = {(float)d, 1.0f / (float)d};
  a.relu = act == GQ_ACT_RELU;
  a.Y = Y;
  a.ldy = ldy;
  a.mean = mean;
  a.rstd = rstd;
  a.bits = relu_bits;
  a.ldrb = ldrb;
  const int vec = vec_of(X, ldx, Y, ldy, type);
  auto s = (cudaStream_t)stream;
  if (type == GQ_F32) return fwd_typed<float>(a, vec, s);
  if (type == GQ_BF16) return fwd_typed<__nv_bfloat16>(a, vec, s);
  return fwd_typed<__half>(a, vec, s);
}

extern "C" size_t gq_layer_norm_bwd_workspace_bytes(int64_t n, int d) {
  if (n < 0 || d < 1 || d > kMaxWidth) return 0;
  return (size_t)bwd_blocks(n, d) * 2 * d * sizeof(float);
}

extern "C" int gq_layer_norm_bwd(const void* dY, int64_t lddy, const void* X, int64_t ldx, int type, int64_t n, int d,
                                 const float* mean, const float* rstd, const float* gamma, int act, double p,
                                 uint64_t seed, const uint32_t* relu_bits, int64_t ldrb, void* dX, int dx_type,
                                 int64_t lddx, float* dgamma, float* dbeta, void* ws, size_t ws_bytes,
                                 gq_stream stream) {
  NormBwd a{};
  if (type_bytes(type) == 0 || (dx_type != type && !(type == GQ_F32 && dx_type == GQ_BF16)) || n < 0 ||
      n > (int64_t)UINT32_MAX || d < 1 || ldx < d || lddy < d || lddx < d ||
      (act != GQ_ACT_NONE && act != GQ_ACT_RELU))
    return GQ_ERR_INVALID_ARG;
  if (act == GQ_ACT_RELU && n > 0 && (relu_bits == nullptr || ldrb < (d + 31) / 32 || !aligned(relu_bits, 4)))
    return GQ_ERR_INVALID_ARG;
  if (!aligned(gamma, 4) || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(dgamma, 4) || !aligned(dbeta, 4))
    return GQ_ERR_INVALID_ARG;
  GQ_TRY(make_drop(p, seed, &a.dr));
  if (d > kMaxWidth) return GQ_ERR_UNSUPPORTED;
  auto s = (cudaStream_t)stream;
  if (n == 0) {  // no rows: the sums are zero
    if (dgamma != nullptr) GQ_TRY_CUDA(cudaMemsetAsync(dgamma, 0, (size_t)d * sizeof(float), s));
    if (dbeta != nullptr) GQ_TRY_CUDA(cudaMemsetAsync(dbeta, 0, (size_t)d * sizeof(float), s));
    return GQ_OK;
  }
  const int esz = type_bytes(type);
  if (dY == nullptr || X == nullptr || dX == nullptr || mean == nullptr || rstd == nullptr || !aligned(dY, esz) ||
      !aligned(X, esz) || !aligned(dX, type_bytes(dx_type)))
    return GQ_ERR_INVALID_ARG;
  const bool sums = dgamma != nullptr || dbeta != nullptr;
  if (sums && (ws == nullptr || ws_bytes < gq_layer_norm_bwd_workspace_bytes(n, d) || !aligned(ws, 4)))
    return GQ_ERR_WORKSPACE;
  a.dY = dY;
  a.X = X;
  a.n = n;
  a.lddy = lddy;
  a.ldx = ldx;
  a.d = d;
  a.dv = {(float)d, 1.0f / (float)d};
  a.mean = mean;
  a.rstd = rstd;
  a.gamma = gamma;
  a.relu = act == GQ_ACT_RELU;
  a.bits = relu_bits;
  a.ldrb = ldrb;
  a.dX = dX;
  a.lddx = lddx;
  a.partial = sums ? static_cast<float*>(ws) : nullptr;
  const int vec = vec_of(X, ldx, dY, lddy, type);
  // a stored vector: as many elements, of dX's type
  a.vec_out = aligned(dX, vec * type_bytes(dx_type)) && lddx % vec == 0;
  int blocks = bwd_blocks(n, d);
  if (type == GQ_F32 && dx_type == GQ_BF16)
    GQ_TRY((bwd_typed<float, __nv_bfloat16>(a, blocks, vec, s)));
  else if (type == GQ_F32)
    GQ_TRY((bwd_typed<float, float>(a, blocks, vec, s)));
  else if (type == GQ_BF16)
    GQ_TRY((bwd_typed<__nv_bfloat16, __nv_bfloat16>(a, blocks, vec, s)));
  else
    GQ_TRY((bwd_typed<__half, __half>(a, blocks, vec, s)));
  if (!sums) return GQ_OK;
  return launch_after(norm_reduce_kernel, dim3((2 * d + 31) / 32), dim3(1024), 0, s, (const float*)a.partial, blocks, d,
                      dgamma, dbeta);
}
