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
// DRAM bound: a row is read once and kept in registers.  Rows of d <= 512
// belong to a group of 8, 16 or 32 lanes (16 elements a lane at most, sums
// by shuffles), wider rows to a thread block (16 elements a thread, sums
// through shared memory).  gamma, beta and the gradient sums of a lane's
// columns stay with the lane over all the rows it visits; the backward's
// column sums are combined per block in a fixed order, written as one
// partial row per block and summed by a second kernel, so results do not
// depend on scheduling.
//
// Dropout draws u(seed, row, column) from the library's counter hash (see
// gq_quantize_pack) and keeps an element when u >= p, so the backward pass
// recomputes the mask from the seed and no mask is stored.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <cstdint>

#include "gq_common.cuh"
#include "gq_internal.cuh"
#include "gq_train.h"

namespace gq {
namespace {

constexpr int kEpt = 16;           // elements of a row per lane or thread
constexpr int kWarpRowMax = 512;   // rows up to here are one warp's (or less)
constexpr int kMaxWidth = 16384;   // 1024 threads x 16 elements
constexpr int kNormThreads = 256;

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

template <int V>
__device__ __forceinline__ void load_param(const float* p, int col, int d, float none, float (&o)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) o[j] = p == nullptr ? none : (col + j < d ? __ldg(p + col + j) : 0.0f);
}

// Dropout: an element is kept when its 23-bit noise code is >= `drop`.
struct Drop {
  uint32_t drop;  // ceil(p 2^23); 0: nothing is dropped and the hash is skipped
  float scale;    // 1 / (1 - p)
  uint32_t key;   // fmix32(low32(seed) ^ high32(seed))
};

__device__ __forceinline__ bool kept(uint32_t krow, int col, uint32_t drop) {
  return (fmix32(krow + (uint32_t)col * 0x9E3779B9u) >> 9) >= drop;
}

// ---------------------------------------------------------------- dropout --
// A block covers rpb rows at a time, tpr threads a row, kDropRows such row
// sets per block, all loaded before the first is used: at 16 bytes a thread
// one load in flight per thread is half of what the memory latency needs.
constexpr int kDropRows = 4;

template <typename T, int V>
__global__ void __launch_bounds__(kNormThreads)
    dropout_kernel(const T* X, int64_t n, int d, int64_t ldx, const Drop dr, T* Y, int64_t ldy, int tpr, int rpb) {
  const int local = (int)threadIdx.x / tpr;
  if (local >= rpb) return;
  const int64_t r0 = (int64_t)blockIdx.x * rpb * kDropRows + local;
  for (int col = ((int)threadIdx.x - local * tpr) * V; col < d; col += tpr * V) {
    float v[kDropRows][V];
#pragma unroll
    for (int u = 0; u < kDropRows; ++u) {
      const int64_t r = r0 + (int64_t)u * rpb;
      if (r < n) load_vec<T, V>(X + r * ldx, col, d, v[u]);
    }
#pragma unroll
    for (int u = 0; u < kDropRows; ++u) {
      const int64_t r = r0 + (int64_t)u * rpb;
      if (r >= n) break;
      const uint32_t kr = row_key(dr.key, (uint32_t)r);
#pragma unroll
      for (int j = 0; j < V; ++j) v[u][j] = kept(kr, col + j, dr.drop) ? v[u][j] * dr.scale : 0.0f;
      store_vec<T, V>(Y + r * ldy, col, d, v[u], true);
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
// complete in every lane of the 32 / V lanes that share it (V = 1: the G
// lanes of the group).
template <int V, int G>
__device__ __forceinline__ uint32_t gather_bits(uint32_t bits, int col) {
  if (V == 1) {
    const uint32_t all = __ballot_sync(FULL, bits);
    return G == 32 ? all : (all >> (threadIdx.x & 31 & ~(G - 1))) & ((1u << (G & 31)) - 1);
  }
  uint32_t w = bits << (col & 31);
#pragma unroll
  for (int o = 1; o < 32 / V; o <<= 1) w |= __shfl_xor_sync(FULL, w, o);
  return w;
}

struct NormFwd {
  const void* X;
  int64_t n, ldx;
  int d;
  const float* gamma;
  const float* beta;
  float eps;
  float fd;  // (float)d; sums are divided by it, so that a constant row's mean is the constant
  int relu;
  Drop dr;
  void* Y;
  int64_t ldy;
  float* mean;
  float* rstd;
  uint32_t* bits;
  int64_t ldrb;
};

// The row's outputs from its centred values xc.  Every lane of the warp
// takes part (the bits are gathered by shuffles); `live` lanes store.
template <typename T, int V, int NV, int G>
__device__ __forceinline__ void norm_emit(const NormFwd& p, int64_t r, bool live, float rstd, int c0, int cstep,
                                          const float (&xc)[NV][V], const float (&ga)[NV][V],
                                          const float (&be)[NV][V]) {
  const uint32_t kr = row_key(p.dr.key, (uint32_t)r);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = c0 + i * cstep;
    float y[V];
    uint32_t pos = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float z = __fmaf_rn(xc[i][j] * rstd, ga[i][j], be[i][j]);
      if (p.relu) {
        const bool on = z > 0.0f;
        pos |= (uint32_t)(on && col + j < p.d) << j;
        z = on ? z : 0.0f;
      }
      if (p.dr.drop != 0) z = kept(kr, col + j, p.dr.drop) ? z * p.dr.scale : 0.0f;
      y[j] = z;
    }
    if (live && col < p.d) store_vec<T, V>(static_cast<T*>(p.Y) + r * p.ldy, col, p.d, y, true);
    if (p.bits != nullptr) {
      const uint32_t w = gather_bits<V, G>(pos, col);
      if (live && (col & 31) == 0 && col < p.d) p.bits[r * p.ldrb + (col >> 5)] = w;
    }
  }
}

// Rows of d <= 512: a group of G lanes per row.
template <typename T, int V, int NV, int G>
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
  for (int64_t rw = warp * kGroups; rw < p.n; rw += step) {
    const int64_t r = rw + sub;
    const bool live = r < p.n;
    const T* x = static_cast<const T*>(p.X) + (live ? r : rw) * p.ldx;
    float v[NV][V];
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      load_vec<T, V>(x, c0 + i * G * V, p.d, v[i]);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) s += v[i][j];
    const float mean = group_sum<G>(s) / p.fd;
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        v[i][j] = c0 + i * G * V + j < p.d ? v[i][j] - mean : 0.0f;
        q = __fmaf_rn(v[i][j], v[i][j], q);
      }
    const float rstd = 1.0f / sqrtf(group_sum<G>(q) / p.fd + p.eps);
    if (live && lane % G == 0) {
      if (p.mean != nullptr) p.mean[r] = mean;
      if (p.rstd != nullptr) p.rstd[r] = rstd;
    }
    norm_emit<T, V, NV, G>(p, r, live, rstd, c0, G * V, v, ga, be);
  }
}

// Wider rows: a block per row, thread t holding columns (i blockDim + t) V.
template <typename T, int V>
__global__ void __launch_bounds__(1024) norm_fwd_block_kernel(const NormFwd p) {
  constexpr int NV = kEpt / V;
  __shared__ float red[2][64];
  const int c0 = (int)threadIdx.x * V, cs = (int)blockDim.x * V;
  int flip = 0;
  for (int64_t r = blockIdx.x; r < p.n; r += gridDim.x) {
    const T* x = static_cast<const T*>(p.X) + r * p.ldx;
    float v[NV][V];
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) load_vec<T, V>(x, c0 + i * cs, p.d, v[i]);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) s += v[i][j];
    const float mean = block_sum2(s, 0.0f, red[flip]).x / p.fd;
    flip ^= 1;
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        v[i][j] = c0 + i * cs + j < p.d ? v[i][j] - mean : 0.0f;
        q = __fmaf_rn(v[i][j], v[i][j], q);
      }
    const float rstd = 1.0f / sqrtf(block_sum2(q, 0.0f, red[flip]).x / p.fd + p.eps);
    flip ^= 1;
    if (threadIdx.x == 0) {
      if (p.mean != nullptr) p.mean[r] = mean;
      if (p.rstd != nullptr) p.rstd[r] = rstd;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {  // one vector at a time: gamma and beta come from L1
      float ga[1][V], be[1][V];
      load_param<V>(p.gamma, c0 + i * cs, p.d, 1.0f, ga[0]);
      load_param<V>(p.beta, c0 + i * cs, p.d, 0.0f, be[0]);
      float one[1][V];
#pragma unroll
      for (int j = 0; j < V; ++j) one[0][j] = v[i][j];
      norm_emit<T, V, 1, 32>(p, r, true, rstd, c0 + i * cs, 0, one, ga, be);
    }
  }
}

// --------------------------------------------------------------- backward --
struct NormBwd {
  const void* dY;
  const void* X;
  int64_t n, lddy, ldx;
  int d;
  float fd;
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

// dz of V columns: the dropout of the forward pass, then its ReLU gate.
template <int V>
__device__ __forceinline__ void gate_dz(const NormBwd& p, int64_t r, uint32_t kr, int col, float (&dz)[V]) {
  if (p.dr.drop != 0) {
#pragma unroll
    for (int j = 0; j < V; ++j) dz[j] = kept(kr, col + j, p.dr.drop) ? dz[j] * p.dr.scale : 0.0f;
  }
  if (p.relu && col < p.d) {
    const uint32_t w = __ldg(p.bits + r * p.ldrb + (col >> 5)) >> (col & 31);
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (((w >> j) & 1u) == 0) dz[j] = 0.0f;
  }
}

template <typename T, typename TO, int V, int NV, int G>
__global__ void __launch_bounds__(kNormThreads) norm_bwd_warp_kernel(const NormBwd p) {
  constexpr int kGroups = 32 / G;
  constexpr int kWarps = kNormThreads / 32;
  extern __shared__ float acc[];  // [warp][2][G * NV * V]
  const int lane = threadIdx.x & 31, sub = lane / G, w = threadIdx.x >> 5;
  const int c0 = (lane % G) * V;
  const int64_t warp = (int64_t)blockIdx.x * kWarps + w;
  const int64_t step = (int64_t)gridDim.x * kWarps * kGroups;
  float ga[NV][V], sg[NV][V], sb[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    load_param<V>(p.gamma, c0 + i * G * V, p.d, 1.0f, ga[i]);
#pragma unroll
    for (int j = 0; j < V; ++j) sg[i][j] = sb[i][j] = 0.0f;
  }
  for (int64_t rw = warp * kGroups; rw < p.n; rw += step) {
    const int64_t r = rw + sub;
    const bool live = r < p.n;
    const int64_t rr = live ? r : rw;
    const T* x = static_cast<const T*>(p.X) + rr * p.ldx;
    const T* dy = static_cast<const T*>(p.dY) + rr * p.lddy;
    float xv[NV][V], dz[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      load_vec<T, V>(x, c0 + i * G * V, p.d, xv[i]);
      load_vec<T, V>(dy, c0 + i * G * V, p.d, dz[i]);
    }
    const float mean = __ldg(p.mean + rr), rstd = __ldg(p.rstd + rr);
    const uint32_t kr = row_key(p.dr.key, (uint32_t)rr);
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      gate_dz<V>(p, rr, kr, c0 + i * G * V, dz[i]);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const bool in = live && c0 + i * G * V + j < p.d;
        const float xh = in ? (xv[i][j] - mean) * rstd : 0.0f;
        const float z = in ? dz[i][j] : 0.0f;
        sg[i][j] = __fmaf_rn(z, xh, sg[i][j]);
        sb[i][j] += z;
        const float g = z * ga[i][j];
        s1 += g;
        s2 = __fmaf_rn(g, xh, s2);
        xv[i][j] = xh;
        dz[i][j] = g;
      }
    }
    const float m1 = group_sum<G>(s1) / p.fd, m2 = group_sum<G>(s2) / p.fd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = c0 + i * G * V;
      float o[V];
#pragma unroll
      for (int j = 0; j < V; ++j) o[j] = rstd * (dz[i][j] - m1 - xv[i][j] * m2);
      if (live && col < p.d) store_vec<TO, V>(static_cast<TO*>(p.dX) + r * p.lddx, col, p.d, o, p.vec_out);
    }
  }
  if (p.partial == nullptr) return;
  constexpr int W = G * NV * V;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float a = sg[i][j], b = sb[i][j];
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

// Wide rows: the block's column sums live in shared memory, each column
// touched by its one owner thread only.
template <typename T, typename TO, int V>
__global__ void __launch_bounds__(1024) norm_bwd_block_kernel(const NormBwd p) {
  constexpr int NV = kEpt / V;
  extern __shared__ float acc[];  // [2][blockDim * kEpt]
  __shared__ float red[2][64];
  const int c0 = (int)threadIdx.x * V, cs = (int)blockDim.x * V;
  const int W = (int)blockDim.x * kEpt;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) acc[c0 + i * cs + j] = acc[W + c0 + i * cs + j] = 0.0f;
  int flip = 0;
  for (int64_t r = blockIdx.x; r < p.n; r += gridDim.x) {
    const T* x = static_cast<const T*>(p.X) + r * p.ldx;
    const T* dy = static_cast<const T*>(p.dY) + r * p.lddy;
    float xv[NV][V], dz[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      load_vec<T, V>(x, c0 + i * cs, p.d, xv[i]);
      load_vec<T, V>(dy, c0 + i * cs, p.d, dz[i]);
    }
    const float mean = __ldg(p.mean + r), rstd = __ldg(p.rstd + r);
    const uint32_t kr = row_key(p.dr.key, (uint32_t)r);
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = c0 + i * cs;
      gate_dz<V>(p, r, kr, col, dz[i]);
      float ga[V];
      load_param<V>(p.gamma, col, p.d, 1.0f, ga);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const bool in = col + j < p.d;
        const float xh = in ? (xv[i][j] - mean) * rstd : 0.0f;
        const float z = in ? dz[i][j] : 0.0f;
        acc[col + j] = __fmaf_rn(z, xh, acc[col + j]);
        acc[W + col + j] += z;
        const float g = z * ga[j];
        s1 += g;
        s2 = __fmaf_rn(g, xh, s2);
        xv[i][j] = xh;
        dz[i][j] = g;
      }
    }
    const float2 s = block_sum2(s1, s2, red[flip]);
    flip ^= 1;
    const float m1 = s.x / p.fd, m2 = s.y / p.fd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = c0 + i * cs;
      float o[V];
#pragma unroll
      for (int j = 0; j < V; ++j) o[j] = rstd * (dz[i][j] - m1 - xv[i][j] * m2);
      if (col < p.d) store_vec<TO, V>(static_cast<TO*>(p.dX) + r * p.lddx, col, p.d, o, p.vec_out);
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

// out[c] = sum over the blocks' partial rows, 32 columns per block, 32 row
// lanes whose sums are added in lane order.
__global__ void __launch_bounds__(1024) norm_reduce_kernel(const float* __restrict__ partial, int blocks, int d,
                                                           float* dgamma, float* dbeta) {
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

// Whether rows of this matrix can be read and written 16 bytes at a time.
bool rows16(const void* p, int64_t ld, int type) { return aligned(p, 16) && ld * type_bytes(type) % 16 == 0; }

int make_drop(double p, uint64_t seed, Drop* d) {
  if (!(p >= 0.0 && p <= 1.0)) return GQ_ERR_INVALID_ARG;
  d->drop = (uint32_t)std::ceil(p * 8388608.0);  // p = 1: above every 23-bit code
  d->scale = p < 1.0 ? (float)(1.0 / (1.0 - p)) : 0.0f;
  d->key = seed_key_host(seed);
  return GQ_OK;
}

int bwd_blocks(int64_t n, int d) {
  // enough blocks to fill the SMs (4 x 256 threads, or about 1024 threads of
  // wide rows, each), and no more partial rows than that
  const int sms = sm_count();
  if (d <= kWarpRowMax) {
    const int64_t want = (n + 7) / 8;
    return (int)(want < 4 * sms ? (want < 1 ? 1 : want) : 4 * sms);
  }
  const int threads = ((d + kEpt - 1) / kEpt + 31) / 32 * 32;
  const int per = threads >= 512 ? (threads > 512 ? 1 : 2) : 1024 / threads;
  const int64_t cap = (int64_t)per * sms;
  return (int)(n < cap ? (n < 1 ? 1 : n) : cap);
}

template <typename T>
int launch_dropout(const void* X, int64_t n, int d, int64_t ldx, const Drop& dr, void* Y, int64_t ldy, bool vec,
                   cudaStream_t s) {
  const int V = vec ? 16 / (int)sizeof(T) : 1;
  const int vpr = (d + V - 1) / V;
  const int passes = (vpr + kNormThreads - 1) / kNormThreads;
  const int tpr = (vpr + passes - 1) / passes;
  const int rpb = kNormThreads / tpr;
  const int64_t blocks = (n + (int64_t)rpb * kDropRows - 1) / ((int64_t)rpb * kDropRows);
  if (blocks > 0x7fffffff) return GQ_ERR_UNSUPPORTED;
  const int threads = (tpr * rpb + 31) / 32 * 32;
  if (vec)
    dropout_kernel<T, 16 / sizeof(T)><<<(unsigned)blocks, threads, 0, s>>>(static_cast<const T*>(X), n, d, ldx, dr,
                                                                          static_cast<T*>(Y), ldy, tpr, rpb);
  else
    dropout_kernel<T, 1><<<(unsigned)blocks, threads, 0, s>>>(static_cast<const T*>(X), n, d, ldx, dr,
                                                             static_cast<T*>(Y), ldy, tpr, rpb);
  return launch_status();
}

template <typename T, int V, int NV, int G>
int fwd_warp(const NormFwd& p, cudaStream_t s) {
  constexpr int rows = kNormThreads / G;
  const int64_t want = (p.n + rows - 1) / rows;
  const int cap = 8 * sm_count();
  norm_fwd_warp_kernel<T, V, NV, G><<<(int)(want < cap ? want : cap), kNormThreads, 0, s>>>(p);
  return launch_status();
}

template <typename T, int V>
int fwd_any(const NormFwd& p, cudaStream_t s) {
  if (p.d <= 8 * V) return fwd_warp<T, V, 1, 8>(p, s);
  if (p.d <= 16 * V) return fwd_warp<T, V, 1, 16>(p, s);
  if (p.d <= 32 * V) return fwd_warp<T, V, 1, 32>(p, s);
  if (p.d <= 64 * V) return fwd_warp<T, V, 2, 32>(p, s);
  if constexpr (V <= 4) {
    if (p.d <= 128 * V) return fwd_warp<T, V, 4, 32>(p, s);
  }
  if constexpr (V == 1) {
    if (p.d <= 512) return fwd_warp<T, V, 16, 32>(p, s);
  }
  const int threads = ((p.d + kEpt - 1) / kEpt + 31) / 32 * 32;
  const int64_t cap = (int64_t)sm_count() * (2048 / threads);
  norm_fwd_block_kernel<T, V><<<(int)(p.n < cap ? p.n : cap), threads, 0, s>>>(p);
  return launch_status();
}

template <typename T, typename TO, int V, int NV, int G>
int bwd_warp(const NormBwd& p, int blocks, cudaStream_t s) {
  const size_t smem = (size_t)(kNormThreads / 32) * 2 * G * NV * V * sizeof(float);
  norm_bwd_warp_kernel<T, TO, V, NV, G><<<blocks, kNormThreads, smem, s>>>(p);
  return launch_status();
}

template <typename T, typename TO, int V>
int bwd_any(const NormBwd& p, int blocks, cudaStream_t s) {
  if (p.d <= 8 * V) return bwd_warp<T, TO, V, 1, 8>(p, blocks, s);
  if (p.d <= 16 * V) return bwd_warp<T, TO, V, 1, 16>(p, blocks, s);
  if (p.d <= 32 * V) return bwd_warp<T, TO, V, 1, 32>(p, blocks, s);
  if (p.d <= 64 * V) return bwd_warp<T, TO, V, 2, 32>(p, blocks, s);
  if constexpr (V <= 4) {
    if (p.d <= 128 * V) return bwd_warp<T, TO, V, 4, 32>(p, blocks, s);
  }
  if constexpr (V == 1) {
    if (p.d <= 512) return bwd_warp<T, TO, V, 16, 32>(p, blocks, s);
  }
  const int threads = ((p.d + kEpt - 1) / kEpt + 31) / 32 * 32;
  const size_t smem = (size_t)2 * threads * kEpt * sizeof(float);
  GQ_TRY_CUDA(cudaFuncSetAttribute(norm_bwd_block_kernel<T, TO, V>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   2 * kMaxWidth * (int)sizeof(float)));
  norm_bwd_block_kernel<T, TO, V><<<blocks, threads, smem, s>>>(p);
  return launch_status();
}

template <typename T, typename TO>
int bwd_typed(const NormBwd& p, int blocks, bool vec, cudaStream_t s) {
  return vec ? bwd_any<T, TO, 16 / sizeof(T)>(p, blocks, s) : bwd_any<T, TO, 1>(p, blocks, s);
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
  if (n == 0) return GQ_OK;
  if (X == nullptr || Y == nullptr || !aligned(X, type_bytes(type)) || !aligned(Y, type_bytes(type)))
    return GQ_ERR_INVALID_ARG;
  const bool vec = rows16(X, ldx, type) && rows16(Y, ldy, type);
  auto s = (cudaStream_t)stream;
  if (type == GQ_F32) return launch_dropout<float>(X, n, d, ldx, dr, Y, ldy, vec, s);
  if (type == GQ_BF16) return launch_dropout<__nv_bfloat16>(X, n, d, ldx, dr, Y, ldy, vec, s);
  return launch_dropout<__half>(X, n, d, ldx, dr, Y, ldy, vec, s);
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
  a.fd = (float)d;
  a.relu = act == GQ_ACT_RELU;
  a.Y = Y;
  a.ldy = ldy;
  a.mean = mean;
  a.rstd = rstd;
  a.bits = relu_bits;
  a.ldrb = ldrb;
  const bool vec = rows16(X, ldx, type) && rows16(Y, ldy, type);
  auto s = (cudaStream_t)stream;
  if (type == GQ_F32) return vec ? fwd_any<float, 4>(a, s) : fwd_any<float, 1>(a, s);
  if (type == GQ_BF16) return vec ? fwd_any<__nv_bfloat16, 8>(a, s) : fwd_any<__nv_bfloat16, 1>(a, s);
  return vec ? fwd_any<__half, 8>(a, s) : fwd_any<__half, 1>(a, s);
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
  a.fd = (float)d;
  a.mean = mean;
  a.rstd = rstd;
  a.gamma = gamma;
  a.relu = act == GQ_ACT_RELU;
  a.bits = relu_bits;
  a.ldrb = ldrb;
  a.dX = dX;
  a.lddx = lddx;
  a.partial = sums ? static_cast<float*>(ws) : nullptr;
  const bool vec = rows16(X, ldx, type) && rows16(dY, lddy, type);
  // bytes of one stored vector: 16 in the inputs' type, 8 for fp32 -> bf16
  const int ob = type_bytes(dx_type) * 16 / esz;
  a.vec_out = aligned(dX, ob) && lddx * type_bytes(dx_type) % ob == 0;
  const int blocks = bwd_blocks(n, d);
  if (type == GQ_F32 && dx_type == GQ_BF16)
    GQ_TRY((bwd_typed<float, __nv_bfloat16>(a, blocks, vec, s)));
  else if (type == GQ_F32)
    GQ_TRY((bwd_typed<float, float>(a, blocks, vec, s)));
  else if (type == GQ_BF16)
    GQ_TRY((bwd_typed<__nv_bfloat16, __nv_bfloat16>(a, blocks, vec, s)));
  else
    GQ_TRY((bwd_typed<__half, __half>(a, blocks, vec, s)));
  if (!sums) return GQ_OK;
  norm_reduce_kernel<<<(2 * d + 31) / 32, 1024, 0, s>>>(a.partial, blocks, d, dgamma, dbeta);
  return launch_status();
}
