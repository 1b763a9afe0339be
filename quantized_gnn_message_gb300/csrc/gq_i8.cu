// gq_i8.cu -- products of 8-bit integers with a scale for each row of both
// operands, and the quantizers that make them.
//
//   s[i] = max_k |x[i,k]| / 127,   q[i,k] = round(x[i,k] / s[i])
//   C[i,j] = act(sa[i] sb[j] sum_k a[i,k] b[j,k] + bias[j])
//
// (Tango Sec. 3.2 quantizes both operands of the update's products.)  The sum of
// products is exact.  This GPU's 8-bit integer tensor rate is about a 25th of
// its bf16 rate, so the integers are multiplied on the fp16 path: every
// 8-bit integer is an fp16 number, a product of two needs 15 bits and a sum of
// 1,024 of them 24, so an fp32 accumulator holds it exactly; accumulators are
// drained into 32-bit integers every 1,024 products, and partial sums of a split
// contraction are added as 64-bit integers.
//
// Tile product: a pair of CTAs (cta_group::2) takes 256 rows of one operand, S,
// and up to 256 of the other, F.  Per step of 64 products in each CTA
//   warp 0   copies its 128 rows of S and its half of F's as fp16 (TMA, a ring
//            of 5 stages of 32 KB),
//   warp 1   issues tcgen05.mma (even CTA),
//   the last eight warps are the epilogue: TMEM -> registers -> scales, bias,
//            activation -> shared memory -> rows of C, while the next tile's
//            products run.
// A step takes 632 cycles, of which the products are 512: 16,384 x 65,536 x
// 1,024 in 1.26 ms, 1.75 PFLOP/s, where the chip holds about 1.72 for long;
// 8,192 cubed, codes widened before and sums drained eight times, 0.66 ms.
// Where S comes as bytes and meets few rows of F, eight more warps widen
// it: bytes cross DRAM and L2, fp16 shared memory only (2,449,029 x 256 codes by
// 256 x 256: 0.61 ms, 5.1 TB/s).  Four bytes become four fp16 in five
// instructions: x ^ 0x80 is x + 128; put under the byte 0x64 it is the fp16 number
// 1024 + 128 + x, and one packed subtraction of 1152 leaves x.
// Rows in full precision of up to 256 values are quantized by such warps on the
// way (2,449,029 x 256 fp32 -> 256: 0.97 ms instead of 0.45 + 0.61).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include <climits>
#include <cmath>
#include <type_traits>

#include "gq_common.cuh"
#include "gq_internal.cuh"
#include "gq_sm100.cuh"
#include "gq_train.h"

namespace gq {
namespace {

// ------------------------------------------------------------- PTX helpers --
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t mapa(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// Arrival on a barrier of either CTA, released at CTA scope, which costs no
// memory barrier.  That will do for an accumulator that has been read
// (tcgen05.wait::ld before it), and for shared memory that was written for the
// tensor cores: it is this CTA's own, read by this SM, written and fenced towards
// the asynchronous proxy before the arrival; what crosses is the barrier alone.
// (With a release at cluster scope a step took 1,380 cycles instead of 630.)
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_alloc2(uint32_t* dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc2(uint32_t taddr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols) : "memory");
}
// a box into this CTA's shared memory, its bytes counted on a barrier of the even CTA
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void umma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n"
      "  .reg .pred p;\n"
      "  setp.ne.b32 p, %4, 0;\n"
      "  tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n"
      "}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// arrives on `bar` of both CTAs once the MMAs issued so far are done
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
// 32 lanes x 32 consecutive columns of TMEM
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&u)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
        "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
        "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
        "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
      : "r"(taddr)
      : "memory");
}
// Bounded wait on a barrier phase, the thread suspended in hardware meanwhile.
// False after the limit, or once another role of the CTA has given up.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort, int* err, int where) {
  const uint32_t b = smem_u32(bar);
  if (mbar_try_wait_u32(b, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait_u32(b, parity)) {
    if (*abort) return false;
    if (clock64() - t0 > kWaitCycles) {
      *abort = 1;
      if (err != nullptr) atomicCAS(err, 0, where);
      return false;
    }
  }
  return true;
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// ------------------------------------------------------------------- types --
// Stores one value of the output type chosen at run time.
__device__ __forceinline__ void store_as(void* base, int64_t i, float x, int type) {
  if (type == GQ_F32)
    static_cast<float*>(base)[i] = x;
  else if (type == GQ_BF16)
    static_cast<__nv_bfloat16*>(base)[i] = __float2bfloat16_rn(x);
  else
    static_cast<__half*>(base)[i] = __float2half_rn(x);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi, int type) {
  if (type == GQ_BF16) return pack_bf16x2(lo, hi);
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// ReLU as the other operators have it: 0 for a NaN
__device__ __forceinline__ float activate(float y, int relu) { return relu ? fmaxf(y, 0.0f) : y; }

// ------------------------------------------------------------- quantization --
// A row's scale is its largest magnitude / 127; a row that holds a NaN or an
// infinity has that scale not finite and codes 0, so that its products are NaN
// as the row's own would be.  Below kTiny a row counts as zero: the
// quotients' arithmetic needs a normal scale.
constexpr float kTiny = 7.888609052210118e-31f;  // 2^-100

struct Scale {
  float s, inv, half;    // inv = 0: the codes are 0
};
__device__ __forceinline__ Scale make_scale(uint32_t bits) {
  const float top = __uint_as_float(bits);
  const bool use = top < INFINITY && top >= kTiny;  // not for a NaN
  const float s = __fdiv_rn(use ? top : 127.0f, 127.0f), inv = __fdiv_rn(1.0f, s);
  Scale r;
  r.s = use ? s : top < kTiny ? 0.0f : __int_as_float(0x7fc00000);
  r.inv = use ? inv : 0.0f;
  r.half = use ? 0.5f * s : 0.0f;
  return r;
}
// round(x / s), ties to even, exactly: q within one of it from the reciprocal,
// then by the remainder x - q s, which a fused multiply-add gives exactly
// (it is a multiple of half a step of s and no larger than s).  q comes by adding
// 1.5 2^23: conversions and roundings go through the special function unit at
// an eighth of the speed.  Four values have one branch for the rare remainder.
constexpr float kMagic = 12582912.0f;
__device__ __forceinline__ float4 quantize4(const float4& x, const Scale& c) {
  const float2 inv = make_float2(c.inv, c.inv), s = make_float2(-c.s, -c.s);
  const float2 up = make_float2(kMagic, kMagic), down = make_float2(-kMagic, -kMagic);
  const float2 xa = make_float2(x.x, x.y), xb = make_float2(x.z, x.w);
  float2 a = add2(fma2(xa, inv, up), down), b = add2(fma2(xb, inv, up), down);
  const float2 ra = fma2(a, s, xa), rb = fma2(b, s, xb);
  const float far = fmaxf(fmaxf(fabsf(ra.x), fabsf(ra.y)), fmaxf(fabsf(rb.x), fabsf(rb.y)));
  if (far >= c.half && c.inv > 0.0f) {  // rare
    auto fix = [&](float q, float r) {
      const bool odd = __float_as_uint(q + kMagic) & 1;
      return fabsf(r) > c.half || (fabsf(r) == c.half && odd) ? q + (r > 0.0f ? 1.0f : -1.0f) : q;
    };
    a = make_float2(fix(a.x, ra.x), fix(a.y, ra.y));
    b = make_float2(fix(b.x, rb.x), fix(b.y, rb.y));
  }
  if (!(c.inv > 0.0f)) a = b = make_float2(0.0f, 0.0f);
  return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ uint32_t code(float q) { return __float_as_uint(q + kMagic); }  // in the low byte
__device__ __forceinline__ uint32_t bytes4(const float4& q) {
  return __byte_perm(__byte_perm(code(q.x), code(q.y), 0x0040), __byte_perm(code(q.z), code(q.w), 0x0040), 0x5410);
}
__device__ __forceinline__ uint2 halves4(const float4& q) {
  const __half2 a = __floats2half2_rn(q.x, q.y), b = __floats2half2_rn(q.z, q.w);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ float quantize1(float x, const Scale& c) {
  return quantize4(make_float4(x, 0.0f, 0.0f, 0.0f), c).x;
}
// 4 bytes -> 4 fp16
__device__ __forceinline__ void widen(uint32_t w, uint32_t& lo, uint32_t& hi) {
  w ^= 0x80808080u;
  const uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
  const __half2 k = __half2half2(__ushort_as_half(0x6480));  // 1152
  const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), k);
  const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), k);
  lo = *reinterpret_cast<const uint32_t*>(&x);
  hi = *reinterpret_cast<const uint32_t*>(&y);
}
// four codes (from floats, or from a word of bytes) and one
__device__ __forceinline__ void put4(int8_t* o, const float4& q) { *reinterpret_cast<uint32_t*>(o) = bytes4(q); }
__device__ __forceinline__ void put4(__half* o, const float4& q) { *reinterpret_cast<uint2*>(o) = halves4(q); }
__device__ __forceinline__ void put4(int8_t* o, uint32_t w) { *reinterpret_cast<uint32_t*>(o) = w; }
__device__ __forceinline__ void put4(__half* o, uint32_t w) {
  uint2 h;
  widen(w, h.x, h.y);
  *reinterpret_cast<uint2*>(o) = h;
}
__device__ __forceinline__ void put1(int8_t* o, float q) { *o = (int8_t)code(q); }
__device__ __forceinline__ void put1(__half* o, float q) { *o = __float2half_rn(q); }
__device__ __forceinline__ uint32_t mag(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// 4 consecutive values of a row
template <typename T>
__device__ __forceinline__ float4 load4(const T* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p) { return *reinterpret_cast<const float4*>(p); }
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xffff0000u));
}
template <>
__device__ __forceinline__ float4 load4<__half>(const __half* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&w.x));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
  return make_float4(a.x, a.y, b.x, b.y);
}

constexpr int kQThreads = 256;

// Rows of up to 128 NV columns that start aligned for four: a warp a row, which it
// holds in registers.
template <typename T, typename O, int NV>
__global__ void __launch_bounds__(kQThreads)
    quant_short_rows_kernel(const T* X, int64_t n, int d, int64_t ldx, O* Q, int64_t ldq, float* S) {
  grid_wait();
  const int lane = threadIdx.x & 31;
  const int64_t r = (int64_t)blockIdx.x * (kQThreads / 32) + (threadIdx.x >> 5);
  if (r >= n) return;
  const T* x = X + r * ldx;
  float4 v[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = i * 128 + lane * 4;
    if (c + 4 <= d)
      v[i] = load4<T>(x + c);
    else
      v[i] = make_float4(c < d ? (float)x[c] : 0.0f, c + 1 < d ? (float)x[c + 1] : 0.0f, c + 2 < d ? (float)x[c + 2] : 0.0f,
                         0.0f);
  }
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) top = max(max(top, mag(v[i].x)), max(mag(v[i].y), max(mag(v[i].z), mag(v[i].w))));
  const Scale c = make_scale(__reduce_max_sync(FULL, top));
  if (lane == 0) S[r] = c.s;
  O* q = Q + r * ldq;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int at = i * 128 + lane * 4;  // ldq is a multiple of 16: the last four may reach behind d
    if (at < d)
      put4(q + at, quantize4(v[i], c));
  }
}

// Other rows: LANES threads a row (a warp up to 4,096 columns, else the block),
// the row read twice, the second time from L1 or L2.
template <typename T, typename O, bool VEC, int LANES>
__global__ void __launch_bounds__(kQThreads)
    quant_rows_kernel(const T* X, int64_t n, int d, int64_t ldx, O* Q, int64_t ldq, float* S) {
  __shared__ uint32_t smax[kQThreads / 32];
  grid_wait();
  const int lane = threadIdx.x % LANES;
  const int64_t r = (int64_t)blockIdx.x * (kQThreads / LANES) + threadIdx.x / LANES;
  const bool live = r < n;
  const T* x = X + (live ? r : 0) * ldx;
  const int d4 = d & ~3;
  uint32_t top = 0;
  if (live) {
    if (VEC) {
#pragma unroll 4
      for (int c = lane * 4; c < d4; c += LANES * 4) {
        const float4 v = load4<T>(x + c);
        top = max(max(top, mag(v.x)), max(mag(v.y), max(mag(v.z), mag(v.w))));
      }
      if (d4 + lane < d) top = max(top, mag((float)x[d4 + lane]));
    } else {
#pragma unroll 8
      for (int c = lane; c < d; c += LANES) top = max(top, mag((float)x[c]));
    }
  }
  top = __reduce_max_sync(FULL, top);
  if (LANES > 32) {
    if ((threadIdx.x & 31) == 0) smax[threadIdx.x >> 5] = top;
    __syncthreads();
    top = smax[0];
    for (int w = 1; w < LANES / 32; ++w) top = max(top, smax[w]);
  }
  if (!live) return;
  const Scale c = make_scale(top);
  if (lane == 0) S[r] = c.s;
  O* q = Q + r * ldq;
  if (VEC) {
#pragma unroll 4
    for (int k = lane * 4; k < d4; k += LANES * 4) {
      const float4 v = load4<T>(x + k);
      put4(q + k, quantize4(v, c));
    }
    if (d4 + lane < d) put1(q + d4 + lane, quantize1((float)x[d4 + lane], c));
  } else {
#pragma unroll 8
    for (int k = lane; k < d; k += LANES) put1(q + k, quantize1((float)x[k], c));
  }
}

// Columns.  First the largest magnitude of each column's pieces and, where asked
// for, their sums: a block takes kColW columns (a thread four of them) and one
// piece of the rows.
constexpr int kColW = 64, kColRows = kQThreads / (kColW / 4), kMaxParts = 128;
template <typename T>
__device__ __forceinline__ float4 load_cols(const T* x, int left, int vec) {  // `left` columns are there
  if (vec && left >= 4) return load4<T>(x);
  return make_float4(left > 0 ? (float)x[0] : 0.0f, left > 1 ? (float)x[1] : 0.0f, left > 2 ? (float)x[2] : 0.0f,
                     left > 3 ? (float)x[3] : 0.0f);
}
// One matrix; two of them share the launches of the backward pass.
template <typename T, typename O>
struct ColJob {
  const T* X;
  int64_t n;
  int d;
  int64_t ldx;
  int vec;               // rows start aligned for four values
  int parts;
  int64_t rows_per;
  uint32_t* top;         // [parts][d]
  float* sums;           // [parts][d], or null
  O* Q;
  int64_t ldq;
  float* S;
  float* colsum;
};
template <typename T, typename O>
struct ColJobs {
  ColJob<T, O> of[2];
};

template <typename T, typename O>
__global__ void __launch_bounds__(kQThreads) col_max_kernel(const __grid_constant__ ColJobs<T, O> jobs) {
  const ColJob<T, O>& p = jobs.of[blockIdx.z];
  const T* X = p.X;
  const int64_t n = p.n, ldx = p.ldx, rows_per = p.rows_per;
  const int d = p.d, vec = p.vec;
  if ((int)blockIdx.x * kColW >= d || (int)blockIdx.y >= p.parts) return;
  __shared__ uint32_t st[kColRows][kColW];
  __shared__ float ss[kColRows][kColW];
  grid_wait();
  const int cv = threadIdx.x % (kColW / 4), ry = threadIdx.x / (kColW / 4);
  const int c = blockIdx.x * kColW + 4 * cv;
  const int64_t r1 = min(n, (blockIdx.y + 1) * rows_per);
  uint32_t m[4] = {0, 0, 0, 0};
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  constexpr int U = 8;
  for (int64_t r = blockIdx.y * rows_per + ry; r < r1; r += U * kColRows) {
    float4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      v[u] = load_cols<T>(X + (r + u * kColRows) * ldx + c, r + u * kColRows < r1 ? d - c : 0, vec);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      m[0] = max(m[0], mag(v[u].x));
      m[1] = max(m[1], mag(v[u].y));
      m[2] = max(m[2], mag(v[u].z));
      m[3] = max(m[3], mag(v[u].w));
      s[0] += v[u].x;
      s[1] += v[u].y;
      s[2] += v[u].z;
      s[3] += v[u].w;
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    st[ry][4 * cv + k] = m[k];
    ss[ry][4 * cv + k] = s[k];
  }
  __syncthreads();
  const int x = threadIdx.x, col = blockIdx.x * kColW + x;
  if (x < kColW && col < d) {
    uint32_t a = 0;
    float b = 0.0f;
#pragma unroll
    for (int k = 0; k < kColRows; ++k) {
      a = max(a, st[k][x]);
      b += ss[k][x];
    }
    p.top[(int64_t)blockIdx.y * d + col] = a;
    if (p.sums != nullptr) p.sums[(int64_t)blockIdx.y * d + col] = b;
  }
}

// Then the pieces' largest (by every block for its 64 columns) and the sums (by one,
// with what the additions lose) together, and tiles of 128 rows turned into 64 rows of 128 codes.
constexpr int kTrRows = 128, kTrPitch = kTrRows / 4 + 1;  // words
template <typename T, typename O>
__global__ void __launch_bounds__(kQThreads) quant_cols_kernel(const __grid_constant__ ColJobs<T, O> jobs) {
  const ColJob<T, O>& p = jobs.of[blockIdx.z];
  const T* X = p.X;
  const int64_t n = p.n, ldx = p.ldx, ldq = p.ldq;
  const int d = p.d, vec = p.vec, parts = p.parts;
  const float* sums = p.sums;
  O* Q = p.Q;
  const int64_t tiles = (n + kTrRows - 1) / kTrRows;
  if ((int)blockIdx.y * kColW >= d || (int64_t)blockIdx.x >= tiles) return;
  __shared__ uint32_t tile[kColW][kTrPitch];
  __shared__ uint32_t smax[4][kColW];
  __shared__ Sum2 ssum[4][kColW];
  __shared__ Scale sc[kColW];
  grid_wait();
  const int t = threadIdx.x, c0 = blockIdx.y * kColW;
  {
    const int x = t % kColW, y = t / kColW;
    uint32_t m = 0;
    Sum2 s{};
    if (c0 + x < d)
#pragma unroll 8
      for (int k = y; k < parts; k += 4) {
        m = max(m, p.top[(int64_t)k * d + c0 + x]);
        if (sums != nullptr && blockIdx.x == 0) s.add(sums[(int64_t)k * d + c0 + x]);
      }
    smax[y][x] = m;
    ssum[y][x] = s;
    __syncthreads();
    if (t < kColW) {
      sc[t] = make_scale(max(max(smax[0][t], smax[1][t]), max(smax[2][t], smax[3][t])));
      if (blockIdx.x == 0 && c0 + t < d) {
        p.S[c0 + t] = sc[t].s;
        if (sums != nullptr) {
          Sum2 all = ssum[0][t];
          for (int k = 1; k < 4; ++k) all.add(ssum[k][t]);
          p.colsum[c0 + t] = all.value();
        }
      }
    }
    __syncthreads();
  }
  const int cv = t % 16, rg = t / 16;  // four columns, four rows
  const int left = d - c0 - 4 * cv;
  for (int64_t k = blockIdx.x; k < tiles; k += gridDim.x) {
    const int64_t r0 = k * kTrRows;
    float4 v[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t r = r0 + (rg + 16 * h) * 4 + j;
        v[h][j] = load_cols<T>(X + r * ldx + c0 + 4 * cv, r < n ? left : 0, vec);
      }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t* o = &tile[4 * cv][rg + 16 * h];
      const Scale a = sc[4 * cv], b = sc[4 * cv + 1], c = sc[4 * cv + 2], e = sc[4 * cv + 3];
      o[0] = bytes4(quantize4(make_float4(v[h][0].x, v[h][1].x, v[h][2].x, v[h][3].x), a));
      o[kTrPitch] = bytes4(quantize4(make_float4(v[h][0].y, v[h][1].y, v[h][2].y, v[h][3].y), b));
      o[2 * kTrPitch] = bytes4(quantize4(make_float4(v[h][0].z, v[h][1].z, v[h][2].z, v[h][3].z), c));
      o[3 * kTrPitch] = bytes4(quantize4(make_float4(v[h][0].w, v[h][1].w, v[h][2].w, v[h][3].w), e));
    }
    __syncthreads();
    // rows of Q are a multiple of 16 codes: those past n are written as 0
    for (int i = t; i < kColW * (kTrRows / 4); i += kQThreads) {
      const int row = i / (kTrRows / 4), w = i % (kTrRows / 4);
      if (c0 + row < d && r0 + 4 * w < n) put4(Q + (int64_t)(c0 + row) * ldq + r0 + 4 * w, tile[row][w]);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------- tile product --
constexpr int kConvWarps = 8, kTeams = 2, kTeamWarps = kConvWarps / kTeams, kEpiWarps = 8;
constexpr int kTile = 256;                 // rows of S a pair, at most as many of F
constexpr int kStep = 64;                  // products of a step
constexpr int kDrain = 16;                 // steps after which an accumulator is drained: 1,024 products
constexpr int kSBytes = 128 * kStep * 2;   // a CTA's half of S in a stage, F's at most as much
constexpr int kStage = 2 * kSBytes;
constexpr int kBytes8 = 128 * kStep;       // S as bytes
constexpr int kStgPitch = 36;              // floats: 32 columns and a shift of 4 banks a row
constexpr int kStg = 32 * kStgPitch * 4;
constexpr int kColVec = 2 * 128 * 4;        // an epilogue warp's columns: scales | biases
constexpr long long kDrainCycles = 4000000;
constexpr int64_t kMaxSplitSteps = 1024;   // 65,536 products: a 32-bit sum holds twice that

// CONV: S arrives as bytes and is widened in the kernel.
template <bool CONV>
struct Shape {
  static constexpr int threads = CONV ? 640 : 384;
  static constexpr int epi0 = threads / 32 - kEpiWarps;  // first epilogue warp
  static constexpr int ring = CONV ? 4 : 5;
  static constexpr int ring8 = CONV ? 6 : 0;
  static constexpr int smem = 1024 + ring * kStage + ring8 * kBytes8 + kEpiWarps * (kStg + kColVec) + 512;
};
static_assert(Shape<true>::ring % kTeams == 0 && Shape<true>::ring8 % kTeams == 0, "a team meets every other stage");

struct TileArgs {
  int64_t M, N;                            // rows of S and F
  int steps, NT, half;                     // F rows of a tile; the epilogue's first column half
  int64_t tm, tn, units;
  int splits, split_steps;
  void* C;
  int64_t ldc;
  int type, relu, swap, vec;               // swap: C[f][s] instead of C[s][f]
  const float* sS;
  const float* sF;
  const float* bias;                       // of F's rows; with swap of S's
  int* part;                               // split sums [split][M][ldp]
  int64_t ldp;
  int* err;
};

struct Unit {
  int64_t mt, nt;
  int split, s0, s1;
};

// Groups of 8 tiles of S share F's tiles: their rows stay in L2 while F streams.
__device__ __forceinline__ Unit get_unit(const TileArgs& p, int64_t u) {
  Unit r;
  const int64_t tiles = p.tm * p.tn;
  r.split = (int)(u / tiles);
  const int64_t t = u - r.split * tiles;
  const int64_t g = t / (8 * p.tn), in = t - g * 8 * p.tn;
  const int64_t gm = min((int64_t)8, p.tm - g * 8);
  r.nt = in / gm;
  r.mt = g * 8 + in - r.nt * gm;
  r.s0 = r.split * p.split_steps;
  r.s1 = min(p.steps, r.s0 + p.split_steps);
  return r;
}

// chunk i of 16 bytes of a [rows][64] byte tile into a [rows][64] fp16 tile, 128-byte swizzle
__device__ __forceinline__ void widen_chunk(uint4 w, uint8_t* dst, int i) {
  uint4 a, b;
  widen(w.x, a.x, a.y);
  widen(w.y, a.z, a.w);
  widen(w.z, b.x, b.y);
  widen(w.w, b.z, b.w);
  const int row = i >> 2, piece = (i & 3) * 2, x = row & 7;
  *reinterpret_cast<uint4*>(dst + row * 128 + ((piece ^ x) << 4)) = a;
  *reinterpret_cast<uint4*>(dst + row * 128 + (((piece + 1) ^ x) << 4)) = b;
}

// 32 rows x 32 columns of sums, lane = row, the tile's columns col0..  cv: the
// columns' scales, and 128 floats on their biases.  SWAP: C may be transposed.
// The warp leaves together: its next access to TMEM is one for all lanes.
template <bool SWAP>
__device__ __forceinline__ void put(const TileArgs& p, int64_t row0, int64_t col0, const float (&v)[32], float sr, float br,
                                    const float* cv, float* stg, int lane) {
  if (SWAP && p.swap) {  // a lane's row is a column of C: lanes write side by side
    const int64_t row = row0 + lane;
    if (row < p.M) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (col0 + j < p.N)
          store_as(p.C, (col0 + j) * p.ldc + row, activate(fmaf(__fmul_rn(v[j], cv[j]), sr, br), p.relu), p.type);
    }
    __syncwarp();
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    *reinterpret_cast<float4*>(stg + lane * kStgPitch + 4 * j) =
        make_float4(v[4 * j] * sr, v[4 * j + 1] * sr, v[4 * j + 2] * sr, v[4 * j + 3] * sr);
  __syncwarp();
  const int rows = (int)min((int64_t)32, p.M - row0);
  if (p.vec && col0 + 32 <= p.N) {
    if (p.type == GQ_F32) {
      const int c = (lane & 7) * 4;
      const float4 sf = *reinterpret_cast<const float4*>(cv + c), b = *reinterpret_cast<const float4*>(cv + 128 + c);
      float* out = static_cast<float*>(p.C) + (row0 + (lane >> 3)) * p.ldc + col0 + c;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int rr = 4 * k + (lane >> 3);
        const float4 x = *reinterpret_cast<const float4*>(stg + rr * kStgPitch + c);
        if (rr < rows)
          st_f4(out, activate(fmaf(x.x, sf.x, b.x), p.relu), activate(fmaf(x.y, sf.y, b.y), p.relu),
                activate(fmaf(x.z, sf.z, b.z), p.relu), activate(fmaf(x.w, sf.w, b.w), p.relu));
        out += 4 * p.ldc;
      }
    } else {
      const int c = (lane & 3) * 8;
      const float4 s0 = *reinterpret_cast<const float4*>(cv + c), s1 = *reinterpret_cast<const float4*>(cv + c + 4);
      const float4 b0 = *reinterpret_cast<const float4*>(cv + 128 + c);
      const float4 b1 = *reinterpret_cast<const float4*>(cv + 132 + c);
      uint16_t* out = static_cast<uint16_t*>(p.C) + (row0 + (lane >> 2)) * p.ldc + col0 + c;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int rr = 8 * k + (lane >> 2);
        const float4 x = *reinterpret_cast<const float4*>(stg + rr * kStgPitch + c);
        const float4 z = *reinterpret_cast<const float4*>(stg + rr * kStgPitch + c + 4);
        const uint32_t w0 = pack2(activate(fmaf(x.x, s0.x, b0.x), p.relu), activate(fmaf(x.y, s0.y, b0.y), p.relu), p.type);
        const uint32_t w1 = pack2(activate(fmaf(x.z, s0.z, b0.z), p.relu), activate(fmaf(x.w, s0.w, b0.w), p.relu), p.type);
        const uint32_t w2 = pack2(activate(fmaf(z.x, s1.x, b1.x), p.relu), activate(fmaf(z.y, s1.y, b1.y), p.relu), p.type);
        const uint32_t w3 = pack2(activate(fmaf(z.z, s1.z, b1.z), p.relu), activate(fmaf(z.w, s1.w, b1.w), p.relu), p.type);
        if (rr < rows) *reinterpret_cast<uint4*>(out) = make_uint4(w0, w1, w2, w3);
        out += 8 * p.ldc;
      }
    }
  } else if (rows > 0 && col0 + lane < p.N) {
    const float sf = cv[lane], b = cv[128 + lane];
    for (int rr = 0; rr < rows; ++rr)
      store_as(p.C, (row0 + rr) * p.ldc + col0 + lane, activate(fmaf(stg[rr * kStgPitch + lane], sf, b), p.relu), p.type);
  }
  __syncwarp();
}

// the same of a split's sums, unscaled
__device__ __forceinline__ void put_part(const TileArgs& p, const Unit& u, int64_t row0, int64_t col0, const int (&v)[32],
                                         float* stg, int lane) {
  int* s = reinterpret_cast<int*>(stg);
#pragma unroll
  for (int j = 0; j < 8; ++j)
    *reinterpret_cast<int4*>(s + lane * kStgPitch + 4 * j) = make_int4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
  __syncwarp();
  const int64_t col = col0 + (lane & 7) * 4;
  int* out = p.part + ((int64_t)u.split * p.M + row0 + (lane >> 3)) * p.ldp + col;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int rr = 4 * k + (lane >> 3);
    if (row0 + rr < p.M && col < p.ldp)
      *reinterpret_cast<int4*>(out) = *reinterpret_cast<const int4*>(s + rr * kStgPitch + (lane & 7) * 4);
    out += 4 * p.ldp;
  }
  __syncwarp();
}

// MULTI: a unit's sum takes several accumulators, or is a part of a split one's.
template <bool CONV, bool MULTI>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Shape<CONV>::threads, 1)
    i8_tiles_kernel(const __grid_constant__ CUtensorMap mS, const __grid_constant__ CUtensorMap mF, const TileArgs p) {
  using Z = Shape<CONV>;
  constexpr int R = Z::ring, R8 = CONV ? Z::ring8 : 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* s16 = smem;
  uint8_t* s8 = s16 + R * kStage;
  float* stg_all = reinterpret_cast<float*>(s8 + Z::ring8 * kBytes8);
  uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(stg_all) + kEpiWarps * (kStg + kColVec));
  uint64_t* empty = full + R;
  uint64_t* tfull = empty + R;
  uint64_t* tempty = tfull + 2;
  uint64_t* full8 = tempty + 2;
  uint64_t* empty8 = full8 + R8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(empty8 + R8);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t cr = cluster_rank();
  if (threadIdx.x == 0) {
    for (int s = 0; s < R; ++s) {
      mbar_init(&full[s], CONV ? 1 + 2 * kTeamWarps : 1);  // TMA's bytes, and both CTAs' widening warps
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < R8; ++s) {
      mbar_init(&full8[s], 1);
      mbar_init(&empty8[s], kTeamWarps);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 2 * kEpiWarps);
    }
    *abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc2(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_wait();
  const int64_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int hn = p.NT / 2;

  // With CONV 3 warpgroups at 48 registers and 2 at 168: the 61,440 (96 a
  // thread) that the block is launched with.
  if (warp < 4) {
    if constexpr (CONV) regs_down<48>();
    if (warp == 0 && lane == 0) {  // fp16 operands: F, and S where it is not widened here
      prefetch_tmap(&mF);
      if (!CONV) prefetch_tmap(&mS);
      const uint32_t bytes = (uint32_t)hn * 128 + (CONV ? 0 : kSBytes);
      int st = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int64_t i = pair; ok && i < p.units; i += pairs) {
        const Unit u = get_unit(p, i);
        const int ys = (int)(u.mt * kTile + cr * 128), yf = (int)(u.nt * p.NT + cr * hn);
        for (int s = u.s0; s < u.s1; ++s) {
          if (!(ok = wait(&empty[st], ph ^ 1, abort, p.err, 31))) break;
          const uint32_t dst = smem_u32(s16 + st * kStage), bar = mapa(smem_u32(&full[st]), 0);
          if (cr == 0) mbar_expect_tx(&full[st], 2 * bytes);
          if (!CONV) tma_load_pair(dst, &mS, s * kStep, ys, bar);
          tma_load_pair(dst + kSBytes, &mF, s * kStep, yf, bar);
          if (++st == R) {
            st = 0;
            ph ^= 1;
          }
        }
      }
    } else if (CONV && warp == 2 && lane == 0) {  // S as bytes
      prefetch_tmap(&mS);
      int st = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int64_t i = pair; ok && i < p.units; i += pairs) {
        const Unit u = get_unit(p, i);
        const int ys = (int)(u.mt * kTile + cr * 128);
        for (int s = u.s0; s < u.s1; ++s) {
          if (!(ok = wait(&empty8[st], ph ^ 1, abort, p.err, 36))) break;
          mbar_expect_tx(&full8[st], kBytes8);
          tma_load_2d(s8 + st * kBytes8, &mS, s * kStep, ys, &full8[st]);
          if (++st == R8) {
            st = 0;
            ph ^= 1;
          }
        }
      }
    } else if (warp == 1 && lane == 0 && cr == 0) {
      // fp16 operands, fp32 sums: the formats are 0
      const uint32_t idesc = (1u << 4) | ((uint32_t)(p.NT >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);
      int st = 0, gen = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int64_t i = pair; ok && i < p.units; i += pairs) {
        const Unit u = get_unit(p, i);
        for (int g = u.s0; ok && g < u.s1; g += kDrain, ++gen) {
          const int a = gen & 1;
          if (!(ok = wait(&tempty[a], ((gen >> 1) & 1) ^ 1, abort, p.err, 32))) break;
          tc_fence_after();
          const uint32_t d = tmem + a * 256;
          const int e = min(u.s1, g + kDrain);
          for (int s = g; s < e; ++s) {
            if (!(ok = wait(&full[st], ph, abort, p.err, 33))) break;
            tc_fence_after();
            const uint32_t ab = smem_u32(s16 + st * kStage), bb = ab + kSBytes;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_pair(d, smem_desc_sw128(ab + 32 * kk, 16, 1024), smem_desc_sw128(bb + 32 * kk, 16, 1024), idesc,
                        s > g || kk > 0);
            commit_pair(&empty[st]);
            if (++st == R) {
              st = 0;
              ph ^= 1;
            }
          }
          if (ok) commit_pair(&tfull[a]);
        }
      }
    }
  } else if (CONV && warp < Z::epi0) {
    // a team of four warps widens every other step: the waits, reads and writes
    // of one step lie under those of the next
    if constexpr (CONV) regs_down<48>();
    const int t = (threadIdx.x - 128) % (32 * kTeamWarps), team = (warp - 4) / kTeamWarps;
    int st = team, st8 = team;
    uint32_t ph = 0, ph8 = 0;
    const uint32_t full0 = mapa(smem_u32(full), 0);
    int turn = 0;
    bool ok = true;
    for (int64_t i = pair; ok && i < p.units; i += pairs) {
      const Unit u = get_unit(p, i);
      for (int s = u.s0; s < u.s1; ++s) {
        const bool mine = turn == team;
        turn = turn + 1 == kTeams ? 0 : turn + 1;
        if (!mine) continue;
        ok = wait(&full8[st8], ph8, abort, p.err, 37);
        if (!(ok = __all_sync(FULL, ok))) break;
        const uint8_t* src = s8 + st8 * kBytes8;
        uint4 w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = *reinterpret_cast<const uint4*>(src + (t + 128 * k) * 16);
        ok = wait(&empty[st], ph ^ 1, abort, p.err, 37);
        if (!(ok = __all_sync(FULL, ok))) break;
        uint8_t* dst = s16 + st * kStage;
#pragma unroll
        for (int k = 0; k < 4; ++k) widen_chunk(w[k], dst, t + 128 * k);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&empty8[st8]);
          arrive_cluster(full0 + st * 8);
        }
        if ((st8 += kTeams) >= R8) {
          st8 = team;
          ph8 ^= 1;
        }
        if ((st += kTeams) >= R) {
          st = team;
          ph ^= 1;
        }
      }
    }
  } else {
    if constexpr (CONV) regs_up<168>();
    const int quarter = warp & 3, part = (warp - Z::epi0) >> 2;
    float* stg = stg_all + (warp - Z::epi0) * ((kStg + kColVec) / 4);
    float* cv = stg + kStg / 4;
    const uint32_t tempty0 = mapa(smem_u32(tempty), 0);
    const int cb = part ? p.half : 0, ce = part ? p.NT : p.half;
    int gen = 0;
    bool ok = true;
    for (int64_t i = pair; ok && i < p.units; i += pairs) {
      const Unit u = get_unit(p, i);
      const int64_t row0 = u.mt * kTile + cr * 128 + quarter * 32, col0 = u.nt * p.NT + cb;
      const int gens = (u.s1 - u.s0 + kDrain - 1) / kDrain;
      const int64_t row = row0 + lane;
      float sr = 0.0f, br = 0.0f;
      if (p.part == nullptr) {  // while the products run
        __syncwarp();           // every lane is done with the last tile's
        if (row < p.M) {
          sr = p.sS[row];
          if (p.swap && p.bias != nullptr) br = p.bias[row];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int64_t c = col0 + 32 * k + lane;
          cv[32 * k + lane] = c < p.N ? p.sF[c] : 0.0f;
          cv[128 + 32 * k + lane] = c < p.N && p.bias != nullptr && !p.swap ? p.bias[c] : 0.0f;
        }
        __syncwarp();
      }
      if constexpr (!MULTI) {
        // the accumulator is the sum
        const int a = gen & 1;
        ok = wait(&tfull[a], (gen >> 1) & 1, abort, p.err, 38);
        ok = __all_sync(FULL, ok);
        if (!ok) break;
        ++gen;
        tc_fence_after();
        const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + a * 256 + cb;
#pragma unroll 1
        for (int c = 0; c < ce - cb; c += 32) {
          uint32_t r[32];
          tmem_ld32(taddr + c, r);
          tmem_ld_wait();
          if (c + 32 >= ce - cb) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_cluster(tempty0 + a * 8);
          }
          float v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
          put<true>(p, row0, col0 + c, v, sr, br, cv + c, stg, lane);
        }
        if (ce <= cb) {  // a tile of 32 columns has none for half of the warps
          __syncwarp();
          if (lane == 0) arrive_cluster(tempty0 + a * 8);
        }
      } else {
        int acc[4][32];
        for (int g = 0; g < gens; ++g, ++gen) {
          const int a = gen & 1;
          ok = wait(&tfull[a], (gen >> 1) & 1, abort, p.err, 38);
          ok = __all_sync(FULL, ok);
          if (!ok) break;
          tc_fence_after();
          const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + a * 256 + cb;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (cb + 32 * c < ce) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint32_t r[16];
                tmem_ld16(taddr + 32 * c + 16 * h, r);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                  const int x = __float2int_rn(__uint_as_float(r[j]));
                  acc[c][16 * h + j] = g == 0 ? x : acc[c][16 * h + j] + x;
                }
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_cluster(tempty0 + a * 8);
        }
        if (!ok) break;
// one copy of what follows for all four: the instruction cache holds it
#pragma unroll 1
        for (int c = 0; c < ce - cb; c += 32) {
          int x[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) x[j] = c == 0 ? acc[0][j] : c == 32 ? acc[1][j] : c == 64 ? acc[2][j] : acc[3][j];
          if (p.part != nullptr) {
            put_part(p, u, row0, col0 + c, x, stg, lane);
          } else {
            float v[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = (float)x[j];
            put<true>(p, row0, col0 + c, v, sr, br, cv + c, stg, lane);
          }
        }
      }
    }
  }
  __syncwarp();
  __syncthreads();
  // after a wait that gave up: copies and products under way (they take
  // microseconds) land before the pair's shared and tensor memory is given up
  if (*abort) {
    const long long t0 = clock64();
    while (clock64() - t0 < kDrainCycles) {
    }
  }
  __syncwarp();  // the lanes' clocks let them go one by one, and what follows is for whole warps
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc2(tmem, 512);
  }
  cluster_sync();
}

// ---------------------------------------------------- rows quantized on the way
// The product of full-precision rows with at most 256 rows of F, up to 256
// values long: a row's scale is known once it is read, so the widening warps
// quantize it between its copy in shared memory and the tensor cores, and DRAM
// sees the rows once and no codes.  A pair of CTAs takes 256 rows; F's half stays
// in shared memory; a CTA's 128 rows arrive in pieces of 16 KB (TMA, three in
// flight) and are whole in fp16 (64 KB) before their products start.
constexpr int kRowPiece = 16384, kRowSlots = 3, kRowK = 256;
constexpr int kRowSteps = kRowK / kStep;
constexpr int kRowThreads = 640;
constexpr int kRowSmem = 1024 + 2 * kRowSteps * kSBytes + kRowSlots * kRowPiece + kEpiWarps * (kStg + kColVec) + 2 * 128 * 4 +
                         512;

// four values of a staged row
template <typename T>
__device__ __forceinline__ float4 staged4(const uint8_t* row, int c) {
  return load4<T>(reinterpret_cast<const T*>(row) + c);
}

template <typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kRowThreads, 1)
    i8_rows_kernel(const __grid_constant__ CUtensorMap mX, const __grid_constant__ CUtensorMap mF, const TileArgs p) {
  constexpr int piece_rows = kRowPiece / (kRowK * (int)sizeof(T)), pieces = 128 / piece_rows;
  constexpr int per_warp = piece_rows / kConvWarps;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* sS = smem;                                   // [step][128 rows][128 bytes]
  uint8_t* sF = sS + kRowSteps * kSBytes;               // [step][NT / 2 rows][128 bytes]
  uint8_t* sX = sF + kRowSteps * kSBytes;               // pieces of rows as they are
  float* stg_all = reinterpret_cast<float*>(sX + kRowSlots * kRowPiece);
  float* scales = stg_all + kEpiWarps * (kStg + kColVec) / 4;  // [2][128]
  uint64_t* xfull = reinterpret_cast<uint64_t*>(scales + 256);
  uint64_t* xempty = xfull + kRowSlots;
  uint64_t* ffull = xempty + kRowSlots;  // F is there (both halves, in the even CTA)
  uint64_t* sfull = ffull + 1;           // both CTAs' rows are quantized (in the even CTA)
  uint64_t* sempty = sfull + 1;          // their products are done
  uint64_t* tfull = sempty + 1;
  uint64_t* tempty = tfull + 2;
  uint64_t* cfull = tempty + 2;          // this CTA's scales of a tile are there
  uint64_t* cempty = cfull + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(cempty + 2);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t cr = cluster_rank();
  if (threadIdx.x == 0) {
    for (int k = 0; k < kRowSlots; ++k) {
      mbar_init(&xfull[k], 1);
      mbar_init(&xempty[k], kConvWarps);
    }
    mbar_init(ffull, 1);
    mbar_init(sfull, 2 * kConvWarps);
    mbar_init(sempty, 1);
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 2 * kEpiWarps);
      mbar_init(&cfull[a], kConvWarps);
      mbar_init(&cempty[a], kEpiWarps);
    }
    *abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc2(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_wait();
  const int64_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int hn = p.NT / 2;

  // 3 warpgroups at 64 registers and 2 at 144: the 61,440 (96 a thread) that the
  // block is launched with
  if (warp < 4) {
    regs_down<64>();
    if (warp == 0 && lane == 0) {
      prefetch_tmap(&mX);
      prefetch_tmap(&mF);
      const uint32_t bar = mapa(smem_u32(ffull), 0);
      if (cr == 0) mbar_expect_tx(ffull, 2u * (uint32_t)(p.steps * hn * 128));
      for (int s = 0; s < p.steps; ++s) tma_load_pair(smem_u32(sF + s * kSBytes), &mF, s * kStep, (int)cr * hn, bar);
      int slot = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int64_t i = pair; ok && i < p.tm; i += pairs) {
        const int y = (int)(i * kTile + cr * 128);
        for (int k = 0; k < pieces; ++k) {
          if (!(ok = wait(&xempty[slot], ph ^ 1, abort, p.err, 41))) break;
          mbar_expect_tx(&xfull[slot], kRowPiece);
          tma_load_2d(sX + slot * kRowPiece, &mX, 0, y + k * piece_rows, &xfull[slot]);
          if (++slot == kRowSlots) {
            slot = 0;
            ph ^= 1;
          }
        }
      }
    } else if (warp == 1 && lane == 0 && cr == 0) {
      const uint32_t idesc = (1u << 4) | ((uint32_t)(p.NT >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);
      bool ok = wait(ffull, 0, abort, p.err, 42);
      int n = 0;
      for (int64_t i = pair; ok && i < p.tm; i += pairs, ++n) {
        const int a = n & 1;
        if (!(ok = wait(&tempty[a], ((n >> 1) & 1) ^ 1, abort, p.err, 43))) break;
        if (!(ok = wait(sfull, n & 1, abort, p.err, 44))) break;
        tc_fence_after();
        const uint32_t d = tmem + a * 256;
        for (int s = 0; s < p.steps; ++s) {
          const uint32_t ab = smem_u32(sS + s * kSBytes), bb = smem_u32(sF + s * kSBytes);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_pair(d, smem_desc_sw128(ab + 32 * kk, 16, 1024), smem_desc_sw128(bb + 32 * kk, 16, 1024), idesc,
                      s > 0 || kk > 0);
        }
        commit_pair(sempty);
        commit_pair(&tfull[a]);
      }
    }
  } else if (warp < 4 + kConvWarps) {
    regs_down<64>();
    const int cw = warp - 4;
    const uint32_t sfull0 = mapa(smem_u32(sfull), 0);
    int slot = 0, n = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int64_t i = pair; ok && i < p.tm; i += pairs, ++n) {
      // the tile before the last's scales have been read, the last tile's products are done
      ok = wait(&cempty[n & 1], ((n >> 1) & 1) ^ 1, abort, p.err, 45) && wait(sempty, (n & 1) ^ 1, abort, p.err, 45);
      if (!(ok = __all_sync(FULL, ok))) break;
      float* sc = scales + (n & 1) * 128;
      for (int k = 0; k < pieces; ++k) {
        ok = wait(&xfull[slot], ph, abort, p.err, 46);
        if (!(ok = __all_sync(FULL, ok))) break;
        const uint8_t* x = sX + slot * kRowPiece + cw * per_warp * kRowK * sizeof(T);
        float4 v[per_warp][2];
#pragma unroll
        for (int r = 0; r < per_warp; ++r) {
          v[r][0] = staged4<T>(x + r * kRowK * sizeof(T), 4 * lane);
          v[r][1] = staged4<T>(x + r * kRowK * sizeof(T), 128 + 4 * lane);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&xempty[slot]);
        Scale c[per_warp];  // the rows' chains of steps lie side by side
#pragma unroll
        for (int r = 0; r < per_warp; ++r) {
          const float4 &u = v[r][0], &w = v[r][1];
          const uint32_t top = max(max(max(mag(u.x), mag(u.y)), max(mag(u.z), mag(u.w))),
                                   max(max(mag(w.x), mag(w.y)), max(mag(w.z), mag(w.w))));
          c[r] = make_scale(__reduce_max_sync(FULL, top));
        }
#pragma unroll
        for (int r = 0; r < per_warp; ++r) {
          const int row = k * piece_rows + cw * per_warp + r;
          if (lane == 0) sc[row] = c[r].s;
          // columns 4 l .. of a 64-column step: 8 bytes of the 16-byte piece l / 2 of the row
          uint8_t* dst = sS + (lane >> 4) * kSBytes + row * 128 + ((((lane & 15) >> 1) ^ (row & 7)) << 4) + (lane & 1) * 8;
          *reinterpret_cast<uint2*>(dst) = halves4(quantize4(v[r][0], c[r]));
          *reinterpret_cast<uint2*>(dst + 2 * kSBytes) = halves4(quantize4(v[r][1], c[r]));
        }
        if (++slot == kRowSlots) {
          slot = 0;
          ph ^= 1;
        }
      }
      if (!ok) break;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&cfull[n & 1]);
        arrive_cluster(sfull0);
      }
    }
  } else {
    regs_up<144>();
    const int quarter = warp & 3, part = (warp - 12) >> 2;
    float* stg = stg_all + (warp - 12) * ((kStg + kColVec) / 4);
    float* cv = stg + kStg / 4;
    const uint32_t tempty0 = mapa(smem_u32(tempty), 0);
    const int cb = part ? p.half : 0, ce = part ? p.NT : p.half;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = cb + 32 * k + lane;
      cv[32 * k + lane] = c < p.N ? p.sF[c] : 0.0f;
      cv[128 + 32 * k + lane] = c < p.N && p.bias != nullptr ? p.bias[c] : 0.0f;
    }
    __syncwarp();
    int n = 0;
    bool ok = true;
    for (int64_t i = pair; ok && i < p.tm; i += pairs, ++n) {
      const int a = n & 1;
      const int64_t row0 = i * kTile + cr * 128 + quarter * 32;
      ok = wait(&cfull[a], (n >> 1) & 1, abort, p.err, 47);
      if (!(ok = __all_sync(FULL, ok))) break;
      const float sr = scales[a * 128 + quarter * 32 + lane];
      __syncwarp();
      if (lane == 0) mbar_arrive(&cempty[a]);
      ok = wait(&tfull[a], (n >> 1) & 1, abort, p.err, 48);
      if (!(ok = __all_sync(FULL, ok))) break;
      tc_fence_after();
      const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + a * 256 + cb;
#pragma unroll 1
      for (int c = 0; c < ce - cb; c += 32) {
        uint32_t r[32];
        tmem_ld32(taddr + c, r);
        tmem_ld_wait();
        if (c + 32 >= ce - cb) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_cluster(tempty0 + a * 8);
        }
        float v[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
        put<false>(p, row0, cb + c, v, sr, 0.0f, cv + c, stg, lane);
      }
      if (ce <= cb) {  // a tile of 32 columns has none for half of the warps
        __syncwarp();
        if (lane == 0) arrive_cluster(tempty0 + a * 8);
      }
    }
  }
  __syncwarp();
  __syncthreads();
  if (*abort) {  // as in the kernel above
    const long long t0 = clock64();
    while (clock64() - t0 < kDrainCycles) {
    }
  }
  __syncwarp();  // the lanes' clocks let them go one by one, and what follows is for whole warps
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc2(tmem, 512);
  }
  cluster_sync();
}

// Bytes as fp16, 16 at a time (a row's bytes up to the next multiple of 16 are read and widened too).
__global__ void __launch_bounds__(256)
    widen_kernel(const int8_t* A, int64_t rows, int per_row, int64_t lda, __half* out, int64_t ldo) {
  grid_wait();
  const int64_t total = rows * per_row;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / per_row, c = (i - r * per_row) * 16;
    const uint4 w = *reinterpret_cast<const uint4*>(A + r * lda + c);
    uint4 a, b;
    widen(w.x, a.x, a.y);
    widen(w.y, a.z, a.w);
    widen(w.z, b.x, b.y);
    widen(w.w, b.z, b.w);
    uint4* o = reinterpret_cast<uint4*>(out + r * ldo + c);
    o[0] = a;
    o[1] = b;
  }
}

// C from the splits' sums, added as 64-bit integers.
__global__ void __launch_bounds__(256) join_kernel(const TileArgs p) {
  grid_wait();
  const int64_t total = p.M * p.ldp;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / p.ldp, c = i - r * p.ldp;
    if (c >= p.N) continue;
    int64_t s = 0;
    for (int k = 0; k < p.splits; ++k) s += p.part[k * total + i];
    const float v = (float)s;
    if (p.swap)
      store_as(p.C, c * p.ldc + r,
               activate(fmaf(__fmul_rn(v, p.sF[c]), p.sS[r], p.bias != nullptr ? p.bias[r] : 0.0f), p.relu), p.type);
    else
      store_as(p.C, r * p.ldc + c,
               activate(fmaf(__fmul_rn(v, p.sS[r]), p.sF[c], p.bias != nullptr ? p.bias[c] : 0.0f), p.relu), p.type);
  }
}

// ---------------------------------------------------------------- few rows --
// Up to kFew rows of A: a warp takes rows of B, its lanes 16 bytes each of a
// row, products by dp4a; A's rows are read through L1 again and again, or, where
// they come in full precision (T) and are short, quantized by every block into
// its shared memory (one launch instead of two: 10,007 x 1,024 codes against a
// row of fp32: 7.7 us instead of 5.1 + 5.2 behind each other).  Bound by reading B,
// from four rows on by dp4a: 4,096 x 4,096 by 1, 2, 4, 8 rows 13, 15, 19, 33 us,
// where the tiles take 22.
constexpr int kFew = 4, kFewCodes = 16384;  // codes that a block quantizes
template <int M, int ROWS, typename T>
__global__ void __launch_bounds__(256)
    few_rows_kernel(const T* A, int64_t lda, const float* sA, const int8_t* B, int64_t N, int64_t ldb,
                    const float* sB, int K, const float* bias, void* C, int64_t ldc, int type, int relu) {
  constexpr bool QUANT = !std::is_same<T, int8_t>::value;
  extern __shared__ __align__(16) uint8_t codes[];
  __shared__ float scale[M];
  grid_wait();
  const int lane = threadIdx.x & 31;
  if constexpr (QUANT) {
    const int pitch = (K + 15) / 16 * 16;
    for (int m = threadIdx.x >> 5; m < M; m += 8) {
      const T* x = A + m * lda;
      uint32_t top = 0;
#pragma unroll 8
      for (int k = lane; k < K; k += 32) top = max(top, mag((float)x[k]));
      const Scale c = make_scale(__reduce_max_sync(FULL, top));
      if (lane == 0) scale[m] = c.s;
#pragma unroll 8
      for (int k = lane; k < K; k += 32) codes[m * pitch + k] = (uint8_t)code(quantize1((float)x[k], c));
    }
    __syncthreads();
  }
  const int64_t j0 = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * ROWS;
  if (j0 >= N) return;
  int acc[M][ROWS];
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int r = 0; r < ROWS; ++r) acc[m][r] = 0;
  for (int k = lane * 16; k < K; k += 512) {
    uint4 b[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
      b[r] = *reinterpret_cast<const uint4*>(B + (j0 + r < N ? j0 + r : N - 1) * ldb + k);
    const int left = K - k;  // bytes past K may hold anything: A's are taken as 0 there
#pragma unroll
    for (int m = 0; m < M; ++m) {
      uint4 a;
      if constexpr (QUANT)
        a = *reinterpret_cast<const uint4*>(codes + m * ((K + 15) / 16 * 16) + k);
      else
        a = *reinterpret_cast<const uint4*>(A + m * lda + k);
      if (left < 16) {
        uint32_t* w = &a.x;
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = left >= 4 * q + 4 ? w[q] : left <= 4 * q ? 0u : w[q] & ((1u << 8 * (left - 4 * q)) - 1);
      }
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        acc[m][r] = __dp4a((int)a.x, (int)b[r].x, acc[m][r]);
        acc[m][r] = __dp4a((int)a.y, (int)b[r].y, acc[m][r]);
        acc[m][r] = __dp4a((int)a.z, (int)b[r].z, acc[m][r]);
        acc[m][r] = __dp4a((int)a.w, (int)b[r].w, acc[m][r]);
      }
    }
  }
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const int s = __reduce_add_sync(FULL, acc[m][r]);
      const int64_t j = j0 + r;
      if (lane == (m * ROWS + r) % 32 && j < N)
        store_as(C, m * ldc + j,
                 activate(fmaf(__fmul_rn((float)s, QUANT ? scale[m] : sA[m]), sB[j], bias != nullptr ? bias[j] : 0.0f), relu),
                 type);
    }
}

// -------------------------------------------------------------------- host --
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

// bytes or fp16 [rows][cols] with row pitch ld (elements); boxes of 64 columns, zeros outside
int make_tmap(CUtensorMap* m, const void* base, bool wide, int64_t cols, int64_t rows, int64_t ld, int box_rows) {
  auto fn = encode_fn();
  if (fn == nullptr) return GQ_ERR_CUDA;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * (wide ? 2 : 1)};
  const cuuint32_t box[2] = {kStep, (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(m, wide ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
                        const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        wide ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? GQ_OK : GQ_ERR_INVALID_ARG;
}

int make_tmap_rows(CUtensorMap* m, const void* X, int type, int64_t cols, int64_t rows, int64_t ld) {
  auto fn = encode_fn();
  if (fn == nullptr) return GQ_ERR_CUDA;
  const int e = type == GQ_F32 ? 4 : 2;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * e};
  const cuuint32_t box[2] = {kRowK, (cuuint32_t)(kRowPiece / (kRowK * e))};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(m, type == GQ_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : type == GQ_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                                                            : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                        2, const_cast<void*>(X), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? GQ_OK : GQ_ERR_INVALID_ARG;
}

bool valid_type(int type) { return type == GQ_F32 || type == GQ_BF16 || type == GQ_F16; }
int type_bytes(int type) { return type == GQ_F32 ? 4 : 2; }
constexpr int64_t kMaxRows = (int64_t)1 << 30;  // tensor maps and coordinates

struct Plan {
  int swap, conv, NT, steps, splits, split_steps;
  int64_t M, N, tm, tn, ldp;
  size_t sums;           // bytes of the splits' sums
};

constexpr int64_t kConvColumns = 2048;

// S is A, unless A has fewer rows than a tile and than B: then B's rows fill
// the tiles, and C is written transposed.  F's tiles are as equal as multiples
// of 32 allow, and up to four more of them where a few tiles would be a wave of
// their own, by the cycles that the plan counts (5,003 x 1,000 by 777 on 76 pairs of
// CTAs: 140 tiles of 128 columns 29.3 us, 100 of 160 32.4, 80 of 224 35.5, cold). S that is given as bytes is widened in the kernel where it meets
// few rows of F, one pass over DRAM as bytes instead of bytes, fp16 out and
// fp16 in; else before it.  65,536 x 1,024 bytes by 256, 512, 1,024, 2,048 rows
// in the kernel 48, 70, 126, 231 us, before it 81, 95, 129, 197; 16,384 x 4,096
// by 64 rows 42 and 82.  Codes that are made in the call (`made`: of A, of B) are
// made as fp16: 131,072 x 1,024 by 512 rows 199 us, as bytes 222.
// The contraction is split where the tiles alone leave more than half of the
// pairs without work, and beyond 65,536 products.
Plan make_plan(int64_t m, int64_t n, int64_t k, bool a_made = false, bool b_made = false) {
  Plan z{};
  z.swap = m < kTile && n > m;
  z.M = z.swap ? n : m;
  z.N = z.swap ? m : n;
  z.conv = z.N < kConvColumns && !(z.swap ? b_made : a_made);
  z.tm = (z.M + kTile - 1) / kTile;
  z.steps = (int)((k + kStep - 1) / kStep);
  const int64_t pairs = sm_count() / 2 > 0 ? sm_count() / 2 : 1;
  const int64_t fewest = (z.N + kTile - 1) / kTile;
  int64_t best = INT64_MAX;
  for (int64_t tn = fewest; tn <= fewest + 4; ++tn) {
    const int64_t nt = ((z.N + tn - 1) / tn + 31) / 32 * 32, real = (z.N + nt - 1) / nt;
    const int64_t waves = (z.tm * real + pairs - 1) / pairs;
    // cycles: steps of at least 400, the last tile's epilogue
    const int64_t cost = waves * z.steps * (nt * 5 / 2 > 400 ? nt * 5 / 2 : 400) + 24 * nt;
    if (cost < best) {
      best = cost;
      z.NT = (int)nt;
      z.tn = real;
    }
    if (z.tm * real < pairs || waves > 4) break;  // the contraction is split, or the last wave matters little
  }
  int64_t want = pairs / (z.tm * z.tn);
  if (want < 1) want = 1;
  const int64_t most = (z.steps + 3) / 4;
  if (want > most) want = most;
  const int64_t least = (z.steps + kMaxSplitSteps - 1) / kMaxSplitSteps;
  if (want < least) want = least;
  int64_t per_split = (z.steps + want - 1) / want;
  if (per_split > kDrain) per_split = (per_split + kDrain - 1) / kDrain * kDrain;
  z.split_steps = (int)per_split;
  z.splits = (int)((z.steps + per_split - 1) / per_split);
  z.ldp = (z.N + 3) / 4 * 4;
  z.sums = z.splits > 1 ? (size_t)z.splits * z.M * z.ldp * 4 : 0;
  return z;
}

bool valid_shape(int64_t m, int64_t n, int64_t k) {
  return m >= 0 && n >= 1 && k >= 1 && m <= kMaxRows && n <= kMaxRows && k <= kMaxRows;
}

bool few(int64_t m, int64_t k) { return m <= kFew && k <= 65536; }  // a 32-bit sum holds twice that

int64_t round16(int64_t x) { return (x + 15) / 16 * 16; }
// rows that every block of the product quantizes for itself.  In the product | before
// it, against 10,007 rows, us: 4 x 256 values 8.9 | 10.9, 1 x 1,024 12.9 | 10.9, 4 x 1,024
// 13.0 | 12.9, 1 x 4,096 27.3 | 27.3, 4 x 4,096 29.3 | 28.3, 1 x 8,192 45.7 | 29.3, 1 x 16,384
// 84.6 | 51.9 (with the launches' gaps, cold; one launch instead of two, which counts
// where calls follow one another).
bool few_codes(int64_t m, int64_t k) { return few(m, k) && m * round16(k) <= kFewCodes; }
size_t round256(size_t x) { return (x + 255) / 256 * 256; }

// One operand of a product: codes as bytes or fp16, rows of a multiple of 16.
struct Operand {
  const void* q;
  int64_t ld;
  const float* scale;
};
// Whether the tile kernel takes A (or B) as fp16.
bool wants_wide(const Plan& z, bool is_a) { return !z.conv || is_a == (z.swap != 0); }
size_t code_bytes(int64_t rows, int64_t k, bool wide) { return round256((size_t)rows * round16(k) * (wide ? 2 : 1)); }

template <int M, typename T>
int few_rows(const T* A, int64_t lda, const float* sA, const Operand& B, int64_t N, int K, const float* bias, void* C,
             int64_t ldc, int type, int relu, cudaStream_t s) {
  constexpr int ROWS = M <= 2 ? 4 : 2;
  const int64_t blocks = (N + 8 * ROWS - 1) / (8 * ROWS);
  const size_t smem = std::is_same<T, int8_t>::value ? 0 : (size_t)M * round16(K);
  return launch_after(few_rows_kernel<M, ROWS, T>, dim3((unsigned)blocks), dim3(256), smem, s, A, lda, sA,
                      static_cast<const int8_t*>(B.q), N, B.ld, B.scale, K, bias, C, ldc, type, relu);
}

template <typename T>
int few_gemm(const T* a, int64_t lda, const float* sA, int64_t m, const Operand& B, int64_t n, int64_t k, const float* bias,
             int relu, void* C, int type, int64_t ldc, cudaStream_t s) {
#define GQ_FEW(I) \
  case I: return few_rows<I, T>(a, lda, sA, B, n, (int)k, bias, C, ldc, type, relu, s);
  switch (m) {
    GQ_FEW(1) GQ_FEW(2) GQ_FEW(3) GQ_FEW(4)
  }
#undef GQ_FEW
  return GQ_ERR_UNSUPPORTED;
}
int few_gemm(const Operand& A, int64_t m, const Operand& B, int64_t n, int64_t k, const float* bias, int relu, void* C,
             int type, int64_t ldc, cudaStream_t s) {
  return few_gemm(static_cast<const int8_t*>(A.q), A.ld, A.scale, m, B, n, k, bias, relu, C, type, ldc, s);
}

int widen(const int8_t* q, int64_t rows, int64_t k, int64_t ld, void* out, cudaStream_t s) {
  const int64_t per_row = round16(k) / 16;
  int64_t blocks = (rows * per_row + 255) / 256;
  if (blocks > 16 * (int64_t)sm_count()) blocks = 16 * (int64_t)sm_count();
  return launch_after(widen_kernel, dim3((unsigned)blocks), dim3(256), 0, s, q, rows, (int)per_row, ld,
                      static_cast<__half*>(out), round16(k));
}

template <bool CONV, bool MULTI>
int launch_tiles(const CUtensorMap& mS, const CUtensorMap& mF, const TileArgs& a, cudaStream_t s) {
  GQ_TRY_CUDA(cudaFuncSetAttribute(i8_tiles_kernel<CONV, MULTI>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   Shape<CONV>::smem));
  const int64_t pairs = sm_count() / 2 > 0 ? sm_count() / 2 : 1;
  const int64_t use = a.units < pairs ? a.units : pairs;
  return launch_after(i8_tiles_kernel<CONV, MULTI>, dim3((unsigned)(2 * use)), dim3(Shape<CONV>::threads), Shape<CONV>::smem, s,
                      mS, mF, a);
}

// The product of operands as wants_wide has them.
int tile_gemm(const Plan& z, const Operand& A, const Operand& B, int64_t k, const float* bias, int relu, void* C, int type,
              int64_t ldc, void* sums, int* err, cudaStream_t s) {
  TileArgs a{};
  a.M = z.M;
  a.N = z.N;
  a.steps = z.steps;
  a.NT = z.NT;
  a.half = (z.NT / 2 + 31) / 32 * 32;
  a.tm = z.tm;
  a.tn = z.tn;
  a.splits = z.splits;
  a.split_steps = z.split_steps;
  a.units = z.tm * z.tn * z.splits;
  a.C = C;
  a.ldc = ldc;
  a.type = type;
  a.relu = relu;
  a.swap = z.swap;
  a.vec = aligned(C, 16) && ldc * type_bytes(type) % 16 == 0;
  const Operand& S = z.swap ? B : A;
  const Operand& F = z.swap ? A : B;
  a.sS = S.scale;
  a.sF = F.scale;
  a.bias = bias;
  a.part = z.splits > 1 ? static_cast<int*>(sums) : nullptr;
  a.ldp = z.ldp;
  a.err = err;
  CUtensorMap mS, mF;
  GQ_TRY(make_tmap(&mS, S.q, !z.conv, k, z.M, S.ld, 128));
  GQ_TRY(make_tmap(&mF, F.q, true, k, z.N, F.ld, z.NT / 2));
  const bool multi = z.splits > 1 || z.steps > kDrain;
  if (z.conv)
    GQ_TRY((multi ? launch_tiles<true, true>(mS, mF, a, s) : launch_tiles<true, false>(mS, mF, a, s)));
  else
    GQ_TRY((multi ? launch_tiles<false, true>(mS, mF, a, s) : launch_tiles<false, false>(mS, mF, a, s)));
  if (a.part == nullptr) return GQ_OK;
  int64_t blocks = (z.M * z.ldp + 255) / 256;
  if (blocks > 65536) blocks = 65536;
  return launch_after(join_kernel, dim3((unsigned)blocks), dim3(256), 0, s, a);
}

// Whether rows of X can be quantized on their way to the product with n rows of F.
// On the way | codes before, 2,449,029 rows, us: fp32 256 -> 256 979 | 1,111, 256 -> 64
// 790 | 813, 256 -> 16 774 | 882, 64 -> 256 843 | 874, 100 -> 47 764 | 762, 128 -> 128
// 786 | 682, 64 -> 64 737 | 575; bf16 256 -> 256 1,172 | 1,059, 128 -> 128 916 | 653,
// 64 -> 64 818 | 597; 20,000 rows of fp32 256 -> 256 28 | 25, 100 of them 19 | 15.  It
// pays for many fp32 rows near its 256 values, what it is built for; narrower ones do
// 256 values' work, and 16-bit ones have less to save.
bool rows_fit(int64_t m, int64_t n, int64_t k) { return m > kFew && n <= kTile && k <= kRowK; }
bool rows_fit(int64_t m, int64_t n, int64_t k, const void* X, int type, int64_t ldx) {
  return rows_fit(m, n, k) && aligned(X, 16) && ldx * type_bytes(type) % 16 == 0;
}

template <typename T>
int launch_rows(const CUtensorMap& mX, const CUtensorMap& mF, const TileArgs& a, cudaStream_t s) {
  GQ_TRY_CUDA(cudaFuncSetAttribute(i8_rows_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRowSmem));
  const int64_t pairs = sm_count() / 2 > 0 ? sm_count() / 2 : 1;
  const int64_t use = a.tm < pairs ? a.tm : pairs;
  return launch_after(i8_rows_kernel<T>, dim3((unsigned)(2 * use)), dim3(kRowThreads), kRowSmem, s, mX, mF, a);
}

// act(X F^T + bias) with X's rows quantized on the way; F as fp16.
int rows_gemm(const void* X, int x_type, int64_t m, int64_t k, int64_t ldx, const Operand& F, int64_t n, const float* bias,
              int relu, void* C, int type, int64_t ldc, int* err, cudaStream_t s) {
  TileArgs a{};
  a.M = m;
  a.N = n;
  a.steps = (int)((k + kStep - 1) / kStep);
  a.NT = (int)((n + 31) / 32 * 32);
  a.half = (a.NT / 2 + 31) / 32 * 32;
  a.tm = (m + kTile - 1) / kTile;
  a.tn = 1;
  a.C = C;
  a.ldc = ldc;
  a.type = type;
  a.relu = relu;
  a.vec = aligned(C, 16) && ldc * type_bytes(type) % 16 == 0;
  a.sF = F.scale;
  a.bias = bias;
  a.err = err;
  CUtensorMap mX, mF;
  GQ_TRY(make_tmap_rows(&mX, X, x_type, k, m, ldx));
  GQ_TRY(make_tmap(&mF, F.q, true, k, n, F.ld, a.NT / 2));
  switch (x_type) {
    case GQ_F32: return launch_rows<float>(mX, mF, a, s);
    case GQ_BF16: return launch_rows<__nv_bfloat16>(mX, mF, a, s);
    default: return launch_rows<__half>(mX, mF, a, s);
  }
}

// Workspace of a product whose operands are given as bytes (a, b) or made in it.
size_t gemm_ws(int64_t m, int64_t n, int64_t k, bool a_bytes, bool b_bytes) {
  if (few(m, k)) return 0;
  const Plan z = make_plan(m, n, k, !a_bytes, !b_bytes);
  return round256(z.sums) + (a_bytes && wants_wide(z, true) ? code_bytes(m, k, true) : 0) +
         (b_bytes && wants_wide(z, false) ? code_bytes(n, k, true) : 0);
}

template <typename T, typename O>
int quant_rows(const T* X, int64_t n, int d, int64_t ldx, O* Q, int64_t ldq, float* S, cudaStream_t s) {
  const bool vec = aligned(X, 4 * sizeof(T)) && ldx % 4 == 0;
  const int per = d <= 4096 ? kQThreads / 32 : 1;
  const int64_t blocks = (n + per - 1) / per;
  if (blocks > 0x7fffffff) return GQ_ERR_UNSUPPORTED;
  auto go = [&](void (*kernel)(const T*, int64_t, int, int64_t, O*, int64_t, float*)) {
    return launch_after(kernel, dim3((unsigned)blocks), dim3(kQThreads), 0, s, X, n, d, ldx, Q, ldq, S);
  };
  if (vec && d <= 1024)
    return go(d <= 128 ? quant_short_rows_kernel<T, O, 1> : d <= 256 ? quant_short_rows_kernel<T, O, 2>
              : d <= 512 ? quant_short_rows_kernel<T, O, 4> : quant_short_rows_kernel<T, O, 8>);
  if (d <= 4096) return go(vec ? quant_rows_kernel<T, O, true, 32> : quant_rows_kernel<T, O, false, 32>);
  return go(vec ? quant_rows_kernel<T, O, true, kQThreads> : quant_rows_kernel<T, O, false, kQThreads>);
}

// Pieces of the columns' first pass: four blocks an SM, at least 64 rows each, and
// no more than every block of the second pass can put together.
int64_t col_parts(int64_t n, int d) {
  const int64_t gx = (d + kColW - 1) / kColW;
  int64_t parts = (4 * (int64_t)sm_count() + gx - 1) / gx;
  const int64_t most = (n + 63) / 64;
  if (parts > most) parts = most;
  if (parts > kMaxParts) parts = kMaxParts;
  return parts < 1 ? 1 : parts;
}
size_t cols_ws(int64_t n, int d, int sums) { return (size_t)col_parts(n, d) * d * 4 * (sums ? 2 : 1); }

template <typename T, typename O>
ColJob<T, O> col_job(const T* X, int64_t n, int d, int64_t ldx, O* Q, int64_t ldq, float* S, float* colsum, void* ws) {
  ColJob<T, O> j{};
  j.X = X;
  j.n = n;
  j.d = d;
  j.ldx = ldx;
  j.vec = aligned(X, 4 * sizeof(T)) && ldx % 4 == 0;
  j.parts = (int)col_parts(n, d);
  j.rows_per = (n + j.parts - 1) / j.parts;
  j.top = static_cast<uint32_t*>(ws);
  j.sums = colsum != nullptr ? reinterpret_cast<float*>(j.top + (int64_t)j.parts * d) : nullptr;
  j.Q = Q;
  j.ldq = ldq;
  j.S = S;
  j.colsum = colsum;
  return j;
}

template <typename T, typename O>
int quant_cols(const ColJobs<T, O>& jobs, int count, cudaStream_t s) {
  unsigned gx = 1, gy = 1;
  int64_t tiles = 1;
  for (int k = 0; k < count; ++k) {
    const ColJob<T, O>& j = jobs.of[k];
    const unsigned w = (unsigned)((j.d + kColW - 1) / kColW);
    const int64_t t = (j.n + kTrRows - 1) / kTrRows;
    if (w > gx) gx = w;
    if ((unsigned)j.parts > gy) gy = (unsigned)j.parts;
    if (t > tiles) tiles = t;
  }
  GQ_TRY(launch_after(col_max_kernel<T, O>, dim3(gx, gy, (unsigned)count), dim3(kQThreads), 0, s, jobs));
  int64_t most = (8 * (int64_t)sm_count() + gx - 1) / gx;
  if (most < 1) most = 1;
  return launch_after(quant_cols_kernel<T, O>, dim3((unsigned)(tiles < most ? tiles : most), gx, (unsigned)count),
                      dim3(kQThreads), 0, s, jobs);
}

template <typename T, typename O>
int quant_to(const void* X, int64_t n, int d, int64_t ldx, int transpose, void* Q, int64_t ldq, float* S, float* colsum,
             void* ws, cudaStream_t s) {
  const T* x = static_cast<const T*>(X);
  O* q = static_cast<O*>(Q);
  if (!transpose) return quant_rows(x, n, d, ldx, q, ldq, S, s);
  ColJobs<T, O> jobs;
  jobs.of[0] = jobs.of[1] = col_job(x, n, d, ldx, q, ldq, S, colsum, ws);
  return quant_cols(jobs, 1, s);
}

int quant(const void* X, int type, int64_t n, int d, int64_t ldx, int transpose, bool wide, void* Q, int64_t ldq, float* S,
          float* colsum, void* ws, cudaStream_t s) {
  switch (type) {
    case GQ_F32:
      return wide ? quant_to<float, __half>(X, n, d, ldx, transpose, Q, ldq, S, colsum, ws, s)
                  : quant_to<float, int8_t>(X, n, d, ldx, transpose, Q, ldq, S, colsum, ws, s);
    case GQ_BF16:
      return wide ? quant_to<__nv_bfloat16, __half>(X, n, d, ldx, transpose, Q, ldq, S, colsum, ws, s)
                  : quant_to<__nv_bfloat16, int8_t>(X, n, d, ldx, transpose, Q, ldq, S, colsum, ws, s);
    default:
      return wide ? quant_to<__half, __half>(X, n, d, ldx, transpose, Q, ldq, S, colsum, ws, s)
                  : quant_to<__half, int8_t>(X, n, d, ldx, transpose, Q, ldq, S, colsum, ws, s);
  }
}

constexpr int kMaxCols = 65535 * kColW / 2;  // quantizer's grid in y
}  // namespace
}  // namespace gq

extern "C" size_t gq_quantize_i8_workspace_bytes(int64_t n, int d, int transpose) {
  if (n < 0 || d < 1 || d > gq::kMaxCols || !transpose) return 0;
  return gq::cols_ws(n, d, 0);
}

extern "C" int gq_quantize_i8(const void* X, int type, int64_t n, int d, int64_t ldx, int transpose, int8_t* Q,
                              int64_t ldq, float* scale, void* ws, size_t ws_bytes, gq_stream stream) {
  using namespace gq;
  if (!valid_type(type) || n < 0 || d < 1 || ldx < d || ldq < (transpose ? n : d) || ldq % 16) return GQ_ERR_INVALID_ARG;
  if (n > kMaxRows || d > kMaxCols) return GQ_ERR_UNSUPPORTED;
  if (n == 0) return GQ_OK;
  if (X == nullptr || Q == nullptr || scale == nullptr || !aligned(X, type_bytes(type)) || !aligned(Q, 16) ||
      !aligned(scale, 4))
    return GQ_ERR_INVALID_ARG;
  if (transpose && (ws == nullptr || !aligned(ws, 16) || ws_bytes < cols_ws(n, d, 0))) return GQ_ERR_WORKSPACE;
  return quant(X, type, n, d, ldx, transpose, false, Q, ldq, scale, nullptr, ws, (cudaStream_t)stream);
}

extern "C" size_t gq_gemm_i8_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  if (!gq::valid_shape(m, n, k) || m == 0) return 0;
  return gq::gemm_ws(m, n, k, true, true);
}

extern "C" int gq_gemm_i8(const int8_t* A, int64_t m, int64_t lda, const float* scale_a, const int8_t* B, int64_t n,
                          int64_t ldb, const float* scale_b, int64_t k, const float* bias, int act, void* C, int type,
                          int64_t ldc, void* ws, size_t ws_bytes, int* dev_err, gq_stream stream) {
  using namespace gq;
  if (m < 0 || n < 1 || k < 1 || !valid_type(type) || (act != GQ_ACT_NONE && act != GQ_ACT_RELU) || lda < k ||
      ldb < k || lda % 16 || ldb % 16 || ldc < n)
    return GQ_ERR_INVALID_ARG;
  if (!valid_shape(m, n, k)) return GQ_ERR_UNSUPPORTED;
  if (m == 0) return GQ_OK;
  if (A == nullptr || B == nullptr || C == nullptr || scale_a == nullptr || scale_b == nullptr || !aligned(A, 16) ||
      !aligned(B, 16) || !aligned(C, type_bytes(type)) || !aligned(scale_a, 4) || !aligned(scale_b, 4) ||
      !aligned(bias, 4) || !aligned(dev_err, 4))
    return GQ_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  Operand a{A, lda, scale_a}, b{B, ldb, scale_b};
  if (few(m, k)) return few_gemm(a, m, b, n, k, bias, act == GQ_ACT_RELU, C, type, ldc, s);
  const Plan z = make_plan(m, n, k);
  const size_t need = gemm_ws(m, n, k, true, true);
  if (need > 0 && (ws == nullptr || ws_bytes < need || !aligned(ws, 256))) return GQ_ERR_WORKSPACE;
  Carve w(ws, ws_bytes);
  if (wants_wide(z, true)) {
    void* q = w.take(code_bytes(m, k, true));
    GQ_TRY(widen(A, m, k, lda, q, s));
    a = Operand{q, round16(k), scale_a};
  }
  if (wants_wide(z, false)) {
    void* q = w.take(code_bytes(n, k, true));
    GQ_TRY(widen(B, n, k, ldb, q, s));
    b = Operand{q, round16(k), scale_b};
  }
  return tile_gemm(z, a, b, k, bias, act == GQ_ACT_RELU, C, type, ldc, z.sums > 0 ? w.take(z.sums) : nullptr, dev_err, s);
}

extern "C" size_t gq_linear_i8_workspace_bytes(int64_t n, int k, int out) {
  using namespace gq;
  if (!valid_shape(n, out, k) || n == 0) return 0;
  if (few_codes(n, k)) return 0;
  const bool wide = !few(n, k) && wants_wide(make_plan(n, out, k, true, false), true);
  const size_t split = code_bytes(n, k, wide) + round256((size_t)n * 4) + gemm_ws(n, out, k, false, true);
  const size_t fused = rows_fit(n, out, k) ? code_bytes(out, k, true) : 0;
  return split > fused ? split : fused;
}

extern "C" int gq_linear_i8(const void* X, int type, int64_t n, int k, int64_t ldx, const int8_t* W, int out,
                            int64_t ldw, const float* scale_w, const float* bias, int act, void* Y, int y_type,
                            int64_t ldy, void* ws, size_t ws_bytes, int* dev_err, gq_stream stream) {
  using namespace gq;
  if (!valid_type(type) || !valid_type(y_type) || n < 0 || k < 1 || out < 1 || ldx < k || ldw < k || ldw % 16 ||
      ldy < out || (act != GQ_ACT_NONE && act != GQ_ACT_RELU))
    return GQ_ERR_INVALID_ARG;
  if (!valid_shape(n, out, k) || k > kMaxCols) return GQ_ERR_UNSUPPORTED;
  if (n == 0) return GQ_OK;
  if (X == nullptr || W == nullptr || Y == nullptr || scale_w == nullptr || !aligned(X, type_bytes(type)) ||
      !aligned(W, 16) || !aligned(Y, type_bytes(y_type)) || !aligned(scale_w, 4) || !aligned(bias, 4) ||
      !aligned(dev_err, 4))
    return GQ_ERR_INVALID_ARG;
  const size_t need = gq_linear_i8_workspace_bytes(n, k, out);
  if (need > 0 && (ws == nullptr || !aligned(ws, 256) || ws_bytes < need)) return GQ_ERR_WORKSPACE;
  cudaStream_t s = (cudaStream_t)stream;
  const int relu = act == GQ_ACT_RELU;
  const int64_t ld = round16(k);
  Carve w(ws, ws_bytes);
  if (rows_fit(n, out, k, X, type, ldx)) {
    void* qw = w.take(code_bytes(out, k, true));
    GQ_TRY(widen(W, out, k, ldw, qw, s));
    return rows_gemm(X, type, n, k, ldx, Operand{qw, ld, scale_w}, out, bias, relu, Y, y_type, ldy, dev_err, s);
  }
  float* sc = static_cast<float*>(w.take((size_t)n * 4));
  if (few_codes(n, k)) {
    const Operand b{W, ldw, scale_w};
    switch (type) {
      case GQ_F32:
        return few_gemm(static_cast<const float*>(X), ldx, nullptr, n, b, out, k, bias, relu, Y, y_type, ldy, s);
      case GQ_BF16:
        return few_gemm(static_cast<const __nv_bfloat16*>(X), ldx, nullptr, n, b, out, k, bias, relu, Y, y_type, ldy, s);
      default: return few_gemm(static_cast<const __half*>(X), ldx, nullptr, n, b, out, k, bias, relu, Y, y_type, ldy, s);
    }
  }
  if (few(n, k)) {
    void* q = w.take(code_bytes(n, k, false));
    GQ_TRY(quant(X, type, n, k, ldx, 0, false, q, ld, sc, nullptr, nullptr, s));
    return few_gemm(Operand{q, ld, sc}, n, Operand{W, ldw, scale_w}, out, k, bias, relu, Y, y_type, ldy, s);
  }
  const Plan z = make_plan(n, out, k, true, false);
  const bool wide = wants_wide(z, true);
  void* q = w.take(code_bytes(n, k, wide));
  GQ_TRY(quant(X, type, n, k, ldx, 0, wide, q, ld, sc, nullptr, nullptr, s));
  Operand b{W, ldw, scale_w};
  if (wants_wide(z, false)) {
    void* qw = w.take(code_bytes(out, k, true));
    GQ_TRY(widen(W, out, k, ldw, qw, s));
    b = Operand{qw, ld, scale_w};
  }
  return tile_gemm(z, Operand{q, ld, sc}, b, k, bias, relu, Y, y_type, ldy, z.sums > 0 ? w.take(z.sums) : nullptr, dev_err,
                   s);
}

namespace gq {
namespace {
// a product of rows (or columns) of two matrices that are quantized for it
struct Side {
  const void* X;
  int type;
  int64_t n;
  int d;
  int64_t ldx;
  int transpose;
};
// two matrices of one type by columns, to the same kind of codes
template <typename T, typename O>
int quant_pair_to(const Side& a, void* qa, float* sa, float* colsum, void* ca, const Side& b, void* qb, float* sb, void* cb,
                  int64_t ld, cudaStream_t s) {
  ColJobs<T, O> jobs;
  jobs.of[0] = col_job(static_cast<const T*>(a.X), a.n, a.d, a.ldx, static_cast<O*>(qa), ld, sa, colsum, ca);
  jobs.of[1] = col_job(static_cast<const T*>(b.X), b.n, b.d, b.ldx, static_cast<O*>(qb), ld, sb, (float*)nullptr, cb);
  return quant_cols(jobs, 2, s);
}
template <typename O>
int quant_pair(const Side& a, void* qa, float* sa, float* colsum, void* ca, const Side& b, void* qb, float* sb, void* cb,
               int64_t ld, cudaStream_t s) {
  switch (a.type) {
    case GQ_F32: return quant_pair_to<float, O>(a, qa, sa, colsum, ca, b, qb, sb, cb, ld, s);
    case GQ_BF16: return quant_pair_to<__nv_bfloat16, O>(a, qa, sa, colsum, ca, b, qb, sb, cb, ld, s);
    default: return quant_pair_to<__half, O>(a, qa, sa, colsum, ca, b, qb, sb, cb, ld, s);
  }
}
size_t product_ws(int64_t m, int64_t n, int64_t k, bool ta, bool tb, bool sums) {
  const bool tiny = few(m, k);
  const Plan z = make_plan(m, n, k, true, true);
  const bool fused = !ta && rows_fit(m, n, k);  // then B is fp16
  return code_bytes(m, k, !tiny && wants_wide(z, true)) + code_bytes(n, k, fused || (!tiny && wants_wide(z, false))) +
         round256((size_t)m * 4) + round256((size_t)n * 4) + (ta ? round256(cols_ws(k, (int)m, sums)) : 0) +
         (tb ? round256(cols_ws(k, (int)n, 0)) : 0) + (tiny ? 0 : round256(z.sums));
}
int product(const Side& a, const Side& b, int64_t m, int64_t n, int64_t k, float* colsum, void* C, int type, int64_t ldc,
            void* ws, size_t ws_bytes, int* err, cudaStream_t s) {
  const bool tiny = few(m, k);
  const Plan z = make_plan(m, n, k, true, true);
  const bool wa = !tiny && wants_wide(z, true), wb = !tiny && wants_wide(z, false);
  const int64_t ld = round16(k);
  Carve w(ws, ws_bytes);
  if (!a.transpose && rows_fit(m, n, k, a.X, a.type, a.ldx)) {
    void* q = w.take(code_bytes(n, k, true));
    float* sc = static_cast<float*>(w.take((size_t)n * 4));
    void* c = b.transpose ? w.take(cols_ws(b.n, b.d, 0)) : nullptr;
    GQ_TRY(quant(b.X, b.type, b.n, b.d, b.ldx, b.transpose, true, q, ld, sc, nullptr, c, s));
    return rows_gemm(a.X, a.type, m, k, a.ldx, Operand{q, ld, sc}, n, nullptr, 0, C, type, ldc, err, s);
  }
  void* qa = w.take(code_bytes(m, k, wa));
  void* qb = w.take(code_bytes(n, k, wb));
  float* sa = static_cast<float*>(w.take((size_t)m * 4));
  float* sb = static_cast<float*>(w.take((size_t)n * 4));
  void* ca = a.transpose ? w.take(cols_ws(a.n, a.d, colsum != nullptr)) : nullptr;
  void* cb = b.transpose ? w.take(cols_ws(b.n, b.d, 0)) : nullptr;
  if (a.transpose && b.transpose && a.type == b.type && wa == wb) {
    GQ_TRY(wa ? quant_pair<__half>(a, qa, sa, colsum, ca, b, qb, sb, cb, ld, s)
              : quant_pair<int8_t>(a, qa, sa, colsum, ca, b, qb, sb, cb, ld, s));
  } else {
    GQ_TRY(quant(a.X, a.type, a.n, a.d, a.ldx, a.transpose, wa, qa, ld, sa, colsum, ca, s));
    GQ_TRY(quant(b.X, b.type, b.n, b.d, b.ldx, b.transpose, wb, qb, ld, sb, nullptr, cb, s));
  }
  const Operand A{qa, ld, sa}, B{qb, ld, sb};
  if (tiny) return few_gemm(A, m, B, n, k, nullptr, 0, C, type, ldc, s);
  return tile_gemm(z, A, B, k, nullptr, 0, C, type, ldc, z.sums > 0 ? w.take(z.sums) : nullptr, err, s);
}
size_t bwd_ws(int64_t n, int k, int out, bool need_dx, bool need_dw) {
  const size_t dx = need_dx ? product_ws(n, k, out, false, true, false) : 0;
  const size_t dw = need_dw ? product_ws(out, k, n, true, true, true) : 0;
  return dx > dw ? dx : dw;
}
}  // namespace
}  // namespace gq

extern "C" size_t gq_linear_i8_bwd_workspace_bytes(int64_t n, int k, int out, int need_dx, int need_dw) {
  using namespace gq;
  if (!valid_shape(n, out, k) || n == 0 || k > kMaxCols || out > kMaxCols) return 0;
  return bwd_ws(n, k, out, need_dx != 0, need_dw != 0);
}

extern "C" int gq_linear_i8_bwd(const void* dY, int64_t lddy, const void* X, int64_t ldx, int type, int64_t n, int k,
                                int out, const void* W, int w_type, int64_t ldw, void* dX, int dx_type, int64_t lddx,
                                void* dW, int dw_type, int64_t lddw, float* dbias, void* ws, size_t ws_bytes,
                                int* dev_err, gq_stream stream) {
  using namespace gq;
  if (!valid_type(type) || n < 0 || k < 1 || out < 1 || lddy < out) return GQ_ERR_INVALID_ARG;
  if (dbias != nullptr && dW == nullptr) return GQ_ERR_INVALID_ARG;
  if (dX != nullptr && (W == nullptr || !valid_type(w_type) || !valid_type(dx_type) || ldw < k || lddx < k ||
                        !aligned(W, type_bytes(w_type)) || !aligned(dX, type_bytes(dx_type))))
    return GQ_ERR_INVALID_ARG;
  if (dW != nullptr && (!valid_type(dw_type) || ldx < k || lddw < k || !aligned(dW, type_bytes(dw_type))))
    return GQ_ERR_INVALID_ARG;
  if (!aligned(dbias, 4) || !aligned(dev_err, 4)) return GQ_ERR_INVALID_ARG;
  if (!valid_shape(n, out, k) || k > kMaxCols || out > kMaxCols) return GQ_ERR_UNSUPPORTED;
  cudaStream_t s = (cudaStream_t)stream;
  if (n == 0) {
    if (dW != nullptr)
      GQ_TRY_CUDA(cudaMemset2DAsync(dW, (size_t)lddw * type_bytes(dw_type), 0, (size_t)k * type_bytes(dw_type),
                                    (size_t)out, s));
    if (dbias != nullptr) GQ_TRY_CUDA(cudaMemsetAsync(dbias, 0, (size_t)out * 4, s));
    return GQ_OK;
  }
  if (dY == nullptr || !aligned(dY, type_bytes(type)) ||
      (dW != nullptr && (X == nullptr || !aligned(X, type_bytes(type)))))
    return GQ_ERR_INVALID_ARG;
  if (dX == nullptr && dW == nullptr) return GQ_OK;
  if (ws == nullptr || !aligned(ws, 256) || ws_bytes < bwd_ws(n, k, out, dX != nullptr, dW != nullptr))
    return GQ_ERR_WORKSPACE;
  if (dX != nullptr)  // dY by rows, W by columns
    GQ_TRY(product(Side{dY, type, n, out, lddy, 0}, Side{W, w_type, out, k, ldw, 1}, n, k, out, nullptr, dX, dx_type, lddx,
                   ws, ws_bytes, dev_err, s));
  if (dW != nullptr)  // both by columns
    GQ_TRY(product(Side{dY, type, n, out, lddy, 1}, Side{X, type, n, k, ldx, 1}, out, k, n, dbias, dW, dw_type, lddw, ws,
                   ws_bytes, dev_err, s));
  return GQ_OK;
}
