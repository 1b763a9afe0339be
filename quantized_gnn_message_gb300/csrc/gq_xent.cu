// gq_xent.cu -- softmax cross entropy of a linear class head over many
// classes, with its gradients, without keeping the logits.
//
//   Z = X W^T (n x C);  lse_i = log sum_c exp(Z_ic);  loss_i = lse_i - Z_iy
//   G = w_i (softmax(Z) - onehot(y));  dX = scale G W;  dW = scale G^T X
//
// Rows without a label take no part: the labelled rows are numbered in order
// by a scan, and copied together unless every row is labelled, so neither
// their number nor what they hold reaches the products.
//
// Products on the tcgen05 tensor cores (bf16 inputs, fp32 sums in TMEM), all
// tiles of one persistent kernel:
//   STATS  Z tile -> running maximum and sum of exponentials per row and run
//          of class tiles, and the label's logit of the rows that have it there
//   GRAD   Z tile again -> G of one piece of the classes, in bf16
//   WHOLE  STATS and GRAD of a tile that holds every class (C <= 256): the
//          logits are read twice from TMEM, and nothing is recomputed
//   DX     dX += G W over the piece (fp32 sums between pieces)
//   DW     dW of the piece's classes = G^T X
// 8 n k C operations where keeping all of Z (4 n C bytes) would need 6.  One
// launch holds the DX and DW tiles of a piece and the GRAD tiles of the next
// (two buffers of G), so that only the last launch has a tail.
//
// Tiles are 256 x up to 256 x 64 for a pair of CTAs (cta_group::2): each CTA
// loads 128 rows of A and half of B's columns, so each operand byte is read
// from L2 once per pair.  Per CTA:
//   warp 0      TMA loads into a ring of five 32 KB stages; both CTAs' bytes
//               arrive on the even CTA's barrier
//   warp 1      (even CTA) one thread issues tcgen05.mma into one of two
//               TMEM accumulators of 256 columns; its commits release the
//               stages of both CTAs
//   warps 2-9   epilogue: lane = row, the chunks of 32 or 64 columns dealt
//               out to two warps per 32 rows; the next tile's products run
//               meanwhile in the other accumulator (16 warps: no faster on
//               short tiles, and 5% slower on long ones, where power counts)
//   warp 10     (even CTA) draws the next unit of work from a counter and
//               posts it to both CTAs.  Which CTA computes a tile does not
//               change its value, so results do not depend on the order.
//
// G is kept in blocks of 64 classes, [class / 64][row][class % 64], so that a
// box of DX (64 classes x 128 rows) or DW (64 x 64) is one contiguous run of
// memory (with rows of a power-of-two pitch 16,384 x 1,024 x 131,072 took 11.4
// ms against 11.0).
//
// Bound: the tensor cores and the power they draw where k is large (16,384 x
// 1,024 x 131,072 with gradients: 11.0 ms, 1.60 PFLOP/s of the 8 n k C, of
// 1.69 that a plain bf16 product sustains); the epilogues and G's way through
// DRAM (written once, read twice: 12.9 GB) where it is small (k = 256: 3.7 ms,
// 1.19 PFLOP/s).  Few classes (2,449,029 x 256 x 47, every row labelled): 0.89 to
// 0.96 ms for 3.2 GB read and 1.6 GB written, 5.0 to 5.4 TB/s.
//
// The label's logit comes out of the same tiles as the sum of exponentials: a dot
// product of its own is cheaper by 1 to 2% of STATS, but sums in another order
// (and the tensor cores truncate), and the difference stood as loss and as
// gradient in rows that are certain of their label.
//
// G is rounded to bf16, the type that the products dX and dW take: each
// entry is off by at most half a step (2^-8 of its value, about as much as
// the rounding of a bf16 result; errors of a sum's entries mostly cancel).
// The common factor `scale` is applied to the fp32 sums instead: within G it
// would put the same rounding error on every row's largest entry, p - 1.
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include <cstdint>
#include <cstring>

#include "gq_common.cuh"
#include "gq_internal.cuh"
#include "gq_sm100.cuh"
#include "gq_train.h"

namespace gq {
namespace {

constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (kEpiWarps + 3);  // TMA, MMA, epilogue, scheduler
constexpr int kParts = kEpiWarps / 4;           // warps that share a row's columns
static_assert(kParts == 2, "WHOLE tiles go by turns to the two warps of 32 rows");
constexpr int kStages = 5;
constexpr int kStageA = 128 * 128;                    // 128 rows x 64 bf16 (or 2 x 64 x 64)
constexpr int kStageBytes = 2 * kStageA;
constexpr int kBox = 4096;       // 32 rows x 64 bf16
constexpr int kStg = 2 * kBox;   // epilogue staging per warp
constexpr int kSlots = 4;        // units of work posted ahead
constexpr int kConsumers = 3 + 2 * kEpiWarps;  // even CTA: TMA, MMA, epilogue; odd CTA: TMA, epilogue
constexpr int kSmem = 1024 + kStages * kStageBytes + kEpiWarps * kStg + 512;
constexpr int kTile = 256;
constexpr long long kDrainCycles = 1 << 21;  // 1 ms
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

enum Mode { STATS, GRAD, WHOLE, DX, DW };

struct Maps {
  CUtensorMap xk[2], xm[2];  // X: [0] as given, [1] the copied labelled rows; K-major / MN-major boxes
  CUtensorMap wk, wm;        // W
  CUtensorMap gk, gm;        // the piece of G read by DX / DW
  CUtensorMap gst;           // the piece of G written by GRAD
  CUtensorMap ox, ow;        // dX, dW
};

struct Args {
  const int* nl;         // number of labelled rows (device)
  int* counter;          // next unit of this launch
  int64_t n, npad;       // rows of X; rounded up to 256
  int k, C;
  int NT, NK, nkt;       // class tile width, k tile width, k tiles
  int stats_tiles, stats_run, stats_units;  // class tiles, tiles per unit, units per row tile (0: none)
  int gc0, gtiles;       // GRAD: first class and class tiles of the piece written (0 tiles: none)
  int pc0, psteps, ptiles;  // DX / DW: first class, 64-class steps, 256-class tiles of the piece read
  int do_dx, do_dw, dw_first;
  int dxs, dws;          // splits of their sums
  int first, last;       // the piece read is the first / last one
  float scale;           // of the results: G is formed without it, see below
  int full;              // the tiles of gtiles are WHOLE (1: losses only, 2: G too)
  const float* wrow;     // per labelled row, for WHOLE: weight, label
  const int* lab;
  float* loss;           // per row of X, nullable
  float* lse;
  const float4* row;     // r, weight / sum of 2^(z L - r), weight, label (as int)
  float* zlab;           // per labelled row, by STATS: the label's logit
  const int* idx;        // labelled row -> row of X
  float2* part;          // [unit * kParts + part][npad]: r, sum
  float* accX;           // [split][row tile][nkt NK][256]
  float* accW;           // [split][class tile][nkt NK][256]
  __nv_bfloat16* dX;
  int64_t lddx;
  __nv_bfloat16* dW;
  int64_t lddw;
  int* err;
};

// ------------------------------------------------------------ PTX helpers --
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
// Arrival on a barrier of either CTA.  CTA scope: what the arrivals follow are
// reads of this warp, not global writes, and a release at cluster scope costs
// a memory barrier each time (a quarter of the warps' stalls; loss and
// gradients of 16,384 x 256 x 131,072 classes 4.93 -> 4.67 ms without it).  At
// this scope the arrival orders nothing that the other CTA sees, so what has
// been read must be in registers before it: a posted unit by a branch on its
// value (Feed::next), an accumulator by tcgen05.wait::ld.
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void expect_cluster(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void st_async(uint32_t addr, int v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.s32 [%0], %1, [%2];" ::"r"(addr), "r"(v),
               "r"(bar)
               : "memory");
}
__device__ __forceinline__ void tmem_alloc2(uint32_t* dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc2(uint32_t taddr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols) : "memory");
}
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
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&r)[32]) {
  uint32_t* u = reinterpret_cast<uint32_t*>(r);
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
// Bounded wait on a barrier phase, the thread suspended in hardware meanwhile
// (spinning warps cost power that the tensor cores could use).  False after
// the limit, or once another role of the CTA has given up.
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
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// z = v where y == j, as a select (the compiler would index the 32 values
// through local memory).
__device__ __forceinline__ void pick(float& z, float v, int y, int j) {
  asm("{\n  .reg .pred p;\n  setp.eq.s32 p, %2, %3;\n  selp.f32 %0, %1, %0, p;\n}" : "+f"(z) : "f"(v), "r"(y), "r"(j));
}
// Rare branches of the epilogue: kept as branches, not as 32 selects a chunk.
__device__ __forceinline__ void keep_branch() { asm volatile("" ::: "memory"); }
__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

// ------------------------------------------------------------------ tiles --
struct Tile {
  int mode, rt, ct, kt, split;
  int s0, steps;  // 64-wide steps of the contraction
  int N;          // columns of the pair's tile
};

// Units are numbered long tiles first (DX / DW by length), then STATS or
// GRAD tiles in groups of 32 row tiles, rows fastest: the rows of a group
// stay in L2 while the class tiles pass.
struct Plan {
  int nl, nrt;
  int64_t ndx, ndw, units;
};

__device__ __forceinline__ Plan make_plan(const Args& p) {
  Plan q;
  q.nl = *p.nl;
  q.nrt = (q.nl + kTile - 1) / kTile;
  q.ndx = p.do_dx ? (int64_t)q.nrt * p.nkt * p.dxs : 0;
  q.ndw = p.do_dw ? (int64_t)p.ptiles * p.nkt * p.dws : 0;
  q.units = q.ndx + q.ndw + (int64_t)q.nrt * (p.gtiles + p.stats_units);
  return q;
}

// the tiles of unit u: `sub` counts them from 0; false past the last one
__device__ __forceinline__ bool get_tile(const Args& p, const Plan& q, int64_t u, int sub, Tile& t) {
  const int64_t nfirst = p.dw_first ? q.ndw : q.ndx;
  const bool out = u < q.ndx + q.ndw;
  if (out) {
    if (sub > 0) return false;
    const bool dw = (u < nfirst) == (p.dw_first != 0);
    const int i = (int)(u < nfirst ? u : u - nfirst);
    t.mode = dw ? DW : DX;
    t.N = p.NK;
    t.kt = i % p.nkt;
    const int splits = dw ? p.dws : p.dxs;
    t.split = i / p.nkt % splits;
    t.rt = t.ct = i / p.nkt / splits;
    const int total = dw ? (q.nl + 63) / 64 : p.psteps;
    const int per = (total + splits - 1) / splits;
    t.s0 = min(total, t.split * per);
    t.steps = min(total, t.s0 + per) - t.s0;
    return true;
  }
  int64_t i = u - q.ndx - q.ndw;
  const int nc = p.gtiles + p.stats_units;
  const int64_t per = (int64_t)32 * nc;
  const int g = (int)(i / per), rem = (int)(i % per);
  const int rows = min(32, q.nrt - g * 32);
  t.rt = g * 32 + rem % rows;
  const int c = rem / rows;
  t.kt = t.split = t.s0 = 0;
  t.steps = (p.k + 63) / 64;
  t.N = p.NT;
  if (p.stats_units > 0) {
    t.mode = STATS;
    t.ct = c * p.stats_run + sub;
    return sub < p.stats_run && t.ct < p.stats_tiles;
  }
  t.mode = p.full ? WHOLE : GRAD;
  t.ct = c;
  return sub == 0;
}

// One role's view of the posted units.
struct Feed {
  uint64_t* full;
  uint32_t empty0;   // slot 0's release barrier in the even CTA (cluster address)
  volatile int* unit;
  int slot = 0;
  uint32_t phase = 0;
  // next unit, or -1 at the end (or after a wait that gave up)
  __device__ __forceinline__ int next(volatile int* abort, int* err, int64_t units) {
    if (!wait(&full[slot], phase, abort, err, 21)) return -1;
    const int u = unit[slot];
    // Behind the last unit nothing is posted, and its slot is not given back.
    // The branch on u is also what keeps the arrival behind the read: the
    // arrival alone would not wait for it, and with shared memory's queue full
    // of an epilogue's global accesses the next unit could overtake the read
    // (the odd CTA's, whose slots another SM fills).
    if (u >= units) return -1;
    arrive_cluster(empty0 + slot * 8);
    if (++slot == kSlots) {
      slot = 0;
      phase ^= 1;
    }
    return u;
  }
};

// --------------------------------------------------------------- epilogue --
// Exponentials are 2^(z L - r) with L = log2(e) in fp32 and an integer r, the
// running maximum of ceil(z L): the fused multiply-add rounds the small
// difference only, rescaling a sum by 2^(r - r') is exact, and L's own error
// (below 2^-26 relative) acts as a change of the logits by that much.
// Where z L is beyond 2^30, its neighbours are 64 and more away and r would be
// off by up to half of that (an exponent of 128 is infinite).  There distinct
// logits are further apart than any exponential holds, and 4^(z - max z) does
// as well: 2^(z M - r) with M = 2 and r = 2 max z, both exact.  r stays
// increasing in max z, and tells by its size which of the two it is.
constexpr float kFar = 1073741824.0f;
__device__ __forceinline__ float ref_of(float top) {
  const float r = top * kLog2e;
  return fabsf(r) < kFar ? ceilf(r) : 2.0f * top;
}
__device__ __forceinline__ float scale_of(float r) { return fabsf(r) < kFar ? kLog2e : 2.0f; }

// This adds 32 more logits to (r, s = sum of 2^(z M - r)); limit: columns of
// the chunk that are classes.
__device__ __forceinline__ void online(float (&v)[32], int limit, float& r, float& s) {
  if (limit < 32) {
    keep_branch();
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j >= limit) v[j] = neg_inf();
  }
  float c[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) c[j] = v[j];
#pragma unroll
  for (int j = 4; j < 28; j += 8)
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = max3(c[i], v[j + 2 * i], v[j + 2 * i + 1]);
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = fmaxf(c[i], v[28 + i]);
  const float rn = fmaxf(r, ref_of(fmaxf(max3(c[0], c[1], c[2]), c[3])));
  // every logit so far -inf: exponentials of -inf - 0, which are zeros
  const float ref = rn == neg_inf() ? 0.0f : rn;
  const float sc = scale_of(ref);
  const float2 m2 = make_float2(sc, sc), nref = make_float2(-ref, -ref);
  float2 a[2] = {make_float2(s * ex2(r - ref), 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
  for (int j = 0; j < 32; j += 2) {
    const float2 x = fma2(make_float2(v[j], v[j + 1]), m2, nref);
    a[(j >> 1) & 1] = add2(a[(j >> 1) & 1], make_float2(ex2(x.x), ex2(x.y)));
  }
  a[0] = add2(a[0], a[1]);
  s = a[0].x + a[0].y;
  r = rn;
}

// A row's values from its r and sum: the loss is taken from the label's logit
// zlab in the form the sum has it, z M - r.
struct RowNorm {
  float ref, ws, glab, loss, lse;  // r; weight / sum; G of the label
};
__device__ __forceinline__ RowNorm norm_of(float ref, float s, float zlab, float weight) {
  RowNorm f;
  const float sc = scale_of(ref), l2 = log2f(s), zl = __fmaf_rn(zlab, sc, -ref);
  const bool far = sc == 2.0f;
  f.ref = ref;
  f.ws = weight / s;
  f.glab = __fmaf_rn(ex2(zl), f.ws, -weight);
  f.loss = far ? __fmaf_rn(-0.5f, zl, l2 * kLn2) : kLn2 * (l2 - zl);
  f.lse = __fmaf_rn(ref, far ? 0.5f : kLn2, l2 * kLn2);
  return f;
}
// entry j of a lane's 128-byte row of a G box
__device__ __forceinline__ void put_box(uint8_t* row, int lane, unsigned j, __nv_bfloat16 v) {
  *reinterpret_cast<__nv_bfloat16*>(row + 16 * ((j >> 3) ^ (lane & 7)) + 2 * (j & 7)) = v;
}

// Instantiated for the kinds of tiles a launch can hold, since the code of
// the others would cost instruction fetches (STATS of 16,384 x 256 x 131,072:
// 0.83 ms with all in one kernel, 0.78 ms alone, before the label's logit and
// the far references came in: 0.80).
enum Kind { LOSSES, PIECE, ONE_TILE };  // STATS | GRAD, DX, DW | WHOLE

template <int KIND>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    xent_tiles_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Args p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* stg_all = smem + kStages * kStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(stg_all + kEpiWarps * kStg);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* ufull = tempty + 2;
  uint64_t* uempty = ufull + kSlots;
  int* unit = reinterpret_cast<int*>(uempty + kSlots);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(unit + kSlots);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t cr = cluster_rank();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], KIND == ONE_TILE ? kEpiWarps : 2 * kEpiWarps);
    }
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&ufull[s], 1);
      mbar_init(&uempty[s], kConsumers);
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
  const Plan q = make_plan(p);
  Feed feed;
  feed.full = ufull;
  feed.empty0 = mapa(smem_u32(uempty), 0);
  feed.unit = unit;

  if (warp == 0) {
    if (lane == 0) {
      const CUtensorMap* xk = &maps.xk[q.nl < p.n];
      const CUtensorMap* xm = &maps.xm[q.nl < p.n];
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      while (ok) {
        const int u = feed.next(abort, p.err, q.units);
        if (u < 0) break;
        Tile t;
        for (int sub = 0; ok && get_tile(p, q, u, sub, t); ++sub) {
          const int hn = t.N / 2;
          const uint32_t bytes = kStageA + (uint32_t)hn * 128;
          for (int s = 0; s < t.steps; ++s) {
            if (!(ok = wait(&empty[stage], phase ^ 1, abort, p.err, 22))) break;
            const uint32_t a = smem_u32(smem + stage * kStageBytes), b = a + kStageA;
            const uint32_t bar = mapa(smem_u32(&full[stage]), 0);
            if (cr == 0) mbar_expect_tx(&full[stage], 2 * bytes);
            const int x = (t.s0 + s) * 64;
            if (KIND != PIECE || t.mode <= WHOLE) {
              const int c0 = (t.mode == STATS ? 0 : p.gc0) + t.ct * p.NT;
              tma_load_pair(a, xk, x, t.rt * kTile + cr * 128, bar);
              tma_load_pair(b, &maps.wk, x, c0 + cr * hn, bar);
            } else {
              const CUtensorMap* bm = t.mode == DX ? &maps.wm : xm;
              const int y = t.mode == DX ? p.pc0 + x : x;
              if (t.mode == DX) {
                tma_load_pair(a, &maps.gk, 0, (t.s0 + s) * (int)p.npad + t.rt * kTile + cr * 128, bar);
              } else {
                const int gy = (t.ct * 4 + cr * 2) * (int)p.npad + x;
                tma_load_pair(a, &maps.gm, 0, gy, bar);
                tma_load_pair(a + 8192, &maps.gm, 0, gy + (int)p.npad, bar);
              }
              for (int j = 0; j < hn; j += 64) tma_load_pair(b + j * 128, bm, t.kt * p.NK + cr * hn + j, y, bar);
            }
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1;
            }
          }
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && cr == 0) {
      int stage = 0, i = 0;
      uint32_t phase = 0;
      bool ok = true;
      while (ok) {
        const int u = feed.next(abort, p.err, q.units);
        if (u < 0) break;
        Tile t;
        for (int sub = 0; ok && get_tile(p, q, u, sub, t); ++sub, ++i) {
          const int a = i & 1;
          if (!(ok = wait(&tempty[a], ((i >> 1) & 1) ^ 1, abort, p.err, 23))) break;
          tc_fence_after();
          const uint32_t d = tmem + a * 256;
          const int amn = KIND == PIECE && t.mode == DW, bmn = KIND == PIECE && t.mode >= DX;
          const uint32_t idesc = idesc_bf16_f32(256, t.N, amn, bmn);
          // 16 contraction elements further: 32 bytes along a K-major row,
          // two 8-row swizzle atoms in an MN-major block
          const uint32_t as = amn ? 2048 : 32, bs = bmn ? 2048 : 32;
          const uint32_t al = amn ? 8192 : 16, bl = bmn ? 8192 : 16;  // next 64-wide MN-major block
          for (int s = 0; s < t.steps; ++s) {
            if (!(ok = wait(&full[stage], phase, abort, p.err, 24))) break;
            tc_fence_after();
            const uint32_t ab = smem_u32(smem + stage * kStageBytes), bb = ab + kStageA;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_pair(d, smem_desc_sw128(ab + as * kk, al, 1024), smem_desc_sw128(bb + bs * kk, bl, 1024), idesc,
                        (s | kk) != 0);
            commit_pair(&empty[stage]);
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1;
            }
          }
          if (ok) commit_pair(&tfull[a]);
        }
      }
    }
  } else if (warp < 2 + kEpiWarps) {
    const int quarter = warp & 3, part = (warp - 2) >> 2;
    const int rit = cr * 128 + quarter * 32 + lane;  // row of the pair's tile
    uint8_t* stg = stg_all + (warp - 2) * kStg;
    const uint32_t tempty0 = mapa(smem_u32(tempty), 0);
    int i = 0, nbox = 0;
    bool ok = true;
    // one unit ahead: its rows' values are on their way while the current
    // unit is worked on
    int un = 0;
    float4 rwn;
    auto fetch = [&]() {
      if (lane == 0) un = feed.next(abort, p.err, q.units);
      un = __shfl_sync(gq::FULL, un, 0);
      rwn = make_float4(0.0f, 0.0f, 0.0f, __int_as_float(-1));
      if (un < 0) return;
      Tile t;
      get_tile(p, q, un, 0, t);
      const int row = t.rt * kTile + rit;
      if (row < q.nl) {
        if (KIND == PIECE && t.mode == GRAD) rwn = p.row[row];
        if (KIND == LOSSES) rwn.w = __int_as_float(p.lab[row]);
        if (KIND == ONE_TILE)
          rwn = make_float4(0.0f, p.wrow[row], __int_as_float(p.idx[row]), __int_as_float(p.lab[row]));
      }
    };
    fetch();
    while (ok && un >= 0) {
      const int u = un;
      float4 rw = rwn;
      fetch();
      Tile t;
      float m = neg_inf(), sum = 0.0f;
      for (int sub = 0; ok && get_tile(p, q, u, sub, t); ++sub, ++i) {
        const int srow = t.rt * kTile + rit;
        const int a = i & 1;
        // a WHOLE tile belongs to one of the two warps of its rows, which
        // take tiles by turns: a lane holds all of its row's classes
        if (KIND == ONE_TILE && a != part) continue;
        int got = 1;
        if (lane == 0) got = wait(&tfull[a], (i >> 1) & 1, abort, p.err, 25);
        ok = __shfl_sync(gq::FULL, got, 0) != 0;
        if (!ok) break;
        tc_fence_after();
        const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + a * 256;
        if (KIND != PIECE) {
          float zl = 0.0f;
          const int lab = __float_as_int(rw.w);
          // most tiles hold the label of none of a warp's rows
          const bool hit = KIND == ONE_TILE || __any_sync(gq::FULL, (unsigned)(lab - t.ct * p.NT) < (unsigned)t.N);
          for (int c = KIND == ONE_TILE ? 0 : part * 32; c < t.N; c += KIND == ONE_TILE ? 32 : 32 * kParts) {
            float v[32];
            tmem_ld32(taddr + c, v);
            tmem_ld_wait();
            const int c0 = t.ct * p.NT + c;  // class of v[0]
            if (KIND == ONE_TILE || (hit && __any_sync(gq::FULL, (unsigned)(lab - c0) < 32u))) {
              if (KIND != ONE_TILE) keep_branch();
#pragma unroll
              for (int j = 0; j < 32; ++j) pick(zl, v[j], lab - c0, j);
              if (KIND == LOSSES && (unsigned)(lab - c0) < 32u) p.zlab[srow] = zl;
            }
            if (c0 < p.C) online(v, p.C - c0, m, sum);
          }
          if (KIND == ONE_TILE) {
            const RowNorm f = norm_of(m == neg_inf() ? 0.0f : m, sum, zl, rw.y);
            if (srow < q.nl) {
              const int to = __float_as_int(rw.z);
              if (p.loss != nullptr) p.loss[to] = f.loss;
              if (p.lse != nullptr) p.lse[to] = f.lse;
              rw = make_float4(f.ref, f.ws, f.glab, rw.w);
            }
          }
        }
        if ((KIND == PIECE && t.mode == GRAD) || (KIND == ONE_TILE && p.full == 2)) {
          const float sc = scale_of(rw.x);
          const bool hit =
              KIND == PIECE &&
              __any_sync(gq::FULL, (unsigned)(__float_as_int(rw.w) - p.gc0 - t.ct * p.NT) < (unsigned)t.N);
          for (int b = KIND == ONE_TILE ? 0 : part * 64; b < t.N; b += KIND == ONE_TILE ? 64 : 64 * kParts) {
            // a box of 32 rows x 64 classes, 128 bytes a row (128-byte
            // swizzle: 16-byte piece j of row `lane` at j ^ (lane & 7))
            uint8_t* box = stg + (nbox & 1) * kBox;
            uint8_t* mine = box + lane * 128;
            const int cl = t.ct * p.NT + b;  // column of G
            const int c0 = p.gc0 + cl;
            const unsigned yl = (unsigned)(__float_as_int(rw.w) - c0);
            float gl = rw.z;  // the label's entry, if it is here
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
              float v[32];
              tmem_ld32(taddr + b + 32 * h, v);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 32; j += 2) {
                const float2 x =
                    fma2(make_float2(v[j], v[j + 1]), make_float2(sc, sc), make_float2(-rw.x, -rw.x));
                const float2 g = mul2(make_float2(ex2(x.x), ex2(x.y)), make_float2(rw.y, rw.y));
                v[j] = g.x;
                v[j + 1] = g.y;
              }
              if (hit && __any_sync(gq::FULL, yl - 32 * h < 32u)) {
                keep_branch();
                float pw = 0.0f;
#pragma unroll
                for (int j = 0; j < 32; ++j) pick(pw, v[j], (int)yl - 32 * h, j);
                if (yl - 32 * h < 32u) gl = pw - rw.z;
              }
              if (h == 0) {
                if (lane == 0) bulk_wait_read<1>();  // the store of two boxes ago has read this buffer
                __syncwarp();
              }
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                uint32_t o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = pack_bf16x2(v[8 * j + 2 * e], v[8 * j + 2 * e + 1]);
                *reinterpret_cast<uint4*>(mine + 16 * ((4 * h + j) ^ (lane & 7))) = make_uint4(o[0], o[1], o[2], o[3]);
              }
            }
            // entries that are not the product's: the label's, p - 1 in fp32,
            // and zeros past the last class and row, whatever the products
            // gave there
            if (yl < 64u) put_box(mine, lane, yl, __float2bfloat16_rn(gl));
            const int zeros = srow < q.nl ? p.C - c0 : 0;
#pragma unroll 1
            for (int j = max(zeros, 0); j < 64; ++j) put_box(mine, lane, j, __float2bfloat16_rn(0.0f));
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&maps.gst, box, 0, (cl >> 6) * (int)p.npad + t.rt * kTile + cr * 128 + quarter * 32);
              bulk_commit();
            }
            ++nbox;
          }
        }
        if (KIND == PIECE && t.mode >= DX) {
          const bool dw = t.mode == DW;
          // fp32 sums that other pieces or splits add to, else the result
          const bool sums = dw ? p.dws > 1 : p.dxs > 1 || !p.last;
          const bool add = !dw && !p.first;
          float* acc = nullptr;
          if (sums || add) {
            const int64_t tile = dw ? (int64_t)t.split * p.ptiles + t.ct : (int64_t)t.split * (p.npad / kTile) + t.rt;
            acc = (dw ? p.accW : p.accX) + (tile * p.nkt + t.kt) * ((int64_t)p.NK * kTile) + rit;
          }
          // rows of the result that follow one another are stored by TMA in
          // boxes of 64 columns; rows scattered among unlabelled ones, and
          // rows whose last 16 bytes are not all theirs (a bulk store would
          // write them), by plain stores.  Either way row `lane` of the
          // staging is 128 bytes, 16-byte piece j at j ^ (lane & 7)
          const bool apart = (!dw && q.nl < p.n) || (p.k & 7) != 0;
          const int r = (dw ? t.ct : t.rt) * kTile + rit;
          int64_t orow = -1;  // row of the result that this lane's sums belong to
          if (apart) {
            if (dw) orow = p.pc0 + r < p.C ? p.pc0 + r : -1;
            else if (r < q.nl) orow = q.nl < p.n ? p.idx[r] : r;
          }
          auto load = [&](int c, float (&v)[32]) {
            if (t.steps > 0) {
              tmem_ld32(taddr + c, v);
              tmem_ld_wait();
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = 0.0f;
            }
            if (add) {  // sums so far are unscaled
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] += acc[(c + j) * kTile];
            }
          };
          for (int b = part * 64; b < t.N; b += 64 * kParts) {
            const int k0 = t.kt * p.NK + b;
            if (!sums && k0 >= p.k) break;
            uint8_t* box = stg + (nbox & 1) * kBox;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
              float v[32];
              load(b + 32 * h, v);
              if (sums) {
#pragma unroll
                for (int j = 0; j < 32; ++j) acc[(b + 32 * h + j) * kTile] = v[j];
                continue;
              }
              if (h == 0) {
                if (lane == 0) bulk_wait_read<1>();
                __syncwarp();
              }
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                uint32_t o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  o[e] = pack_bf16x2(v[8 * j + 2 * e] * p.scale, v[8 * j + 2 * e + 1] * p.scale);
                *reinterpret_cast<uint4*>(box + lane * 128 + 16 * ((4 * h + j) ^ (lane & 7))) =
                    make_uint4(o[0], o[1], o[2], o[3]);
              }
            }
            if (sums) continue;
            ++nbox;
            if (!apart) {
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                const int y = (dw ? p.pc0 + t.ct * kTile : t.rt * kTile) + cr * 128 + quarter * 32;
                if (y < (dw ? p.C : q.nl)) tma_store_2d(dw ? &maps.ow : &maps.ox, box, k0, y);
                bulk_commit();
              }
              continue;
            }
            if (lane == 0) bulk_commit();  // an empty group: this box has no bulk store to wait for
            __syncwarp();
#pragma unroll
            for (int it = 0; it < 8; ++it) {
              const int rr = it * 4 + (lane >> 3), j = lane & 7;
              const uint4 o = *reinterpret_cast<const uint4*>(box + rr * 128 + 16 * (j ^ (rr & 7)));
              const int64_t to = __shfl_sync(gq::FULL, orow, rr);
              if (to < 0) continue;
              const int col = k0 + 8 * j;
              __nv_bfloat16* dst = (dw ? p.dW + to * p.lddw : p.dX + to * p.lddx) + col;
              if (col + 8 <= p.k) {
                *reinterpret_cast<uint4*>(dst) = o;
              } else {
                const uint32_t e[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
                for (int x = 0; x < 8; ++x)
                  if (col + x < p.k) dst[x] = __ushort_as_bfloat16((unsigned short)(e[x >> 1] >> (16 * (x & 1))));
              }
            }
            __syncwarp();
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(tempty0 + a * 8);
        if (KIND == LOSSES && (sub + 1 == p.stats_run || t.ct + 1 == p.stats_tiles))
          p.part[(int64_t)(t.ct / p.stats_run * kParts + part) * p.npad + srow] = make_float2(m, sum);
      }
    }
    if (lane == 0) bulk_wait<0>();  // every TMA store of this warp done
  } else if (lane == 0 && cr == 0) {
    int slot = 0;
    uint32_t phase = 0;
    while (wait(&uempty[slot], phase ^ 1, abort, p.err, 26)) {
      const int64_t next = atomicAdd(p.counter, 1);
      const int u = next < q.units ? (int)next : 0x7fffffff;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint32_t bar = mapa(smem_u32(&ufull[slot]), r);
        expect_cluster(bar, 4);
        st_async(mapa(smem_u32(&unit[slot]), r), u, bar);
      }
      if (u == 0x7fffffff) break;
      if (++slot == kSlots) {
        slot = 0;
        phase ^= 1;
      }
    }
  }
  __syncwarp();
  __syncthreads();
  // after a wait that gave up: loads, products and posts under way (they take
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

// ------------------------------------------------------- rows with a label --
// The labelled rows in order.  Blocks take consecutive segments: a first
// kernel counts, the second sums the counts before its segment and numbers.
constexpr int kScanThreads = 1024;

__device__ __forceinline__ bool labelled(int y, int C) { return (unsigned)y < (unsigned)C; }

__global__ void __launch_bounds__(kScanThreads) xent_count_kernel(const int* __restrict__ labels, int64_t n, int C,
                                                                 int64_t seg, int* cnt) {
  __shared__ int s;
  if (threadIdx.x == 0) s = 0;
  __syncthreads();
  const int64_t e = min(n, (blockIdx.x + 1) * seg);
  int c = 0;
  for (int64_t r = blockIdx.x * seg + threadIdx.x; r < e; r += kScanThreads) c += labelled(labels[r], C);
  c = __reduce_add_sync(gq::FULL, c);
  if ((threadIdx.x & 31) == 0) atomicAdd(&s, c);  // integers: the order does not matter
  __syncthreads();
  if (threadIdx.x == 0) cnt[blockIdx.x] = s;
}

struct ScanOut {
  int* nl;
  int* pos;       // row of X -> labelled row, or -1
  int* idx;
  int* lab;
  float* wrow;
  float* loss;
  float* lse;
  int* counters;  // of the tile launches, zeroed here
  int n_counters;
};

__global__ void __launch_bounds__(kScanThreads)
    xent_scan_kernel(const int* labels, const float* weight, int64_t n, int C, int64_t seg, const int* cnt,
                     const ScanOut o) {
  grid_wait();
  __shared__ int ws[32];
  __shared__ int base;
  if (threadIdx.x == 0) base = 0;
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x > 0) {
    int c = 0;
    for (int b = threadIdx.x; b < (int)blockIdx.x; b += kScanThreads) c += cnt[b];
    c = __reduce_add_sync(gq::FULL, c);
    if (lane == 0) atomicAdd(&base, c);
    __syncthreads();
  } else {
    for (int j = threadIdx.x; j < o.n_counters; j += kScanThreads) o.counters[j] = 0;
  }
  const int64_t b0 = blockIdx.x * seg, e = min(n, b0 + seg);
  int at = base;
  for (int64_t r0 = b0; r0 < e; r0 += kScanThreads) {
    const int64_t r = r0 + threadIdx.x;
    const int y = r < e ? labels[r] : -1;
    const bool on = labelled(y, C);
    const unsigned bal = __ballot_sync(gq::FULL, on);
    if (lane == 0) ws[warp] = __popc(bal);
    __syncthreads();
    const int mine = ws[lane];
    const int before = __reduce_add_sync(gq::FULL, lane < warp ? mine : 0);
    const int all = __reduce_add_sync(gq::FULL, mine);
    if (r < e) {
      const int to = on ? at + before + __popc(bal & ((1u << lane) - 1)) : -1;
      o.pos[r] = to;
      if (on) {
        o.idx[to] = (int)r;
        o.lab[to] = y;
        o.wrow[to] = weight != nullptr ? weight[r] : 1.0f;
      } else {
        if (o.loss != nullptr) o.loss[r] = 0.0f;
        if (o.lse != nullptr) o.lse[r] = 0.0f;
      }
    }
    at += all;
    __syncthreads();
  }
  if (blockIdx.x == gridDim.x - 1 && threadIdx.x == 0) *o.nl = at;
}

// Unless every row is labelled: the labelled rows of X copied together (zeros
// up to a multiple of 256 rows) and zeros in the other rows of dX.
__global__ void __launch_bounds__(256)
    xent_rows_kernel(const __nv_bfloat16* X, int64_t n, int k, int64_t ldx, const int* pos, const int* nl,
                     __nv_bfloat16* Xc, int64_t ldc, __nv_bfloat16* dX, int64_t lddx, int per_warp) {
  grid_wait();
  const int m = *nl;
  if (m == n) return;
  const int lane = threadIdx.x & 31;
  const int64_t pad_end = n + ((m + kTile - 1) / kTile * (int64_t)kTile - m);  // rows of zeros behind Xc
  const int64_t step = (int64_t)gridDim.x * 8 * per_warp;
  for (int64_t r0 = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * per_warp; r0 < pad_end; r0 += step) {
    // per_warp rows (at most 32) of a warp, their places read at once
    const int64_t mine = r0 + lane;
    const int at = lane < per_warp && mine < n ? pos[mine] : -1;
    const unsigned on = __ballot_sync(gq::FULL, at >= 0);
    for (int i = 0; i < per_warp && r0 + i < pad_end; ++i) {  // zeros
      const int64_t r = r0 + i;
      if (on >> i & 1) continue;
      __nv_bfloat16* dst = r >= n ? Xc + (m + (r - n)) * ldc : dX != nullptr ? dX + r * lddx : nullptr;
      if (dst == nullptr) continue;
      for (int c = lane * 8; c < k; c += 256) {
        if (c + 8 <= k) *reinterpret_cast<uint4*>(dst + c) = make_uint4(0, 0, 0, 0);
        else
          for (int j = c; j < k; ++j) dst[j] = __float2bfloat16_rn(0.0f);
      }
    }
    for (unsigned left = on; left != 0; left &= left - 1) {
      const int i = __ffs(left) - 1;
      const __nv_bfloat16* x = X + (r0 + i) * ldx;
      __nv_bfloat16* dst = Xc + (int64_t)__shfl_sync(gq::FULL, at, i) * ldc;
      for (int c = lane * 8; c < k; c += 256) {
        if (c + 8 <= k) *reinterpret_cast<uint4*>(dst + c) = __ldg(reinterpret_cast<const uint4*>(x + c));
        else
          for (int j = c; j < k; ++j) dst[j] = x[j];
      }
    }
  }
}

// lse and loss of 32 labelled rows per block from the runs' (r, sum) pairs:
// 32 lanes of runs per row, joined in lane order.
__global__ void __launch_bounds__(1024)
    xent_join_kernel(const float2* part, int runs, int64_t npad, const int* nl, const int* idx, const float* zlab,
                     const float* wrow, const int* lab, float4* rowinfo, float* loss, float* lse) {
  __shared__ float sm[32][33], ss[32][33];
  grid_wait();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int rows = *nl;
  for (int64_t r0 = (int64_t)blockIdx.x * 32; r0 < rows; r0 += (int64_t)gridDim.x * 32) {
    const int64_t row = r0 + lane;
    float r = neg_inf(), s = 0.0f;
    for (int u = w; u < runs; u += 32) {
      const float2 v = part[(int64_t)u * npad + row];
      const float rn = fmaxf(r, v.x), ref = rn == neg_inf() ? 0.0f : rn;
      s = s * ex2(r - ref) + v.y * ex2(v.x - ref);
      r = rn;
    }
    sm[w][lane] = r;
    ss[w][lane] = s;
    __syncthreads();
    if (w == 0 && row < rows) {
      for (int j = 1; j < 32; ++j) r = fmaxf(r, sm[j][lane]);
      const float ref = r == neg_inf() ? 0.0f : r;
      s = 0.0f;
      for (int j = 0; j < 32; ++j) s += ss[j][lane] * ex2(sm[j][lane] - ref);
      const RowNorm f = norm_of(ref, s, zlab[row], wrow[row]);
      if (rowinfo != nullptr) rowinfo[row] = make_float4(f.ref, f.ws, wrow[row], __int_as_float(lab[row]));
      const int to = idx[row];
      if (loss != nullptr) loss[to] = f.loss;
      if (lse != nullptr) lse[to] = f.lse;
    }
    __syncthreads();
  }
}

// Sums of the splits in order -> bf16 rows.  A block: 256 rows of one tile,
// COLS columns: 8, a whole 16-byte store per row, or 2 where so few blocks
// would leave SMs idle.
template <int COLS>
__global__ void __launch_bounds__(256)
    xent_sum_kernel(const float* acc, int splits, int64_t split_stride, int64_t tile_stride, const int* nl, int64_t n,
                    const int* idx, int row0, int C, int k, float scale, __nv_bfloat16* out, int64_t ldo) {
  grid_wait();
  const int c0 = blockIdx.y * COLS;
  const int64_t r = (int64_t)blockIdx.x * kTile + threadIdx.x;
  int64_t to;
  if (idx != nullptr) {
    if (r >= *nl) return;
    to = *nl < n ? idx[r] : r;
  } else {
    to = row0 + r;
    if (to >= C) return;
  }
  const float* a = acc + blockIdx.x * tile_stride + (int64_t)c0 * kTile + threadIdx.x;
  float v[COLS] = {};
#pragma unroll 8
  for (int s = 0; s < splits; ++s)
#pragma unroll
    for (int j = 0; j < COLS; ++j) v[j] += a[s * split_stride + j * kTile];
#pragma unroll
  for (int j = 0; j < COLS; ++j) v[j] *= scale;
  __nv_bfloat16* dst = out + to * ldo + c0;
  if (COLS == 8 && c0 + 8 <= k) {
    *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                pack_bf16x2(v[4 % COLS], v[5 % COLS]),
                                                pack_bf16x2(v[6 % COLS], v[7 % COLS]));
  } else {
#pragma unroll
    for (int j = 0; j < COLS; ++j)
      if (c0 + j < k) dst[j] = __float2bfloat16_rn(v[j]);
  }
}

// ------------------------------------------------------------------- host --
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

// bf16 [outer][inner] of row pitch ld: boxes of 64 x bo (128-byte rows), zeros
// out of bounds
int tmap(CUtensorMap* m, const void* base, int64_t inner, int64_t outer, int64_t ld, int bo) {
  auto fn = encode_fn();
  if (fn == nullptr) return GQ_ERR_CUDA;
  const cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)outer};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)bo};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r =
      fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? GQ_OK : GQ_ERR_INVALID_ARG;
}

int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Bytes of one buffer of G.  Long pieces keep the sums of DX long and the
// launches few: 128 MB 5.8 ms, 512 MB 5.0 ms, 2 GB 4.9 ms on the first version
// of 16,384 x 256 x 131,072; 1 GB is within 1% of 2 GB.
constexpr int64_t kPieceBytes = (int64_t)1024 << 20;

struct Sizes {
  int64_t npad, nrt;
  int clusters;
  int NT, ctiles;             // class tile width and tiles
  int NK, nkt;
  int run, units;             // STATS
  int per_piece, pieces;      // class tiles of a piece; pieces
  int64_t Cp;                 // classes of a piece
  int dxs, dws;
  int scan_blocks;
  int64_t seg;
};

Sizes make_sizes(int64_t n, int k, int C, bool grad) {
  Sizes z{};
  z.npad = up(n, kTile);
  z.nrt = z.npad / kTile;
  z.clusters = sm_count() / 2 > 0 ? sm_count() / 2 : 1;
  z.NT = (int)up(cdiv(C, cdiv(C, kTile)), 64);
  z.ctiles = (int)cdiv(C, z.NT);
  z.NK = (int)up(cdiv(k, cdiv(k, kTile)), 128);
  z.nkt = (int)cdiv(k, z.NK);
  // runs of class tiles per row tile: long runs leave few pairs to join,
  // about eight units per CTA pair leave a short tail
  int64_t run = z.nrt * z.ctiles / (8 * z.clusters);
  z.run = (int)(run < 1 ? 1 : run > 16 ? 16 : run);
  z.units = (int)cdiv(z.ctiles, z.run);
  z.seg = up(cdiv(n, 256), kScanThreads);
  z.scan_blocks = (int)cdiv(n, z.seg);
  if (!grad) return z;
  int64_t t = kPieceBytes / (z.npad * z.NT * 2);
  t = t < 1 ? 1 : t > z.ctiles ? z.ctiles : t;
  z.per_piece = (int)cdiv(z.ctiles, cdiv(z.ctiles, t));  // pieces of nearly equal size
  z.pieces = (int)cdiv(z.ctiles, z.per_piece);
  z.Cp = (int64_t)z.per_piece * z.NT;
  // Long sums are split where a launch would otherwise wait for them: no
  // tile longer than a CTA pair's share of the launch, none below 32 steps
  // (a split writes and reads 256 x NK fp32 sums, about 16 steps' time).
  const int64_t sx = z.Cp / 64, sw = z.npad / 64, ptiles = cdiv(z.Cp, kTile);
  const int64_t total = z.nrt * z.nkt * sx + ptiles * z.nkt * sw + (z.pieces > 1 ? z.nrt * z.per_piece * cdiv(k, 64) : 0);
  int64_t share = total / z.clusters;
  if (share < 32) share = 32;
  z.dxs = (int)cdiv(sx, share);
  z.dws = (int)cdiv(sw, share);
  return z;
}

struct Ws {
  int* nl;
  int* counters;
  int n_counters;
  int *cnt, *pos, *idx, *lab;
  float *wrow, *zlab;
  float4* row;
  float2* part;
  void* Xc;
  void* G[2];
  float *accX, *accW;
};

Carve carve(void* ws, size_t bytes, const Sizes& z, int64_t n, int k, bool grad, Ws& w) {
  Carve c(ws, bytes);
  w.n_counters = 2 + (grad ? z.pieces : 0);
  w.nl = static_cast<int*>(c.take(256));
  w.counters = static_cast<int*>(c.take((size_t)w.n_counters * 4));
  w.cnt = static_cast<int*>(c.take((size_t)z.scan_blocks * 4));
  w.pos = static_cast<int*>(c.take((size_t)n * 4));
  w.idx = static_cast<int*>(c.take((size_t)z.npad * 4));
  w.lab = static_cast<int*>(c.take((size_t)z.npad * 4));
  w.wrow = static_cast<float*>(c.take((size_t)z.npad * 4));
  w.Xc = c.take((size_t)z.npad * round8(k) * 2);
  if (z.ctiles > 1) {  // WHOLE tiles keep these to themselves
    w.zlab = static_cast<float*>(c.take((size_t)z.npad * 4));
    w.part = static_cast<float2*>(c.take((size_t)z.units * kParts * z.npad * sizeof(float2)));
    if (grad) w.row = static_cast<float4*>(c.take((size_t)z.npad * 16));
  }
  if (!grad) return c;
  w.G[0] = c.take((size_t)z.npad * z.Cp * 2);
  w.G[1] = z.pieces > 1 ? c.take((size_t)z.npad * z.Cp * 2) : w.G[0];
  const size_t tile = (size_t)z.nkt * z.NK * kTile * 4;
  if (z.pieces > 1 || z.dxs > 1) w.accX = static_cast<float*>(c.take(z.dxs * z.nrt * tile));
  if (z.dws > 1) w.accW = static_cast<float*>(c.take(z.dws * cdiv(z.Cp, kTile) * tile));
  return c;
}

int check_shape(int64_t n, int k, int C) {
  if (n < 0 || k < 1 || C < 1) return GQ_ERR_INVALID_ARG;
  if (n > (1 << 28) || C > (1 << 30) || k > 16384) return GQ_ERR_UNSUPPORTED;
  // units of one launch are numbered in 31 bits
  if (cdiv(n, kTile) * cdiv(C, 64) > INT32_MAX / 4) return GQ_ERR_UNSUPPORTED;
  return GQ_OK;
}

int launch_sum(int64_t tiles, const float* acc, int splits, int64_t split_stride, int64_t tile_stride, const int* nl,
               int64_t n, const int* idx, int row0, int C, int k, float scale, __nv_bfloat16* out, int64_t ldo,
               cudaStream_t s) {
  if (tiles * cdiv(k, 8) < 2 * sm_count())
    return launch_after(xent_sum_kernel<2>, dim3((unsigned)tiles, (unsigned)cdiv(k, 2)), dim3(256), 0, s, acc, splits,
                        split_stride, tile_stride, nl, n, idx, row0, C, k, scale, out, ldo);
  return launch_after(xent_sum_kernel<8>, dim3((unsigned)tiles, (unsigned)cdiv(k, 8)), dim3(256), 0, s, acc, splits,
                      split_stride, tile_stride, nl, n, idx, row0, C, k, scale, out, ldo);
}

template <int KIND>
int launch_kind(const Maps& m, const Args& a, const Sizes& z, cudaStream_t s) {
  GQ_TRY_CUDA(cudaFuncSetAttribute(xent_tiles_kernel<KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem));
  return launch_after(xent_tiles_kernel<KIND>, dim3(2 * z.clusters), dim3(kThreads), kSmem, s, m, a);
}

int launch_tiles(const Maps& m, Args& a, const Sizes& z, cudaStream_t s) {
  GQ_TRY(a.full ? launch_kind<ONE_TILE>(m, a, z, s)
                : a.stats_units > 0 ? launch_kind<LOSSES>(m, a, z, s) : launch_kind<PIECE>(m, a, z, s));
  ++a.counter;
  return GQ_OK;
}

}  // namespace
}  // namespace gq

using namespace gq;

extern "C" size_t gq_linear_xent_workspace_bytes(int64_t n, int k, int C, int need_grad) {
  if (check_shape(n, k, C) != GQ_OK || n == 0) return 0;
  Ws w{};
  return carve(nullptr, 0, make_sizes(n, k, C, need_grad != 0), n, k, need_grad != 0, w).used;
}

extern "C" int gq_linear_xent(const uint16_t* X, int64_t n, int k, int64_t ldx, const uint16_t* W, int C, int64_t ldw,
                              const int32_t* labels, const float* weight, float scale, float* loss, float* lse,
                              uint16_t* dX, int64_t lddx, uint16_t* dW, int64_t lddw, void* ws, size_t ws_bytes,
                              int* dev_err, gq_stream stream) {
  GQ_TRY(check_shape(n, k, C));
  auto s = (cudaStream_t)stream;
  if (dW != nullptr && (lddw < k || lddw % 8 || !aligned(dW, 16))) return GQ_ERR_INVALID_ARG;
  if (n == 0) {  // no rows: dW = 0
    if (dW != nullptr) GQ_TRY_CUDA(cudaMemset2DAsync(dW, (size_t)lddw * 2, 0, (size_t)k * 2, (size_t)C, s));
    return GQ_OK;
  }
  if (X == nullptr || W == nullptr || labels == nullptr || ldx < k || ldw < k || ldx % 8 || ldw % 8 ||
      !aligned(X, 16) || !aligned(W, 16) || !aligned(labels, 4) || !aligned(weight, 4) || !aligned(loss, 4) ||
      !aligned(lse, 4) || !aligned(dev_err, 4))
    return GQ_ERR_INVALID_ARG;
  if (dX != nullptr && (lddx < k || lddx % 8 || !aligned(dX, 16))) return GQ_ERR_INVALID_ARG;
  const bool grad = dX != nullptr || dW != nullptr;
  const Sizes z = make_sizes(n, k, C, grad);
  Ws w{};
  if (ws == nullptr || !aligned(ws, 256) || !carve(ws, ws_bytes, z, n, k, grad, w).ok()) return GQ_ERR_WORKSPACE;

  if (z.scan_blocks > 1) {
    xent_count_kernel<<<z.scan_blocks, kScanThreads, 0, s>>>(labels, n, C, z.seg, w.cnt);
    GQ_TRY(launch_status());
  }
  const ScanOut so{w.nl, w.pos, w.idx, w.lab, w.wrow, loss, lse, w.counters, w.n_counters};
  if (z.scan_blocks > 1)
    GQ_TRY(launch_after(xent_scan_kernel, dim3(z.scan_blocks), dim3(kScanThreads), 0, s, labels, weight, n, C, z.seg,
                        w.cnt, so));
  else
    xent_scan_kernel<<<1, kScanThreads, 0, s>>>(labels, weight, n, C, z.seg, w.cnt, so);
  GQ_TRY(launch_status());
  const int64_t ldc = round8(k);
  const int64_t warps = (int64_t)sm_count() * 64, share = cdiv(n + kTile, warps);
  const int per_warp = share > 32 ? 32 : (int)share;
  const int64_t rb = cdiv(n + kTile, 8 * per_warp);
  GQ_TRY(launch_after(xent_rows_kernel, dim3((unsigned)(rb < warps / 8 ? rb : warps / 8)), dim3(256), 0, s,
                      reinterpret_cast<const __nv_bfloat16*>(X), n, k, ldx, w.pos, w.nl,
                      static_cast<__nv_bfloat16*>(w.Xc), ldc, reinterpret_cast<__nv_bfloat16*>(dX), lddx, per_warp));

  Maps m;
  memset(&m, 0, sizeof(m));
  GQ_TRY(tmap(&m.xk[0], X, k, n, ldx, 128));
  GQ_TRY(tmap(&m.xk[1], w.Xc, k, z.npad, ldc, 128));
  GQ_TRY(tmap(&m.wk, W, k, C, ldw, z.NT / 2));
  Args a{};
  a.nl = w.nl;
  a.counter = w.counters;
  a.n = n;
  a.npad = z.npad;
  a.k = k;
  a.C = C;
  a.NT = z.NT;
  a.NK = z.NK;
  a.nkt = z.nkt;
  a.row = w.row;
  a.zlab = w.zlab;
  a.idx = w.idx;
  a.part = w.part;
  a.err = dev_err;
  a.wrow = w.wrow;
  a.lab = w.lab;
  a.loss = loss;
  a.lse = lse;
  const bool whole = z.ctiles == 1;
  if (whole) {
    a.full = grad ? 2 : 1;
    a.gtiles = 1;
    if (!grad) return launch_tiles(m, a, z, s);
  } else {
    a.stats_tiles = z.ctiles;
    a.stats_run = z.run;
    a.stats_units = z.units;
    GQ_TRY(launch_tiles(m, a, z, s));
    const int64_t jb = cdiv(n, 32), jcap = (int64_t)sm_count() * 2;
    GQ_TRY(launch_after(xent_join_kernel, dim3((unsigned)(jb < jcap ? jb : jcap)), dim3(1024), 0, s, w.part,
                        kParts * z.units, z.npad, w.nl, w.idx, w.zlab, w.wrow, w.lab, grad ? w.row : nullptr, loss,
                        lse));
    if (!grad) return GQ_OK;
    a.stats_units = 0;
  }

  GQ_TRY(tmap(&m.xm[0], X, k, n, ldx, 64));
  GQ_TRY(tmap(&m.xm[1], w.Xc, k, z.npad, ldc, 64));
  GQ_TRY(tmap(&m.wm, W, k, C, ldw, 64));
  a.scale = scale;
  a.dxs = z.dxs;
  a.dws = z.dws;
  a.accX = w.accX;
  a.accW = w.accW;
  a.dX = reinterpret_cast<__nv_bfloat16*>(dX);
  a.lddx = lddx;
  a.dW = reinterpret_cast<__nv_bfloat16*>(dW);
  a.lddw = lddw;
  if (dX != nullptr) GQ_TRY(tmap(&m.ox, dX, k, n, lddx, 32));
  if (dW != nullptr) GQ_TRY(tmap(&m.ow, dW, k, C, lddw, 32));
  const int64_t tile = (int64_t)z.nkt * z.NK * kTile;
  const int64_t gy = z.Cp / 64 * z.npad;  // 64-class blocks of G, one after the other
  for (int i = 0; i <= z.pieces; ++i) {  // GRAD of piece i beside DX and DW of piece i - 1
    const int done = i - 1;
    a.gc0 = i * (int)z.Cp;
    a.gtiles = i < z.pieces ? (z.ctiles - i * z.per_piece < z.per_piece ? z.ctiles - i * z.per_piece : z.per_piece) : 0;
    if (i < z.pieces) GQ_TRY(tmap(&m.gst, w.G[i & 1], 64, gy, 64, 32));
    int ptiles = 0;
    if (i > 0) {
      const int classes = (done + 1 < z.pieces ? z.per_piece : z.ctiles - done * z.per_piece) * z.NT;
      ptiles = (int)cdiv(classes, kTile);
      GQ_TRY(tmap(&m.gk, w.G[done & 1], 64, gy, 64, 128));
      GQ_TRY(tmap(&m.gm, w.G[done & 1], 64, gy, 64, 64));
      a.pc0 = done * (int)z.Cp;
      a.psteps = classes / 64;
      a.ptiles = ptiles;
      a.do_dx = dX != nullptr;
      a.do_dw = dW != nullptr;
      a.dw_first = z.npad / 64 / z.dws > a.psteps / z.dxs;
      a.first = done == 0;
      a.last = i == z.pieces;
    }
    if (i > 0) a.full = 0;
    GQ_TRY(launch_tiles(m, a, z, s));
    if (i > 0 && dW != nullptr && z.dws > 1)
      GQ_TRY(launch_sum(ptiles, w.accW, z.dws, ptiles * tile, tile, w.nl, n, nullptr, a.pc0, C, k, scale, a.dW, lddw, s));
  }
  if (dX != nullptr && z.dxs > 1)
    GQ_TRY(launch_sum(z.nrt, w.accX, z.dxs, z.nrt * tile, tile, w.nl, n, w.idx, 0, C, k, scale, a.dX, lddx, s));
  return GQ_OK;
}
