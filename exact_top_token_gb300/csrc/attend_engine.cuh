// attend_engine.cuh -- attention of each query over its own selected rows on
// the tensor cores (hytopk_attend).
//
// One work item is a query and up to N of the heads that share a cache head.
// Its selected rows are gathered 128 at a time; a tile is scored and summed in
// the transposed form, because a query has few heads and many rows:
//
//   S^T [128 rows x N heads]  = K . Q^T        (K and Q K-major)
//   O^T [d x N heads]        += V^T . P^T      (V as gathered: M = d contiguous;
//                                               P [row][head]: N contiguous)
//
// Rows fill the 128 lanes of the tensor core whatever the number of heads is
// (N = 16 costs an eighth of N = 128), and a thread of the softmax owns one
// row: its validity and its e4m3 scales are private to it, and the sum over
// rows is kept per thread and joined once per item.
//
// Softmax without a running maximum per tile. The weights p = 2^(s - m) are
// stored in bf16 and summed in fp32, both with 8 exponent bits, so m need not
// be the maximum: any m well within 2^126 of it gives the same relative precision.
// m is the column maximum of the first tile with a valid row; later tiles only
// test s - m <= 24 in powers of two (one vote of the warpgroup per tile; a weight of
// 2^24 times V below 2^88 still sums in fp32), and the rare tile that fails raises m
// and scales O and the sums.
//
// fp32 results: P is written as three bf16 parts (24 bits); the first two are
// multiplied side by side (twice the columns) and the third adds to the second's,
// so that the largest sums take one addition per 16 rows. The tensor core's fp32
// additions truncate, and a long chain of them drifts (128 of them: 2e-6 of the
// result), so O is read out and added up in registers every kChunk tiles. bf16
// results use one part, whose rounding is of the size of the result's own, and one chain
// (1024 additions for 16384 rows: at that rate 2e-5, a hundredth of it).
//
// e4m3 rows are widened to bf16, which holds every e4m3 value: the codes land in the
// first half of their tile's place in shared memory and warps of their own widen them
// there. K's row scale joins the factor of the row's scores, V's multiplies its weights.
// 4096 queries of 64 heads, 2048 rows of 128 columns: bf16 rows 531 us (518 TFLOP/s, rows
// gathered at 8.1 TB/s), e4m3 rows 706 us; 128 heads 711 and 924 us. Bound by the warp
// instructions of a tile, on four schedulers: 3400, 6340 and 7780 for 16, 64 and 128 heads
// of bf16 rows, 5530 and 8150 for 16 and 64 of e4m3 ones. The last 64 heads add 5.6 for 32
// scores, so of the 6340 under a quarter are the scores' own; the rest is paid per warp and
// tile.
// For e4m3 rows, widening each row in a producer's registers took 1667 us; multiplying the
// codes, with q and P in two e4m3 parts, 771 us; copies and widening by the same warps,
// through a ring of its own, 742 us; widening to f16 with q and P in f16 694 us, but 128
// heads 1316 us, and weights 2^-31 of the largest were lost.
//
//   first warps   softmax (2 or 4 warpgroups, each with its share of the N head
//                 columns), O read-out
//   4 or 8 warps  producers: rows by cp.async, queries
//   2, 4 or 8     e4m3 rows only: widening
//   last warp     MMA issuer, TMEM
// A tile is a chain of short steps in different warps, so what counts is the
// length of each step: no division, no wait for a load and little code per tile
// (the roles share one instruction cache).
//
// Few items: a cluster of S CTAs shares an item, each taking a share of its
// tiles; the partial O, m and sums are joined through distributed shared memory.
#pragma once

#include <cuda_bf16.h>

#include "attend.h"
#include "early.cuh"
#include "tc.cuh"

namespace hytopk {
namespace att {

constexpr int kSplits = 8;  // CTAs that share an item, at most (a portable cluster)
constexpr int kChunk = 4;  // tiles summed on the tensor core where the result is fp32
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLargest = 3.402823466e38f;

// N, the head columns of an item, is the smallest instance that holds a group's heads:
// 16, 64 or, for bf16 results of d <= 128, 128; larger groups take several items, each
// gathering the rows anew. 4096 queries, 2048 rows of 128 columns, bf16 and e4m3 rows: 16
// heads 407 and 508 us with N = 16, 521 and 677 with 64; 32 heads, with 64, 522 and 680; 128
// heads 709 and 1028 us (now 924) with N = 128, 1055 and 1373 with two items of 64.
template <int D_, int N_, bool E4_, bool F32_, int CTAS_ = 1>
struct Cfg {
  static constexpr int D = D_, N = N_;
  static constexpr bool E4 = E4_, F32 = F32_;
  // CTAs of an SM. A tile of few heads is a chain that leaves the SM idle, so where shared
  // memory and registers hold two CTAs (N = 16, d = 64) and there are more items than SMs,
  // two run: 1024 queries of 32 heads on 8 cache heads, 2048 rows of 64 columns: bf16 519 us
  // instead of 669, e4m3 711 instead of 753. With fewer items the shorter ring loses (16
  // queries: 18 us instead of 16).
  static constexpr int CTAS = CTAS_;
  static constexpr int SWG = N >= 64 ? 4 : 2;     // softmax warpgroups
  static constexpr int SWARPS = 4 * SWG;
  static constexpr int HG = N / SWG;              // head columns of each: 8, 16 or 32
  static constexpr int PARTS = F32 ? 3 : 1;
  static constexpr float kSlack = 24.0f;  // m is raised when s - m passes this (log2)
  // columns of the second product: P rows are whole 128-byte atoms of 64 heads
  // (columns N.. of a narrower item are never read)
  static constexpr int NP = N < 64 ? 64 : N;
  static constexpr int RB = 2 * D;             // row bytes of the operands
  using Geo = tc::Geo<RB>;
  static constexpr int SLOT = 128 * RB;        // one K or V tile
  static constexpr int PBYTES = NP / 64 * 16384;
  static constexpr int OBLK = D <= 128 ? 1 : D / 128;  // blocks of 128 result columns
  static constexpr int OCOLS = F32 ? 2 * NP : NP;      // accumulator columns of a block
  static constexpr int QBYTES = N * RB;
  static constexpr int QB = N <= 64 && D <= 128 ? 2 : 1;
  // P buffers: two, unless their three parts, 128 heads or wide e4m3 rows leave no
  // room for the ring
  static constexpr int PB = F32 || N > 64 || (E4 && D == 256) ? 1 : 2;
  // Warps that copy rows, and (e4m3) warps that widen them: as many as leave a thread 72
  // registers for N = 64 and 80 for N = 128, where up to 32 bytes spill. (1024 queries of
  // 32 heads on 8 cache heads: 1019 us with 8 widening warps, 1102 with 4.)
  static constexpr int PWARPS = E4 || N > 64 ? 4 : 8;
  static constexpr int VWARPS = !E4 ? 0 : N > 64 ? 2 : N > 16 || CTAS > 1 ? 4 : 8;
  static constexpr int RPW = 128 / PWARPS;        // rows of a tile per copying warp
  static constexpr int THREADS = (SWARPS + PWARPS + VWARPS + 1) * 32;
  static constexpr int MMA_WARP = SWARPS + PWARPS + VWARPS;
  // m, scale factors, 1 / sum [N] each; per-quadrant sums or maxima [4][N]
  static constexpr int MISC = (3 + 4) * N * 4 + 512;
  static constexpr int SR = E4 ? 8 : 0;           // tiles of k and v scales [2][128]
  static constexpr int FIXED = PB * PARTS * PBYTES + QB * QBYTES + SR * 1024 + MISC + 1024;
  static constexpr int ALL = CTAS > 1 ? 113 * 1024 : 227 * 1024;  // shared memory of a CTA
  static constexpr int NS_MAX = (ALL - FIXED) / SLOT;
  static constexpr int NS = NS_MAX < 8 ? NS_MAX : 8;
  static constexpr int RING_OFF = 0;
  static constexpr int P_OFF = NS * SLOT;
  static constexpr int Q_OFF = P_OFF + PB * PARTS * PBYTES;
  static constexpr int SCALE_OFF = Q_OFF + QB * QBYTES;
  static constexpr int MISC_OFF = SCALE_OFF + SR * 1024;
  static constexpr int SMEM = MISC_OFF + MISC + 1024;
  static constexpr int S_COL = 0, O_COL = CTAS > 1 ? 64 : 256, COLS = CTAS > 1 ? 256 : 512;
  static_assert(2 * N <= O_COL && O_COL + 2 * OBLK * OCOLS <= COLS, "TMEM columns");
  static_assert(NS >= 2 && SMEM <= ALL, "shared memory");
  static_assert(NS * SLOT >= N * D * 4, "partial results of a split item");
  // Scales of tile j are copied once K's slot of the ring is free: V's before with NS
  // odd, so the softmax is done with tile j - (NS + 1) / 2; K's with NS even, so the
  // scores of tile j - NS / 2 are done, and for them the softmax has read tile
  // j - NS / 2 - 2.
  static_assert(!E4 || SR >= (NS % 2 ? (NS + 1) / 2 : NS / 2 + 2), "scales");
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 at a time: (a0, a1) * (b, b) + (c0, c1), and sums.
__device__ __forceinline__ void fma2(float& a0, float& a1, float b, float c0, float c1) {
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %2};\n"
      " mov.b64 z, {%3, %4};\n fma.rn.f32x2 x, x, y, z;\n mov.b64 {%0, %1}, x;\n}\n"
      : "+f"(a0), "+f"(a1)
      : "f"(b), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void add2(float& a0, float& a1, float b0, float b1) {
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %3};\n"
      " add.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}\n"
      : "+f"(a0), "+f"(a1)
      : "f"(b0), "f"(b1));
}
__device__ __forceinline__ void mul2(float& a0, float& a1, float b0, float b1) {
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %3};\n"
      " mul.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}\n"
      : "+f"(a0), "+f"(a1)
      : "f"(b0), "f"(b1));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// the two values minus their bf16 parts (exact)
__device__ __forceinline__ void take_bf16(uint32_t part, float& lo, float& hi) {
  lo -= __uint_as_float(part << 16);
  hi -= __uint_as_float(part & 0xFFFF0000u);
}

// Wait for a phase of `bar`; gives up (false, abort flag and status bit) when
// another role has, or after kTries tests of at most 2 us each. The same as
// tc::mbar_wait in a few instructions, since a tile passes a dozen of them.
constexpr int kTries = 1 << 20;
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort,
                                         uint32_t* status) {
  if (tc::mbar_try_wait(bar, parity)) return true;
#pragma unroll 1
  for (int i = 0; i < kTries; ++i) {
    if (tc::mbar_try_wait_suspend(bar, parity, tc::kSuspendHintNs)) return true;
    if (*abort) return false;
  }
  *abort = 1;
  if (status) atomicOr(status, tc::kDevTimeout);
  return false;
}

template <int W>
__device__ __forceinline__ void tmem_issue(uint32_t addr, float (&v)[W]) {
  if constexpr (W == 32) tc::tmem_ld32(addr, v);
  else if constexpr (W == 16) tc::tmem_ld16(addr, v);
  else tc::tmem_ld8(addr, v);
}
template <int W>
__device__ __forceinline__ void tmem_load(uint32_t addr, float (&v)[W]) {
  tmem_issue(addr, v);
  tc::tmem_wait_ld(v);
}
// two blocks of columns, one wait after the other's
template <int W>
__device__ __forceinline__ void tmem_load2(uint32_t a, uint32_t b, float (&v)[W], float (&x)[W]) {
  tmem_issue(a, v);
  tmem_issue(b, x);
  tc::tmem_wait_ld(v);
  tc::tmem_wait_ld(x);
}

__device__ __forceinline__ void tmem_store8(uint32_t addr, const float (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(
                   addr),
               "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// The sum or maximum of each of W columns over the warp's 32 lanes, by a
// butterfly that halves the columns a lane still carries. Lane l ends up with
// column l * W / 32 (W = 32: its own column; W = 8: four lanes share one).
template <int W, bool MAX>
__device__ __forceinline__ float reduce_columns(float (&v)[W], int lane) {
  int cur = W;
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) {
    if (cur >= 2) {
      const int half = cur / 2;
      const bool upper = (lane & off) != 0;
#pragma unroll
      for (int i = 0; i < W / 2; ++i) {
        if (i < half) {
          const float send = upper ? v[i] : v[half + i];
          const float keep = upper ? v[half + i] : v[i];
          const float got = __shfl_xor_sync(0xffffffffu, send, off);
          v[i] = MAX ? fmaxf(keep, got) : keep + got;
        }
      }
      cur = half;
    } else {
      const float got = __shfl_xor_sync(0xffffffffu, v[0], off);
      v[0] = MAX ? fmaxf(v[0], got) : v[0] + got;
    }
  }
  return v[0];
}

// 16-byte chunk of heads h .. h+7 of row r in the P tile
__device__ __forceinline__ uint32_t p_offset(int r, int h) {
  return (uint32_t)((h >> 6) * 16384 + (r >> 3) * 1024 + (r & 7) * 128 +
                    ((((h & 63) >> 3) ^ (r & 7)) << 4));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ uint2 ld_shared8(uint32_t src) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(src) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared16(uint32_t dst, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}
// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(tc::smem_u32(bar))
               : "memory");
}

__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t map_cluster(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}
template <int V>
struct Int {
  static constexpr int value = V;
};

struct Plan {
  int splits;   // CTAs per item (cluster size), 1: none
  int blocks;   // head blocks per cache head
  int heads;    // heads per block (the last may have fewer)
  int tiles;    // tiles of 128 rows per item
  int items;    // n * Hkv * blocks
  int stride;   // items between a CTA's items, and the same as (t, hk, b) digits
  int st, sh, sb;
};

template <class C>
__global__ void __launch_bounds__(C::THREADS, C::CTAS) k_attend(const Args a, const Plan pl) {
  constexpr int D = C::D, N = C::N, HG = C::HG, NS = C::NS, NP = C::NP;
  using Geo = typename C::Geo;
  extern __shared__ __align__(1024) uint8_t smem_dyn[];
  uint8_t* smem = tc::align1024(smem_dyn);
  uint8_t* ring = smem + C::RING_OFF;
  uint8_t* pbuf = smem + C::P_OFF;
  float* nm_s = reinterpret_cast<float*>(smem + C::MISC_OFF);  // [N] minus each head's reference
  float* f_s = nm_s + N;                                       // [N] factor of a raised reference
  float* il_s = f_s + N;                                      // [N] 1 / sum (split: the sum)
  float* quad_s = il_s + N;                                   // [4][N]
  uint64_t* bars = reinterpret_cast<uint64_t*>(quad_s + 4 * N);
  uint64_t* full = bars;
  uint64_t* empty = full + NS;
  uint64_t* q_full = empty + NS;
  uint64_t* q_empty = q_full + 2;
  uint64_t* s_full = q_empty + 2;
  uint64_t* s_empty = s_full + 2;
  uint64_t* p_full = s_empty + 2;
  uint64_t* p_empty = p_full + 2;
  uint64_t* o_full = p_empty + 2;
  uint64_t* o_empty = o_full + 2;
  uint64_t* landed = o_empty + 2;  // e4m3: [NS] codes are there
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(landed + NS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  // through a shuffle, so that the compiler knows the roles' branches are uniform
  // and keeps the MMA issuer's state in uniform registers
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  uint32_t rank = 0;
  if (pl.splits > 1) asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      tc::mbar_init(full + i, C::E4 ? C::VWARPS : C::PWARPS * 32);
      tc::mbar_init(landed + i, C::PWARPS * 32);
      tc::mbar_init(empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(q_full + i, C::PWARPS);
      tc::mbar_init(q_empty + i, 1);
      tc::mbar_init(s_full + i, 1);
      tc::mbar_init(s_empty + i, C::SWARPS);
      tc::mbar_init(o_full + i, 1);
      tc::mbar_init(o_empty + i, C::SWARPS);
      tc::mbar_init(p_full + i, C::SWARPS);
      tc::mbar_init(p_empty + i, 1);
    }
    *abort_flag = 0;
    tc::fence_barrier_init();
  }
  if (warp == C::MMA_WARP) {
    tc::tmem_alloc(tmem_slot, C::COLS);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  allow_next();
  wait_for_earlier();

  // items of this CTA: first, first + stride, ...; its tiles of each: [tile0, tile0 + ntile)
  const int first = (int)blockIdx.x / pl.splits;
  const int n_mine = pl.items > first ? (pl.items - 1 - first) / pl.stride + 1 : 0;
  const int tile0 = (int)((int64_t)pl.tiles * rank / pl.splits);
  const int ntile = (int)((int64_t)pl.tiles * (rank + 1) / pl.splits) - tile0;
  const int total = n_mine * ntile;
  const int Hq = a.Hkv * a.G;

  // A role's walk over its tiles in order: item (query t, cache head hk, head
  // block b) and tile i of it. Items advance by the stride's digits.
  struct Walk {
    int i, t, hk, b;
  };
  Walk start;
  start.i = 0;
  start.b = first % pl.blocks;
  start.hk = first / pl.blocks % a.Hkv;
  start.t = first / pl.blocks / a.Hkv;
  auto walk_next = [&](Walk& w) {
    if (++w.i == ntile) {
      w.i = 0;
      w.b += pl.sb;
      w.hk += pl.sh;
      w.t += pl.st;
      if (w.b >= pl.blocks) {
        w.b -= pl.blocks;
        ++w.hk;
      }
      if (w.hk >= a.Hkv) {
        w.hk -= a.Hkv;
        ++w.t;
      }
    }
  };
  auto first_head = [&](const Walk& w) { return w.hk * a.G + w.b * pl.heads; };
  auto head_count = [&](const Walk& w) { return min(pl.heads, a.G - w.b * pl.heads); };
  // Index entry j of query t as stored (-1 past the list), and the row it selects
  // (-1: none). Entries are loaded a tile or two ahead and only looked at when
  // they are used: a test right after the load would wait for it.
  auto entry_of = [&](int t, int j) -> int {
    return j < a.k_top ? ld_after(a.idx + (size_t)t * a.k_top + j) : -1;
  };
  auto row_of = [&](int e) -> int { return e >= a.L || e < 0 ? -1 : e; };

  if (warp >= C::SWARPS && warp < C::SWARPS + C::PWARPS) {
    // ---------------- producers ----------------
    const int tid = threadIdx.x - C::SWARPS * 32;
    const int pw = warp - C::SWARPS;
    // this warp's writes to a buffer are done: one arrival per warp
    auto publish = [&](uint64_t* bar) {
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar);
    };
    // the item's query rows, zero beyond its heads
    constexpr int QCPR = 2 * D / 16;
    constexpr int QPER = (N * QCPR + C::PWARPS * 32 - 1) / (C::PWARPS * 32);  // chunks of a thread
    constexpr int QU = QPER < 4 ? QPER : 4;                                   // at a time
    auto fetch_query = [&](const Walk& w, int p, uint4 (&v)[QU]) {
      const uint4* src = reinterpret_cast<const uint4*>(
          static_cast<const uint8_t*>(a.q) + ((size_t)w.t * a.q_row + (size_t)first_head(w) * D) * 2);
      const int nh = head_count(w);
#pragma unroll
      for (int u = 0; u < QU; ++u) {
        const int f = (p + u) * C::PWARPS * 32 + tid;
        v[u] = make_uint4(0, 0, 0, 0);
        if (f / QCPR < nh) v[u] = ld_after(src + f);
      }
    };
    // stores the chunks that are fetched already (v: the first) and the rest
    auto store_query = [&](int qi, const Walk& w, uint4 (&v)[QU]) -> bool {
      const int qb = qi % C::QB;
      const bool ok = wait_bar(q_empty + qb, ((qi / C::QB) & 1) ^ 1, abort_flag, a.status);
      if (!__all_sync(0xffffffffu, ok)) return false;
      uint8_t* dst = smem + C::Q_OFF + qb * C::QBYTES;
#pragma unroll 1
      for (int p = 0; p < QPER; p += QU) {
        if (p) fetch_query(w, p, v);
#pragma unroll
        for (int u = 0; u < QU; ++u) {
          const int f = (p + u) * C::PWARPS * 32 + tid, r = f / QCPR, c = f % QCPR;
          if (N * QCPR % (C::PWARPS * 32) && f >= N * QCPR) continue;
          *reinterpret_cast<uint4*>(dst + Geo::chunk_offset(r, c, N)) = v[u];
        }
      }
      publish(q_full + qb);
      return true;
    };
    // Warp w gathers rows RPW w .. of every tile, CPR lanes per row. The tile's
    // period was these loops at one time: rows come from their lanes first, a
    // source address is one multiply-add, and the swizzled destinations repeat
    // every 8 rows. The codes of an e4m3 row take the first 128-byte lines of its place
    // (a row's pieces that went to several lines were fetched one by one).
    constexpr int ES = C::E4 ? 1 : 2;
    constexpr int CPR = D * ES / 16;  // 4, 8, 16 or 32 lanes a row
    constexpr int SHIFT = CPR == 32 ? 5 : CPR == 16 ? 4 : CPR == 8 ? 3 : 2;
    constexpr int RPP = 32 / CPR;
    constexpr int PASSES = C::RPW / RPP;
    const int c = lane & (CPR - 1);
    uint32_t pat[8 / RPP];
#pragma unroll
    for (int p = 0; p < 8 / RPP; ++p) {
      const uint32_t r = p * RPP + (lane >> SHIFT);
      pat[p] = (uint32_t)(c >> 3) * 16384 + pw * C::RPW * 128 + r * 128 + (((c & 7) ^ r) << 4);
    }
    const uint32_t scale0 = tc::smem_u32(smem + C::SCALE_OFF) + (pw * C::RPW + lane) * 4;
    int slot = 0;
    uint32_t phase = 1;
    bool ok = true;
    Walk w = start, wn = w;  // this tile; the next one
    int qi = 0;
    int e_next = total > 0 ? entry_of(w.t, tile0 * 128 + pw * C::RPW + lane % C::RPW) : -1;
#pragma unroll 1
    for (int g = 0; g < total && ok; ++g, w = wn) {
      // an item's queries load while its first rows do
      uint4 qv[QU];
      if (w.i == 0) fetch_query(w, 0, qv);
      const int s_own = row_of(e_next);
      int rows[PASSES];
#pragma unroll
      for (int p = 0; p < PASSES; ++p)
        rows[p] = __shfl_sync(0xffffffffu, s_own, p * RPP + (lane >> SHIFT));
      if (g + 1 < total) {
        walk_next(wn);
        e_next = entry_of(wn.t, (tile0 + wn.i) * 128 + pw * C::RPW + lane % C::RPW);
      }
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv) {
        ok = __all_sync(0xffffffffu, wait_bar(empty + slot, phase, abort_flag, a.status));
        if (!ok) break;
        const uint32_t dst = tc::smem_u32(ring + slot * C::SLOT);
        const uint8_t* base = static_cast<const uint8_t*>(kv ? a.v : a.k) +
                              (size_t)w.hk * D * ES + c * 16;
        const uint32_t row_bytes = (uint32_t)((kv ? a.v_row : a.k_row) * ES);
#pragma unroll
        for (int p = 0; p < PASSES; ++p)
          cp_async16(dst + pat[p % (8 / RPP)] + p * RPP / 8 * 1024,
                     base + (uint64_t)(uint32_t)max(rows[p], 0) * row_bytes, rows[p] >= 0);
        // arrives for this thread when its copies so far have landed; the MMA
        // issuer's proxy fence makes them visible to the tensor core
        if (C::E4 && kv == 0) {
          // with K's, the scales of this warp's rows (0 for no row)
          const uint32_t sc = scale0 + (g & (C::SR - 1)) * 1024;
          const size_t at = (size_t)max(s_own, 0) * a.Hkv + w.hk;
          cp_async4(sc, a.k_scale + at, s_own >= 0);
          cp_async4(sc + 512, a.v_scale + at, s_own >= 0);
        }
        cp_async_arrive((C::E4 ? landed : full) + slot);
        if (++slot == NS) {
          slot = 0;
          phase ^= 1u;
        }
        // Between K and V: with two slots V waits for the product of the tile before,
        // which the MMA issuer starts only after this tile's scores.
        if (kv == 0 && w.i == 0 && !(ok = store_query(qi++, w, qv))) break;
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (C::E4 && warp >= C::SWARPS + C::PWARPS && warp < C::MMA_WARP) {
    // ---------------- e4m3: codes to bf16, in place ----------------
    // A lane takes 8 codes to one 16-byte chunk, LPR lanes a row; all codes of the rows
    // at hand are read before the first chunk is written.
    constexpr int LPR = D / 8 < 32 ? D / 8 : 32, RPP = 32 / LPR;
    constexpr int ROWS = 128 / (C::VWARPS ? C::VWARPS : 1);
    constexpr int U = 8 / RPP;  // passes at a time: the swizzle repeats every 8 rows
    const int cl = lane % LPR, rl = lane / LPR;
    uint32_t src[U], dst[U];
#pragma unroll
    for (int p = 0; p < U; ++p) {
      const int r = (warp - C::SWARPS - C::PWARPS) * ROWS + p * RPP + rl;
      src[p] = tc::smem_u32(ring) + Geo::chunk_offset(r, cl / 2, 128) + (cl & 1) * 8;
      dst[p] = tc::smem_u32(ring) + Geo::chunk_offset(r, cl, 128);
    }
    int slot = 0;
    uint32_t phase = 0;
#pragma unroll 1
    for (int h = 0; h < 2 * total; ++h) {
      if (!__all_sync(0xffffffffu, wait_bar(landed + slot, phase, abort_flag, a.status))) break;
      const uint32_t at = slot * C::SLOT;
      uint2 x[2][U];  // the rows at hand and the next ones
#pragma unroll
      for (int p = 0; p < U; ++p) x[0][p] = ld_shared8(src[p] + at);
#pragma unroll
      for (int r8 = 0; r8 < ROWS / 8; ++r8) {
        if (r8 + 1 < ROWS / 8) {
#pragma unroll
          for (int p = 0; p < U; ++p)
            x[(r8 + 1) & 1][p] = ld_shared8(src[p] + at + (r8 + 1) * 1024);
        }
        __syncwarp();
#pragma unroll
        for (int p = 0; p < U; ++p)
          st_shared16(dst[p] + at + r8 * 1024, e4m3x8_to_bf16(x[r8 & 1][p]));
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(full + slot);
      if (++slot == NS) {
        slot = 0;
        phase ^= 1u;
      }
    }
  } else if (warp == C::MMA_WARP) {
    // ---------------- MMA issuer ----------------
    // The whole warp keeps the (uniform) state and waits; one elected lane
    // issues. A single-lane branch would move every descriptor word through the
    // vector registers, which took 100 cycles per product.
    constexpr uint32_t ID_S = tc::instr_desc(0, 128, N);
    constexpr uint32_t ID_O = tc::instr_desc(0, 128, NP) | (1u << 15) | (1u << 16);
    constexpr uint32_t ID_O2 = tc::instr_desc(0, 128, C::OCOLS) | (1u << 15) | (1u << 16);
    constexpr uint32_t D_HI = (1024u >> 4) | (1u << 14) | (2u << 29);  // 8-row groups, SW128
    // 14 address bits: in a cluster, shared addresses carry the CTA's rank above them
    auto low = [](const void* p) { return (tc::smem_u32(p) >> 4) & 0x3FFFu; };
    const uint32_t ring_lo = low(ring), p_lo = low(pbuf), q_lo = low(smem + C::Q_OFF);
    constexpr uint32_t LBO_K = 1u << 16, LBO_MN = (16384u >> 4) << 16;
    auto desc = [&](uint32_t lo) { return tc::desc_from_words(lo, D_HI); };
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, wait_bar(bar, parity, abort_flag, a.status)) != 0;
    };
    struct At {
      int i, qi, slot;  // tile of its item, item, ring slot
      uint32_t phase;
    };
    auto step = [&](At& w) {
      if (++w.i == ntile) {
        w.i = 0;
        ++w.qi;
      }
      w.slot += 2;
      if (w.slot >= NS) {
        w.slot -= NS;
        w.phase ^= 1u;
      }
    };
    At ws{0, 0, 0, 0}, wo{0, 0, 1 % NS, 0};
    int nc = 0;  // accumulations of O begun: items, or chunks of them
    auto scores = [&](int g) -> bool {
      const int qb = ws.qi % C::QB;
      if (ws.i == 0 && !wait(q_full + qb, (ws.qi / C::QB) & 1)) return false;
      if (!wait(full + ws.slot, ws.phase)) return false;
      if (!wait(s_empty + (g & 1), ((g >> 1) & 1) ^ 1)) return false;
      tc::fence_proxy_async_smem();
      tc::fence_after_sync();
      const uint32_t ad = (ring_lo + ws.slot * (C::SLOT >> 4)) | LBO_K;
      const uint32_t bd = (q_lo + qb * (C::QBYTES >> 4)) | LBO_K;
      if (elect_one()) {
#pragma unroll
        for (int j = 0; j < C::RB / 32; ++j)
          tc::mma<0>(tmem + C::S_COL + (g & 1) * N,
                        desc(ad + (Geo::step_offset(j, 128) >> 4)),
                        desc(bd + (Geo::step_offset(j, N) >> 4)), ID_S, j > 0 ? 1u : 0u);
        tc::mma_commit(s_full + (g & 1));
        tc::mma_commit(empty + ws.slot);
        if (ws.i == ntile - 1) tc::mma_commit(q_empty + qb);
      }
      __syncwarp();
      step(ws);
      return true;
    };
    auto weighted = [&](int g) -> bool {
      const int ic = C::F32 ? wo.i % kChunk : wo.i, pb = g % C::PB;
      const int ob = nc & 1;
      if (ic == 0 && !wait(o_empty + ob, ((nc >> 1) & 1) ^ 1)) return false;
      if (!wait(full + wo.slot, wo.phase)) return false;
      if (!wait(p_full + pb, (g / C::PB) & 1)) return false;
      tc::fence_proxy_async_smem();
      tc::fence_after_sync();
      const uint32_t ad = (ring_lo + wo.slot * (C::SLOT >> 4)) | LBO_MN;
      const uint32_t bd = (p_lo + pb * (C::PARTS * C::PBYTES >> 4)) | LBO_MN;
      if (elect_one()) {
#pragma unroll
        for (int blk = 0; blk < C::OBLK; ++blk) {
#pragma unroll
          for (int part = 0; part < C::PARTS; part += 2) {
#pragma unroll
            for (int s = 0; s < 8; ++s)  // 16 rows
              // d = 64 has one 64-column atom; the second one that M = 128 takes is
              // whatever follows the tile, and fills accumulator lanes never read
              tc::mma<0>(tmem + C::O_COL + (ob * C::OBLK + blk) * C::OCOLS + (part ? NP : 0),
                         desc(ad + ((blk * 32768 + s * 2048) >> 4)),
                         desc(bd + ((part * C::PBYTES + s * 2048) >> 4)), part ? ID_O : ID_O2,
                         (ic > 0 || part > 0 || s > 0) ? 1u : 0u);
          }
        }
        tc::mma_commit(p_empty + pb);
        tc::mma_commit(empty + wo.slot);
        if (wo.i == ntile - 1 || (C::F32 && ic == kChunk - 1)) tc::mma_commit(o_full + ob);
      }
      if (wo.i == ntile - 1 || (C::F32 && ic == kChunk - 1)) ++nc;
      __syncwarp();
      step(wo);
      return true;
    };
    if (total > 0 && scores(0)) {
      for (int g = 0; g < total; ++g) {
        if (g + 1 < total && !scores(g + 1)) break;
        if (!weighted(g)) break;
      }
    }
  } else if (warp < C::SWARPS) {
    // ---------------- softmax: TMEM lane = selected row ----------------
    const int wg = warp >> 2, quad = warp & 3;
    const int row = quad * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const int c0 = wg * HG;  // first head column of this warpgroup
    const int bar = 1 + wg;
    const float c_scale = a.scale * kLog2e;
    constexpr int LPC = 32 / HG;  // lanes that share a column after reduce_columns
    float l[HG], v[HG];
    bool have = false;  // some row of the item so far is valid (the same for the warpgroup)
    int e_next = -1;  // this row's entry as stored, of the next tile
    Walk wf = start;  // the tile whose entry was loaded last
    int ahead = 0;    // tiles whose entries were loaded
    auto next_entry = [&]() -> int {
      if (ahead >= total) return -1;
      if (ahead++) walk_next(wf);
      return entry_of(wf.t, (tile0 + wf.i) * 128 + row);
    };
    e_next = next_entry();
    Walk w = start;
    int qi = 0;
    // An accumulation of O that is still to be read: the item before, or (fp32) a
    // chunk of an item. Its result goes out with the item's last.
    bool pend = false, pend_last = false, pend_any = false;
    int pend_nh = 0, nc = 0;  // accumulations read so far
    size_t pend_at = 0;
    constexpr int SUMS = C::F32 ? C::OBLK * HG : 1;
    float o_sum[SUMS];  // fp32: the item's chunks so far
    if constexpr (C::F32) {
#pragma unroll
      for (int u = 0; u < SUMS; ++u) o_sum[u] = 0.0f;
    }
    auto read_out = [&]() -> bool {
      const int ob = nc & 1;
      const bool ok = wait_bar(o_full + ob, (nc >> 1) & 1, abort_flag, a.status);
      if (tc::bar_or(bar, 128, !ok)) return false;
      tc::fence_after_sync();
#pragma unroll 1
      for (int blk = 0; blk < C::OBLK; ++blk) {
        const int d = blk * 128 + row;
        if (blk * 128 + quad * 32 >= D || c0 >= pend_nh) continue;
        const uint32_t o_addr = tmem + lane_off + C::O_COL + (ob * C::OBLK + blk) * C::OCOLS + c0;
        float o[HG];
        if constexpr (!C::F32) {
          tmem_load(o_addr, o);
        } else {
          float y[HG];
          tmem_load2(o_addr, o_addr + NP, o, y);
#pragma unroll
          for (int u = 0; u < HG; ++u) o[u] += y[u];
        }
        if constexpr (C::F32) {
#pragma unroll
          for (int u = 0; u < HG; ++u) {
            o[u] += o_sum[u];
            o_sum[u] = pend_last ? 0.0f : o[u];
          }
          if (!pend_last) continue;
        }
        // a split item's part stays unnormalised: [head][d] in the ring, idle by now
        float* part = reinterpret_cast<float*>(ring) + c0 * D + d;
#pragma unroll
        for (int u = 0; u < HG; ++u) {
          if (c0 + u < pend_nh) {
            const size_t at = pend_at + (size_t)(c0 + u) * D + d;
            if (pl.splits > 1) {
              part[u * D] = pend_any ? o[u] : 0.0f;
            } else {
              const float y = pend_any ? o[u] * il_s[c0 + u] : 0.0f;
              if constexpr (C::F32) static_cast<float*>(a.out)[at] = y;
              else static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(y);
            }
          }
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(o_empty + ob);
      pend = false;
      ++nc;
      return true;
    };
#pragma unroll 1
    for (int g = 0; g <= total; ++g) {
      if (g < total) {
        if (w.i == 0) {
          have = false;
#pragma unroll
          for (int u = 0; u < HG; ++u) l[u] = 0.0f;
        }
        const bool valid = row_of(e_next) >= 0;
        if (e_next != -1 && !valid && wg == 0 && a.status) atomicOr(a.status, HYTOPK_DEV_BAD_INDEX);
        e_next = next_entry();
        bool ok = wait_bar(s_full + (g & 1), (g >> 1) & 1, abort_flag, a.status);
        ok = __all_sync(0xffffffffu, ok);
        tc::fence_after_sync();
        const uint32_t s_addr = tmem + lane_off + C::S_COL + (g & 1) * N + c0;
        const float* sc = reinterpret_cast<const float*>(smem + C::SCALE_OFF) +
                          (g & (C::SR - 1)) * 256 + row;
        const float c = !valid ? 0.0f : C::E4 ? c_scale * sc[0] : c_scale;
        const float vs = C::E4 ? sc[128] : 1.0f;
        tmem_load(s_addr, v);
        bool over = !have && valid;
        if (have) {
#pragma unroll
          for (int u = 0; u < HG; u += 2)
            fma2(v[u], v[u + 1], c, nm_s[c0 + u], nm_s[c0 + u + 1]);
          float top = -INFINITY;
#pragma unroll
          for (int u = 0; u < HG; u += 2) top = max3(top, v[u], v[u + 1]);
          over = valid && top > C::kSlack;
        }
        if (tc::bar_or(bar, 128, over || !ok)) {
          // every product so far must be done before O is scaled
          if (have && g > 0)
            ok = ok && wait_bar(p_empty + (g - 1) % C::PB, ((g - 1) / C::PB) & 1, abort_flag,
                                a.status);
          if (tc::bar_or(bar, 128, !ok)) break;
          // raise (or set) the references to this tile's column maxima
          tmem_load(s_addr, v);
#pragma unroll
          for (int u = 0; u < HG; ++u) v[u] = valid ? __fmul_rn(v[u], c) : -INFINITY;
          const float top = reduce_columns<HG, true>(v, lane);
          if (lane % LPC == 0) quad_s[quad * N + c0 + lane / LPC] = top;
          tc::bar_sync(bar, 128);
          if (row < HG) {
            const int col = c0 + row;
            const float high = fmaxf(fmaxf(quad_s[col], quad_s[N + col]),
                                     fmaxf(quad_s[2 * N + col], quad_s[3 * N + col]));
            // (finite below: where all scores so far are -inf, so are their differences to it)
            const float m = fmaxf(have ? fmaxf(-nm_s[col], high) : high, -kLargest);
            f_s[col] = have ? ex2(-nm_s[col] - m) : 1.0f;
            nm_s[col] = -m;
          }
          tc::bar_sync(bar, 128);
          if (have) {
            if (C::F32 && pend && !read_out()) break;  // the chunk before, before its sums scale
#pragma unroll
            for (int u = 0; u < HG; ++u) {
              l[u] *= f_s[c0 + u];
              if (C::F32) o_sum[u] *= f_s[c0 + u];
            }
            if ((C::F32 ? w.i % kChunk : w.i) > 0) {
#pragma unroll 1
              for (int cc = 0; cc < C::OBLK * (C::OCOLS / NP) * HG; cc += 8) {
                const int blk = cc / HG, h = c0 + cc % HG;  // NP columns from block to block
                const uint32_t addr =
                    tmem + lane_off + C::O_COL + (nc & 1) * C::OBLK * C::OCOLS + blk * NP + h;
                float o[8];
                tmem_load(addr, o);
#pragma unroll
                for (int u = 0; u < 8; ++u) o[u] *= f_s[h + u];
                tmem_store8(addr, o);
              }
              tc::tmem_wait_st();
            }
          }
          have = true;
          tmem_load(s_addr, v);
          // the products rounded as the references were (packed ones would be fused with
          // the sum): of scores of 2^30 the largest would not be 0 otherwise
#pragma unroll
          for (int u = 0; u < HG; ++u)  // (volatile: loaded together they spill)
            v[u] = __fadd_rn(__fmul_rn(v[u], c), static_cast<volatile float*>(nm_s)[c0 + u]);
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(s_empty + (g & 1));
        // the weights of this row, rounded (or split) to bf16
        const bool off = !valid || !have;
        if (__any_sync(0xffffffffu, off)) {
#pragma unroll
          for (int u = 0; u < HG; ++u) v[u] = off ? -INFINITY : v[u];
        }
#pragma unroll
        for (int u = 0; u < HG; u += 2) {
          v[u] = ex2(v[u]);
          v[u + 1] = ex2(v[u + 1]);
          add2(l[u], l[u + 1], v[u], v[u + 1]);
          if (C::E4) mul2(v[u], v[u + 1], vs, vs);
        }
        // the buffer's previous product (a failed wait ends the warpgroup together
        // at its next vote)
        wait_bar(p_empty + g % C::PB, ((g / C::PB) & 1) ^ 1, abort_flag, a.status);
        uint8_t* p_dst = pbuf + (g % C::PB) * C::PARTS * C::PBYTES;
#pragma unroll
        for (int part = 0; part < C::PARTS; ++part) {
#pragma unroll
          for (int u = 0; u < HG; u += 8) {
            uint32_t x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              x[e] = pack_bf16(v[u + 2 * e], v[u + 2 * e + 1]);
              if (part + 1 < C::PARTS) take_bf16(x[e], v[u + 2 * e], v[u + 2 * e + 1]);
            }
            *reinterpret_cast<uint4*>(p_dst + part * C::PBYTES + p_offset(row, c0 + u)) =
                make_uint4(x[0], x[1], x[2], x[3]);
          }
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(p_full + g % C::PB);
      }
      // the accumulation before, while this tile's product runs
      if (pend && !read_out()) break;
      if (C::F32 && g < total && w.i % kChunk == kChunk - 1 && w.i < ntile - 1) {
        pend = true;
        pend_last = false;
        pend_nh = head_count(w);
      }
      if (g < total && w.i == ntile - 1) {
        // the item's sums over its rows: lanes, then quadrants
#pragma unroll
        for (int u = 0; u < HG; ++u) v[u] = l[u];
        const float sum = reduce_columns<HG, false>(v, lane);
        if (lane % LPC == 0) quad_s[quad * N + c0 + lane / LPC] = sum;
        tc::bar_sync(bar, 128);
        const int h0 = first_head(w), nh = head_count(w);
        if (row < HG) {
          const int col = c0 + row;
          const float z = have ? (quad_s[col] + quad_s[N + col]) +
                                     (quad_s[2 * N + col] + quad_s[3 * N + col])
                               : 0.0f;
          if (pl.splits > 1) {
            il_s[col] = z;
            if (!have) nm_s[col] = INFINITY;
          } else {
            il_s[col] = z == 0.0f ? 0.0f : 1.0f / z;  // 0: every score is -inf
            if (a.lse && col < nh)
              a.lse[(size_t)w.t * Hq + h0 + col] =
                  have ? (log2f(z) - nm_s[col]) * kLn2 : -INFINITY;
          }
        }
        tc::bar_sync(bar, 128);
        pend = pend_last = true;
        pend_any = have;
        pend_nh = nh;
        pend_at = ((size_t)w.t * Hq + h0) * D;
        ++qi;
      }
      walk_next(w);
    }
  }
  if (pl.splits > 1) {
    // Join the cluster's parts: each rank takes a share of the item's nh x d values, four
    // at a time. First what each CTA's part of a head counts, its references and sums read
    // once; reading them for every value took 3 of a single token's 14 us.
    __syncwarp();
    cluster_sync();
    if (!*abort_flag) {
      const int h0 = first_head(start), nh = head_count(start);
      const uint32_t part_a = tc::smem_u32(ring), m_a = tc::smem_u32(nm_s), l_a = tc::smem_u32(il_s);
      float* fac = reinterpret_cast<float*>(pbuf);  // [splits][N], idle by now
      const int all = nh * (D / 4), per = (all + pl.splits - 1) / pl.splits;
      const int lo = min(all, (int)rank * per), hi = min(all, lo + per);
      auto join = [&](auto parts) {
        constexpr int S = decltype(parts)::value;
        const int h = (lo * 4) / D + (int)threadIdx.x;  // of this share's heads
        if (h * D < hi * 4) {
          float m[S], z[S], top = -INFINITY, sum = 0.0f;
#pragma unroll
          for (int r = 0; r < S; ++r) {
            m[r] = -ld_cluster(map_cluster(m_a + h * 4, r));
            z[r] = ld_cluster(map_cluster(l_a + h * 4, r));
          }
#pragma unroll
          for (int r = 0; r < S; ++r) top = fmaxf(top, m[r]);
#pragma unroll
          for (int r = 0; r < S; ++r) {
            m[r] = m[r] == -INFINITY ? 0.0f : ex2(m[r] - top);
            sum += m[r] * z[r];
          }
          const bool any = sum != 0.0f;
#pragma unroll
          for (int r = 0; r < S; ++r) fac[r * N + h] = any ? m[r] / sum : 0.0f;
          if (a.lse && h * D >= lo * 4)
            a.lse[(size_t)start.t * Hq + h0 + h] = any ? (top + log2f(sum)) * kLn2 : -INFINITY;
        }
        __syncthreads();
#pragma unroll 1
        for (int f = lo + (int)threadIdx.x; f < hi; f += C::THREADS) {
          float4 o[S], y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
          for (int r = 0; r < S; ++r) o[r] = ld_cluster4(map_cluster(part_a + f * 16, r));
#pragma unroll
          for (int r = 0; r < S; ++r) {
            const float x = fac[r * N + f * 4 / D];
            y.x += x * o[r].x;
            y.y += x * o[r].y;
            y.z += x * o[r].z;
            y.w += x * o[r].w;
          }
          const size_t at = ((size_t)start.t * Hq + h0) * D + (size_t)f * 4;
          if constexpr (C::F32)
            *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = y;
          else
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + at) =
                make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
        }
      };
      if (pl.splits == 2) join(Int<2>{});
      else if (pl.splits == 4) join(Int<4>{});
      else join(Int<8>{});
    }
    cluster_sync();
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == C::MMA_WARP) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, C::COLS);
  }
}

// Launch one instance: the plan of head blocks and, with few items, of splits.
template <class C>
cudaError_t launch_attend(const Args& a, int sms, cudaStream_t st) {
  auto kernel = k_attend<C>;
  static unsigned long long opted_in = 0;
  static int fits[64][4];  // of each device, clusters of 2, 4 and 8 that run at once, + 1
  Plan pl{};
  pl.blocks = (a.G + C::N - 1) / C::N;
  pl.heads = (a.G + pl.blocks - 1) / pl.blocks;
  pl.tiles = (a.k_top + 127) / 128;
  pl.items = a.n * a.Hkv * pl.blocks;
  pl.splits = 1;
  // Split while every CTA has a tile and all clusters run at once: a second wave costs
  // more than the longest split saves (64 heads, 2048 rows: 14 tokens 13 us in clusters
  // of 8, 15 in clusters of 4; 16 tokens, of whose clusters of 8 not all fit, 23 and 15;
  // one token 12, 14, 21 and 29 us in 8, 4, 2 and 1; 12 us with 16 CTAs).
  while (pl.splits < kSplits && 2 * pl.splits <= pl.tiles &&
         (int64_t)pl.items * 2 * pl.splits <= sms &&
         pl.items <= clusters_at_once(reinterpret_cast<const void*>(kernel), C::THREADS, C::SMEM,
                                      2 * pl.splits, &opted_in, fits))
    pl.splits *= 2;
  const int ctas = pl.items < C::CTAS * sms ? pl.items : C::CTAS * sms;
  pl.stride = pl.splits > 1 ? pl.items : ctas;
  pl.sb = pl.stride % pl.blocks;
  pl.sh = pl.stride / pl.blocks % a.Hkv;
  pl.st = pl.stride / pl.blocks / a.Hkv;
  return launch_opted_in(reinterpret_cast<const void*>(kernel), C::SMEM, &opted_in, [&] {
    return launch_early(kernel, pl.splits > 1 ? pl.items * pl.splits : ctas, C::THREADS, C::SMEM,
                        st, pl.splits, a, pl);
  });
}

}  // namespace att
}  // namespace hytopk
