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
// be the maximum: any m within 2^64 of it gives the same relative precision.
// m is the column maximum of the first tile with a valid row; later tiles only
// test s - m <= 64 (one vote of the warpgroup per tile), and the rare tile that
// fails raises m and scales O and the sums.
//
// fp32 results: P is written as three bf16 parts (24 bits) and multiplied
// three times; bf16 results use one part, whose rounding is of the size of the
// result's own.
//
//   warps 0..7    softmax (warpgroup g: heads g N/2 ..), O read-out
//   warps 8..11   producers (bf16: cp.async; e4m3: converted to bf16 on the way)
//   warp 12       MMA issuer, TMEM
//
// Few items: a cluster of S CTAs shares an item, each taking a share of its
// tiles; the partial O, m and sums are joined through distributed shared memory.
#pragma once

#include <cuda_bf16.h>

#include "attend.h"
#include "tc.cuh"

namespace hytopk {
namespace att {

constexpr int kSoftmaxWarps = 8;
constexpr float kSlack = 64.0f;  // largest s - m (log2) before m is raised
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <int D_, int N_, bool E4_, bool F32_>
struct Cfg {
  static constexpr int D = D_, N = N_;
  static constexpr bool E4 = E4_, F32 = F32_;
  static constexpr int HG = N / 2;             // heads of a softmax warpgroup
  static constexpr int CH = HG < 32 ? HG : 32; // S columns held in registers at once
  static constexpr int PARTS = F32 ? 3 : 1;
  // columns of the second product: P rows are whole 128-byte atoms of 64 heads
  // (columns N.. of a narrower item are never read)
  static constexpr int NP = N < 64 ? 64 : N;
  static constexpr int RB = 2 * D;             // bf16 row bytes
  using Geo = tc::Geo<RB>;
  static constexpr int SLOT = 128 * RB;        // one K or V tile
  static constexpr int PBYTES = NP / 64 * 16384;
  static constexpr int OBLK = D <= 128 ? 1 : D / 128;  // blocks of 128 result columns
  static constexpr int QBYTES = N * RB;
  static constexpr int QB = N <= 64 && D <= 128 ? 2 : 1;
  // P buffers: two, unless their three parts or 128 heads leave no room for the ring
  static constexpr int PB = F32 || N > 64 ? 1 : 2;
  static constexpr int PWARPS = 4;
  static constexpr int THREADS = (kSoftmaxWarps + PWARPS + 1) * 32;
  static constexpr int MMA_WARP = kSoftmaxWarps + PWARPS;
  // m, scale factors, 1 / sum [N] each; per-quadrant sums or maxima [4][N]
  static constexpr int MISC = (3 + 4) * N * 4 + 512;
  static constexpr int FIXED = PB * PARTS * PBYTES + QB * QBYTES + MISC + 1024;
  static constexpr int NS_MAX = (227 * 1024 - FIXED) / SLOT;
  static constexpr int NS = NS_MAX < 8 ? NS_MAX : 8;
  static constexpr int RING_OFF = 0;
  static constexpr int P_OFF = NS * SLOT;
  static constexpr int Q_OFF = P_OFF + PB * PARTS * PBYTES;
  static constexpr int MISC_OFF = Q_OFF + QB * QBYTES;
  static constexpr int SMEM = MISC_OFF + MISC + 1024;
  static constexpr int S_COL = 0, O_COL = 256;
  static_assert(2 * N <= 256 && 2 * OBLK * NP <= 256, "TMEM columns");
  static_assert(NS >= 2 && SMEM <= 227 * 1024, "shared memory");
  static_assert(NS * SLOT >= N * D * 4, "partial results of a split item");
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

template <int W>
__device__ __forceinline__ void tmem_load(uint32_t addr, float (&v)[W]) {
  if constexpr (W == 32) tc::tmem_ld32(addr, v);
  else if constexpr (W == 16) tc::tmem_ld16(addr, v);
  else tc::tmem_ld8(addr, v);
  tc::tmem_wait_ld(v);
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

struct Plan {
  int splits;   // CTAs per item (cluster size), 1: none
  int blocks;   // head blocks per cache head
  int heads;    // heads per block (the last may have fewer)
  int tiles;    // tiles of 128 rows per item
  int items;    // n * Hkv * blocks
};

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) k_attend(const Args a, const Plan pl) {
  constexpr int D = C::D, N = C::N, HG = C::HG, CH = C::CH, NS = C::NS, NP = C::NP;
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
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(o_empty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t rank = 0;
  if (pl.splits > 1) asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      tc::mbar_init(full + i, C::E4 ? C::PWARPS : C::PWARPS * 32);
      tc::mbar_init(empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(q_full + i, C::PWARPS);
      tc::mbar_init(q_empty + i, 1);
      tc::mbar_init(s_full + i, 1);
      tc::mbar_init(s_empty + i, kSoftmaxWarps);
      tc::mbar_init(o_full + i, 1);
      tc::mbar_init(o_empty + i, kSoftmaxWarps);
      tc::mbar_init(p_full + i, kSoftmaxWarps);
      tc::mbar_init(p_empty + i, 1);
    }
    *abort_flag = 0;
    tc::fence_barrier_init();
  }
  if (warp == C::MMA_WARP) {
    tc::tmem_alloc(tmem_slot, 512);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  // items of this CTA: first, first + stride, ...; its tiles of each: [tile0, tile0 + ntile)
  const int first = (int)(blockIdx.x / pl.splits), stride = (int)(gridDim.x / pl.splits);
  const int n_mine = pl.items > first ? (pl.items - 1 - first) / stride + 1 : 0;
  const int tile0 = (int)((int64_t)pl.tiles * rank / pl.splits);
  const int ntile = (int)((int64_t)pl.tiles * (rank + 1) / pl.splits) - tile0;
  const int total = n_mine * ntile;
  const int Hq = a.Hkv * a.G;

  struct Item {
    int t, hk, h0, nh;  // query, cache head, first head, heads
  };
  auto item_of = [&](int i) -> Item {
    const int it = first + i * stride;
    const int b = it % pl.blocks, r = it / pl.blocks;
    Item x;
    x.hk = r % a.Hkv;
    x.t = r / a.Hkv;
    x.h0 = x.hk * a.G + b * pl.heads;
    x.nh = min(pl.heads, a.G - b * pl.heads);
    return x;
  };
  // A role's walk over its tiles in order: the item and tile of tile g, kept by
  // steps (an item costs divisions; a tile must not).
  struct Walk {
    int qi, i, t, hk;  // item, tile within it, its query and cache head
  };
  auto walk_start = [&]() -> Walk {
    const Item x = item_of(0);
    return Walk{0, 0, x.t, x.hk};
  };
  auto walk_next = [&](Walk& w) {
    if (++w.i == ntile) {
      w.i = 0;
      const Item x = item_of(++w.qi);
      w.t = x.t;
      w.hk = x.hk;
    }
  };
  // Index entry j of query t as stored (-1 past the list), and the row it selects
  // (-1: none). Entries are loaded a tile or two ahead and only looked at when
  // they are used: a test right after the load would wait for it.
  auto entry_of = [&](int t, int j) -> int {
    return j < a.k_top ? __ldg(a.idx + (size_t)t * a.k_top + j) : -1;
  };
  auto row_of = [&](int e) -> int { return e >= a.L || e < 0 ? -1 : e; };

  if (warp >= kSoftmaxWarps && warp < C::MMA_WARP) {
    // ---------------- producers ----------------
    const int tid = threadIdx.x - kSoftmaxWarps * 32;
    const int pw = warp - kSoftmaxWarps;
    // this warp's writes to a buffer are done: one arrival per warp
    auto publish = [&](uint64_t* bar) {
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar);
    };
    // the item's query rows, zero beyond its heads
    auto load_query = [&](int qi) -> bool {
      const int qb = qi % C::QB;
      const bool ok = tc::mbar_wait(q_empty + qb, ((qi / C::QB) & 1) ^ 1, abort_flag, a.status);
      if (!__all_sync(0xffffffffu, ok)) return false;
      const Item x = item_of(qi);
      const uint8_t* src = static_cast<const uint8_t*>(a.q) +
                           ((size_t)x.t * a.q_row + (size_t)x.h0 * D) * 2;
      uint8_t* dst = smem + C::Q_OFF + qb * C::QBYTES;
      constexpr int CPR = C::RB / 16;
      for (int f = tid; f < N * CPR; f += C::PWARPS * 32) {
        const int r = f / CPR, c = f % CPR;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r < x.nh) v = __ldg(reinterpret_cast<const uint4*>(src + (size_t)r * C::RB) + c);
        *reinterpret_cast<uint4*>(dst + Geo::chunk_offset(r, c, N)) = v;
      }
      publish(q_full + qb);
      return true;
    };
    if constexpr (!C::E4) {
      // warp w gathers rows 32w .. 32w + 31 of every tile, CPR lanes per row
      constexpr int CPR = C::RB / 16;
      constexpr int RPP = CPR >= 32 ? 1 : 32 / CPR;
      constexpr int PASSES = 32 / RPP;              // row groups per warp and tile
      constexpr int SHIFT = CPR >= 32 ? 5 : (CPR == 16 ? 4 : 3);  // lanes per row
      int slot = 0;
      uint32_t phase = 1;
      bool ok = true;
      Walk w = walk_start(), wn = w;  // this tile; the next one
      int s_next = total > 0 ? entry_of(w.t, tile0 * 128 + tid) : -1;
      for (int g = 0; g < total && ok; ++g, w = wn) {
        if (w.i == 0 && !load_query(w.qi)) break;
        // every pass's row first, so that the copies go out back to back
        const int s_own = row_of(s_next);
        int rows[PASSES];
#pragma unroll
        for (int p = 0; p < PASSES; ++p)
          rows[p] = __shfl_sync(0xffffffffu, s_own, p * RPP + (lane >> SHIFT));
        if (g + 1 < total) {
          walk_next(wn);
          s_next = entry_of(wn.t, (tile0 + wn.i) * 128 + tid);
        }
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          ok = __all_sync(0xffffffffu, tc::mbar_wait(empty + slot, phase, abort_flag, a.status));
          if (!ok) break;
          const uint32_t dst = tc::smem_u32(ring + slot * C::SLOT);
          const int c = lane & ((1 << SHIFT) - 1);
          const uint8_t* base = static_cast<const uint8_t*>(kv ? a.v : a.k) +
                                (size_t)w.hk * C::RB + c * 16;
          const int64_t row_bytes = (kv ? a.v_row : a.k_row) * 2;
#pragma unroll
          for (int p = 0; p < PASSES; ++p) {
            const int s = rows[p];
            const uint8_t* src = base + (s >= 0 ? s * row_bytes : 0);
            cp_async16(dst + Geo::chunk_offset(pw * 32 + p * RPP + (lane >> SHIFT), c, 128), src,
                       s >= 0);
          }
          // arrives for this thread when its copies so far have landed; the MMA
          // issuer's proxy fence makes them visible to the tensor core
          cp_async_arrive(full + slot);
          if (++slot == NS) {
            slot = 0;
            phase ^= 1u;
          }
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
      // Warp w converts rows 32w .. 32w + 31 of every tile, CPR lanes of 16 codes
      // per row. A tile is two or four chunks of up to 8 loads a lane (K's, then
      // V's); two chunks are in registers, so that one is always in flight.
      constexpr int CPR = D / 16;          // 4, 8 or 16
      constexpr int RPP = 32 / CPR;
      constexpr int PASSES = 32 / RPP;
      constexpr int CP = PASSES < 8 ? PASSES : 8;  // passes of a chunk
      constexpr int NCH = 2 * PASSES / CP;         // chunks of a tile (K and V)
      const int c = lane % CPR;
      uint4 buf[2][CP];
      auto issue = [&](int hk, int s_own, int ch, uint4 (&v)[CP]) {
        const bool isv = ch >= NCH / 2;
        const uint8_t* base =
            static_cast<const uint8_t*>(isv ? a.v : a.k) + (size_t)hk * D + c * 16;
        const int64_t row_bytes = isv ? a.v_row : a.k_row;
        const int p0 = (ch % (NCH / 2)) * CP;
        int rows[CP];
#pragma unroll
        for (int p = 0; p < CP; ++p)
          rows[p] = __shfl_sync(0xffffffffu, s_own, (p0 + p) * RPP + lane / CPR);
#pragma unroll
        for (int p = 0; p < CP; ++p)
          v[p] = rows[p] >= 0 ? __ldg(reinterpret_cast<const uint4*>(base + rows[p] * row_bytes))
                              : make_uint4(0, 0, 0, 0);
      };
      int slot = 0;
      uint32_t phase = 1;
      auto store = [&](int ch, const uint4 (&v)[CP]) -> bool {
        if (ch % (NCH / 2) == 0 &&
            !__all_sync(0xffffffffu, tc::mbar_wait(empty + slot, phase, abort_flag, a.status)))
          return false;
        uint8_t* dst = ring + slot * C::SLOT;
        const int p0 = (ch % (NCH / 2)) * CP;
#pragma unroll
        for (int p = 0; p < CP; ++p) {
          const int r = pw * 32 + (p0 + p) * RPP + lane / CPR;
          *reinterpret_cast<uint4*>(dst + Geo::chunk_offset(r, 2 * c, 128)) =
              e4m3x8_to_bf16(make_uint2(v[p].x, v[p].y));
          *reinterpret_cast<uint4*>(dst + Geo::chunk_offset(r, 2 * c + 1, 128)) =
              e4m3x8_to_bf16(make_uint2(v[p].z, v[p].w));
        }
        if (ch % (NCH / 2) == NCH / 2 - 1) {
          publish(full + slot);
          if (++slot == NS) {
            slot = 0;
            phase ^= 1u;
          }
        }
        return true;
      };
      Walk w = walk_start(), wn = w;  // this tile; the next one
      auto own = [&](const Walk& x) { return entry_of(x.t, (tile0 + x.i) * 128 + tid); };
      int s_own = total > 0 ? row_of(own(w)) : -1, s_next = -1;
      if (total > 0) {
        issue(w.hk, s_own, 0, buf[0]);
        issue(w.hk, s_own, 1, buf[1]);
      }
      if (total > 1) {
        walk_next(wn);
        s_next = row_of(own(wn));
      }
      // the entry of the tile after the next is in flight while a tile is stored
      Walk wf = wn;
      int e_far = -1;
      if (total > 2) {
        walk_next(wf);
        e_far = own(wf);
      }
      bool ok = true;
      for (int g = 0; g < total && ok; ++g) {
        if (w.i == 0 && !load_query(w.qi)) break;
#pragma unroll
        for (int ch = 0; ch < NCH; ++ch) {
          if (!store(ch, buf[ch & 1])) {
            ok = false;
            break;
          }
          if (ch + 2 < NCH) issue(w.hk, s_own, ch + 2, buf[ch & 1]);
          else if (g + 1 < total) issue(wn.hk, s_next, ch + 2 - NCH, buf[ch & 1]);
        }
        w = wn;
        wn = wf;
        s_own = s_next;
        s_next = row_of(e_far);
        if (g + 3 < total) {
          walk_next(wf);
          e_far = own(wf);
        }
      }
    }
  } else if (warp == C::MMA_WARP) {
    // ---------------- MMA issuer ----------------
    // The whole warp keeps the (uniform) state and waits; one elected lane
    // issues. A single-lane branch would move every descriptor word through the
    // vector registers, which took 100 cycles per product.
    constexpr uint32_t ID_S = tc::instr_desc(0, 128, N);
    constexpr uint32_t ID_O = tc::instr_desc(0, 128, NP) | (1u << 15) | (1u << 16);
    constexpr uint32_t D_HI = (1024u >> 4) | (1u << 14) | (2u << 29);  // 8-row groups, SW128
    // 14 address bits: in a cluster, shared addresses carry the CTA's rank above them
    auto low = [](const void* p) { return (tc::smem_u32(p) >> 4) & 0x3FFFu; };
    const uint32_t ring_lo = low(ring), p_lo = low(pbuf), q_lo = low(smem + C::Q_OFF);
    constexpr uint32_t LBO_K = 1u << 16, LBO_MN = (16384u >> 4) << 16;
    auto desc = [&](uint32_t lo) { return tc::desc_from_words(lo, D_HI); };
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, abort_flag, a.status)) != 0;
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
    auto scores = [&](int g) -> bool {
      const int qb = ws.qi % C::QB;
      if (ws.i == 0 && !wait(q_full + qb, (ws.qi / C::QB) & 1)) return false;
      if (!wait(full + ws.slot, ws.phase)) return false;
      if (!wait(s_empty + (g & 1), ((g >> 1) & 1) ^ 1)) return false;
      if (!C::E4) tc::fence_proxy_async_smem();
      tc::fence_after_sync();
      const uint32_t ad = (ring_lo + ws.slot * (C::SLOT >> 4)) | LBO_K;
      const uint32_t bd = (q_lo + qb * (C::QBYTES >> 4)) | LBO_K;
      if (elect_one()) {
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
          tc::mma<0>(tmem + C::S_COL + (g & 1) * N, desc(ad + (Geo::step_offset(j, 128) >> 4)),
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
      const int ob = wo.qi & 1, pb = g % C::PB;
      if (wo.i == 0 && !wait(o_empty + ob, ((wo.qi >> 1) & 1) ^ 1)) return false;
      if (!wait(full + wo.slot, wo.phase)) return false;
      if (!wait(p_full + pb, (g / C::PB) & 1)) return false;
      if (!C::E4) tc::fence_proxy_async_smem();
      tc::fence_after_sync();
      const uint32_t ad = (ring_lo + wo.slot * (C::SLOT >> 4)) | LBO_MN;
      const uint32_t bd = (p_lo + pb * (C::PARTS * C::PBYTES >> 4)) | LBO_MN;
      if (elect_one()) {
#pragma unroll
        for (int blk = 0; blk < C::OBLK; ++blk) {
#pragma unroll
          for (int part = 0; part < C::PARTS; ++part) {
#pragma unroll
            for (int s = 0; s < 8; ++s)  // 16 rows each
              // d = 64 has one 64-column atom; the second one that M = 128 takes is
              // whatever follows the tile, and fills accumulator lanes never read
              tc::mma<0>(tmem + C::O_COL + (ob * C::OBLK + blk) * NP,
                         desc(ad + ((blk * 32768 + s * 2048) >> 4)),
                         desc(bd + ((part * C::PBYTES + s * 2048) >> 4)), ID_O,
                         (wo.i > 0 || part > 0 || s > 0) ? 1u : 0u);
          }
        }
        tc::mma_commit(p_empty + pb);
        tc::mma_commit(empty + wo.slot);
        if (wo.i == ntile - 1) tc::mma_commit(o_full + ob);
      }
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
  } else if (warp < kSoftmaxWarps) {
    // ---------------- softmax: TMEM lane = selected row ----------------
    const int wg = warp >> 2, quad = warp & 3;
    const int row = quad * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const int c0 = wg * HG;  // first head column of this warpgroup
    const float c_scale = a.scale * kLog2e;
    float l[HG];
    bool have = false;  // some row of the item so far is valid (the same for the warpgroup)
    // this row's entry two tiles ahead as stored, its scales one tile ahead
    int e_next = -1, e_far = -1;
    float ks_next = 1.0f, vs_next = 1.0f;
    auto load_scales = [&](int e, int hk) {
      if (C::E4) {
        const int s = row_of(e);
        ks_next = s >= 0 ? __ldg(a.k_scale + (size_t)s * a.Hkv + hk) : 1.0f;
        vs_next = s >= 0 ? __ldg(a.v_scale + (size_t)s * a.Hkv + hk) : 1.0f;
      }
    };
    // the item's result from O, once its last product is done
    auto finish = [&](int qi, bool any) -> bool {
      const Item x = item_of(qi);
      const int ob = qi & 1;
      const bool ok = tc::mbar_wait(o_full + ob, (qi >> 1) & 1, abort_flag, a.status);
      if (tc::bar_or(1 + wg, 128, !ok)) return false;
      tc::fence_after_sync();
#pragma unroll
      for (int blk = 0; blk < C::OBLK; ++blk) {
        const int d = blk * 128 + row;
        if (blk * 128 + quad * 32 >= D) continue;
#pragma unroll
        for (int cc = 0; cc < HG; cc += CH) {
          if (c0 + cc >= x.nh) continue;
          float v[CH];
          tmem_load(tmem + lane_off + C::O_COL + (ob * C::OBLK + blk) * NP + c0 + cc, v);
          if (pl.splits > 1) {
            // partial results for the cluster: [head][d] in the ring, which is idle now
            float* part = reinterpret_cast<float*>(ring);
#pragma unroll
            for (int u = 0; u < CH; ++u)
              if (c0 + cc + u < x.nh) part[(c0 + cc + u) * D + d] = any ? v[u] : 0.0f;
          } else {
            const size_t at = ((size_t)x.t * Hq + x.h0 + c0 + cc) * D + d;
#pragma unroll
            for (int u = 0; u < CH; ++u) {
              if (c0 + cc + u < x.nh) {
                const float o = any ? v[u] * il_s[c0 + cc + u] : 0.0f;
                if constexpr (C::F32) static_cast<float*>(a.out)[at + (size_t)u * D] = o;
                else static_cast<__nv_bfloat16*>(a.out)[at + (size_t)u * D] = __float2bfloat16_rn(o);
              }
            }
          }
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(o_empty + ob);
      return true;
    };
    Walk wf = walk_start();  // the tile whose entry is loaded: one ahead (e4m3: two)
    int qi = 0, i = -1;
    if (total > 0) {
      e_next = entry_of(wf.t, (tile0 + wf.i) * 128 + row);
      load_scales(e_next, wf.hk);
    }
    int hk_far = 0;
    if (C::E4 && total > 1) {
      walk_next(wf);
      e_far = entry_of(wf.t, (tile0 + wf.i) * 128 + row);
      hk_far = wf.hk;
    }
    bool pend_any = false;
    for (int g = 0; g < total; ++g) {
      if (++i == ntile) {
        i = 0;
        ++qi;
      }
      if (i == 0) {
        have = false;
#pragma unroll
        for (int u = 0; u < HG; ++u) l[u] = 0.0f;
      }
      const bool valid = row_of(e_next) >= 0;
      if (e_next != -1 && !valid && wg == 0 && a.status) atomicOr(a.status, HYTOPK_DEV_BAD_INDEX);
      const float c = valid ? c_scale * ks_next : 0.0f;
      const float vs = vs_next;
      if (C::E4) {
        e_next = e_far;
        load_scales(e_next, hk_far);
        if (g + 2 < total) {
          walk_next(wf);
          e_far = entry_of(wf.t, (tile0 + wf.i) * 128 + row);
          hk_far = wf.hk;
        }
      } else if (g + 1 < total) {
        walk_next(wf);
        e_next = entry_of(wf.t, (tile0 + wf.i) * 128 + row);
      }
      bool ok = tc::mbar_wait(s_full + (g & 1), (g >> 1) & 1, abort_flag, a.status);
      ok = __all_sync(0xffffffffu, ok);
      tc::fence_after_sync();
      const uint32_t s_addr = tmem + lane_off + C::S_COL + (g & 1) * N + c0;
      float v[CH];
      bool over = !have && valid;
      if (have) {
        float top = -INFINITY;
#pragma unroll
        for (int cc = 0; cc < HG; cc += CH) {
          tmem_load(s_addr + cc, v);
#pragma unroll
          for (int u = 0; u < CH; u += 2) {
            fma2(v[u], v[u + 1], c, nm_s[c0 + cc + u], nm_s[c0 + cc + u + 1]);
            top = max3(top, v[u], v[u + 1]);
          }
        }
        over = valid && top > kSlack;
      }
      bool reload = HG > CH;  // v holds this tile's s - m
      if (tc::bar_or(1 + wg, 128, over || !ok)) {
        // every product so far must be done before O is scaled
        if (have && g > 0)
          ok = ok && tc::mbar_wait(p_empty + (g - 1) % C::PB, ((g - 1) / C::PB) & 1, abort_flag,
                                   a.status);
        if (tc::bar_or(1 + wg, 128, !ok)) break;
        // raise (or set) the references to this tile's column maxima
#pragma unroll
        for (int cc = 0; cc < HG; cc += CH) {
          tmem_load(s_addr + cc, v);
#pragma unroll
          for (int u = 0; u < CH; ++u) v[u] = valid ? v[u] * c : -INFINITY;
          const float top = reduce_columns<CH, true>(v, lane);
          if (lane % (32 / CH) == 0) quad_s[quad * N + c0 + cc + lane / (32 / CH)] = top;
        }
        tc::bar_sync(1 + wg, 128);
        for (int h = row; h < HG; h += 128) {
          const int col = c0 + h;
          const float top = fmaxf(fmaxf(quad_s[col], quad_s[N + col]),
                                  fmaxf(quad_s[2 * N + col], quad_s[3 * N + col]));
          const float m = have ? fmaxf(-nm_s[col], top) : top;
          f_s[col] = have ? ex2(-nm_s[col] - m) : 1.0f;
          nm_s[col] = -m;
        }
        tc::bar_sync(1 + wg, 128);
        if (have) {
#pragma unroll
          for (int u = 0; u < HG; ++u) l[u] *= f_s[c0 + u];
          if (i > 0) {
#pragma unroll 1
            for (int blk = 0; blk < C::OBLK; ++blk) {
#pragma unroll 1
              for (int cc = 0; cc < HG; cc += 8) {
                const uint32_t addr =
                    tmem + lane_off + C::O_COL + ((qi & 1) * C::OBLK + blk) * NP + c0 + cc;
                float o[8];
                tmem_load(addr, o);
#pragma unroll
                for (int u = 0; u < 8; ++u) o[u] *= f_s[c0 + cc + u];
                tmem_store8(addr, o);
              }
            }
            tc::tmem_wait_st();
          }
        }
        have = true;
        reload = true;
      }
      // the weights of this row, rounded (or split) to bf16
      const bool all_valid = __all_sync(0xffffffffu, valid);
      uint8_t* p_dst = pbuf + (g % C::PB) * C::PARTS * C::PBYTES;
#pragma unroll
      for (int cc = 0; cc < HG; cc += CH) {
        if (have) {
          if (reload) {
            tmem_load(s_addr + cc, v);
#pragma unroll
            for (int u = 0; u < CH; u += 2)
              fma2(v[u], v[u + 1], c, nm_s[c0 + cc + u], nm_s[c0 + cc + u + 1]);
          }
          if (!all_valid) {
#pragma unroll
            for (int u = 0; u < CH; ++u) v[u] = valid ? v[u] : -INFINITY;
          }
#pragma unroll
          for (int u = 0; u < CH; u += 2) {
            v[u] = ex2(v[u]);
            v[u + 1] = ex2(v[u + 1]);
            add2(l[cc + u], l[cc + u + 1], v[u], v[u + 1]);
            if (C::E4) fma2(v[u], v[u + 1], vs, 0.0f, 0.0f);
          }
        } else {
#pragma unroll
          for (int u = 0; u < CH; ++u) v[u] = 0.0f;
        }
        if (cc == 0) {
          // the buffer's previous product
          if (cc + CH >= HG) {
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(s_empty + (g & 1));
          }
          ok = tc::mbar_wait(p_empty + g % C::PB, ((g / C::PB) & 1) ^ 1, abort_flag, a.status);
          // (a failed wait ends the warpgroup together at its next vote)
        }
#pragma unroll
        for (int part = 0; part < C::PARTS; ++part) {
#pragma unroll
          for (int u = 0; u < CH; u += 8) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              w[e] = pack_bf16(v[u + 2 * e], v[u + 2 * e + 1]);
              if (part + 1 < C::PARTS) take_bf16(w[e], v[u + 2 * e], v[u + 2 * e + 1]);
            }
            *reinterpret_cast<uint4*>(p_dst + part * C::PBYTES + p_offset(row, c0 + cc + u)) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      tc::fence_before_sync();
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (HG > CH) tc::mbar_arrive(s_empty + (g & 1));
        tc::mbar_arrive(p_full + g % C::PB);
      }
      // the previous item's result, while this item's first product runs
      if (i == 0 && qi > 0 && ntile > 1 && !finish(qi - 1, pend_any)) break;
      if (i == ntile - 1) {
        // sums over the rows: lanes, then quadrants
        if (ntile == 1 && qi > 0 && !finish(qi - 1, pend_any)) break;
        const Item x = item_of(qi);
#pragma unroll
        for (int cc = 0; cc < HG; cc += CH) {
#pragma unroll
          for (int u = 0; u < CH; ++u) v[u] = l[cc + u];
          const float sum = reduce_columns<CH, false>(v, lane);
          if (lane % (32 / CH) == 0) quad_s[quad * N + c0 + cc + lane / (32 / CH)] = sum;
        }
        tc::bar_sync(1 + wg, 128);
        for (int h = row; h < HG; h += 128) {
          const int col = c0 + h;
          const float sum = have ? (quad_s[col] + quad_s[N + col]) +
                                       (quad_s[2 * N + col] + quad_s[3 * N + col])
                                 : 0.0f;
          if (pl.splits > 1) {
            il_s[col] = sum;
            if (!have) nm_s[col] = INFINITY;
          } else {
            il_s[col] = 1.0f / sum;
            if (a.lse && col < x.nh)
              a.lse[(size_t)x.t * Hq + x.h0 + col] =
                  have ? (log2f(sum) - nm_s[col]) * kLn2 : -INFINITY;
          }
        }
        tc::bar_sync(1 + wg, 128);
        pend_any = have;
        if (qi == n_mine - 1 && !finish(qi, have)) break;
      }
    }
  }
  if (pl.splits > 1) {
    // join the cluster's parts: rank r takes heads r, r + splits, ... of the one item
    __syncwarp();
    cluster_sync();
    if (n_mine > 0 && !*abort_flag) {
      const Item x = item_of(0);
      const uint32_t part_a = tc::smem_u32(ring), m_a = tc::smem_u32(nm_s), l_a = tc::smem_u32(il_s);
      for (int f = threadIdx.x; f < x.nh * D; f += C::THREADS) {
        const int h = f / D, d = f - h * D;
        if (h % pl.splits != (int)rank) continue;
        float top = -INFINITY;
        for (int r = 0; r < pl.splits; ++r)
          top = fmaxf(top, -ld_cluster(map_cluster(m_a + h * 4, r)));
        float sum = 0.0f, o = 0.0f;
        for (int r = 0; r < pl.splits; ++r) {
          const float m = -ld_cluster(map_cluster(m_a + h * 4, r));
          if (m == -INFINITY) continue;
          const float w = ex2(m - top);
          sum += w * ld_cluster(map_cluster(l_a + h * 4, r));
          o += w * ld_cluster(map_cluster(part_a + (h * D + d) * 4, r));
        }
        const bool any = top != -INFINITY;
        o = any ? o / sum : 0.0f;
        const size_t at = ((size_t)x.t * Hq + x.h0 + h) * D + d;
        if constexpr (C::F32) static_cast<float*>(a.out)[at] = o;
        else static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(o);
        if (d == 0 && a.lse)
          a.lse[(size_t)x.t * Hq + x.h0 + h] = any ? (top + log2f(sum)) * kLn2 : -INFINITY;
      }
    }
    cluster_sync();
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == C::MMA_WARP) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// Launch one instance: the plan of head blocks and, with few items, of splits.
template <class C>
cudaError_t launch_attend(const Args& a, int sms, cudaStream_t st) {
  auto kernel = k_attend<C>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  Plan pl{};
  pl.blocks = (a.G + C::N - 1) / C::N;
  pl.heads = (a.G + pl.blocks - 1) / pl.blocks;
  pl.tiles = (a.k_top + 127) / 128;
  pl.items = a.n * a.Hkv * pl.blocks;
  pl.splits = 1;
  // split while every SM still gets at most one CTA and every CTA a tile
  while (pl.splits < 8 && 2 * pl.splits <= pl.tiles &&
         (int64_t)pl.items * 2 * pl.splits <= sms)
    pl.splits *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(pl.splits > 1 ? pl.items * pl.splits : (pl.items < sms ? pl.items : sms)));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)pl.splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pl.splits > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, a, pl);
}

}  // namespace att
}  // namespace hytopk
