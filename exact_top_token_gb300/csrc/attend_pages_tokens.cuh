// attend_pages_tokens.cuh -- attention over a cache in pages where each sequence has one new row
// or none, and at most 16 heads share a cache head (hytopk_attend_pages).
//
// An item is a sequence's row and the heads that share a cache head, few, and every key is seen
// by all of them. So the keys are the 128 lanes of the tensor core, and nothing is
// computed for rows that no head uses:
//
//   S^T [128 keys x N]  = K . Q^T      (K from tensor memory, Q from shared memory)
//   O^T [d x N]        += V^T . P^T    (both from shared memory, d and the heads contiguous)
//
// The mathematics, the types and the shares of the work are those of the general kernel
// (attend_pages_engine.cuh): f16 operands, weights 2^(s + b - m) with b of v's scale, m whole
// numbers that are raised when a weight would pass 2^11, the slow form. Here a thread of the
// softmax owns a key: k's scale, b, and whether the key is seen are its own, the denominators are
// summed per thread and joined at an item's end, and m is agreed on by a vote of the four warps, a
// tile.
// Keys past the context's end, the same for all heads, have v replaced by zeros as it is
// widened, so that NaN codes there reach nothing.
//
// 64 sequences over up to 16384 keys, 32 heads of 128 on 8, take 167 us, 5.8 TB/s of the 6.7 that a
// copy reaches (the general kernel 221). Memory bounds it, shared memory is just behind: of a tile
// 32 KB come as codes and 152 KB pass through shared memory, 1190 cycles where memory's share of an
// SM takes 1400; the general kernel passes 224 KB, f16 keys and operands of 128 rows among them,
// and here the keys' f16 form goes to tensor memory. A tile is a chain of short steps of
// single warps, a few hundred cycles each however little they do, so what counts is that no
// warp has too many of them: with both products in one warp, or the scales beside the copies
// or the widening, that warp took 2000 cycles a tile (205 us); with the pages of four tiles
// looked up at once and the scales beside the segments a tile takes 1400. Items of 17 to 64 heads, with 64
// columns, took 134 us where the general kernel took 87 (one token over 2^20 keys, 64 heads). Heads
// of 64 columns, otherwise as above: 146 us, 3.3 TB/s; half the bytes of each tile, so the chain
// of its steps bounds it.
//
//   warp 0        products with V; tensor memory
//   warp 1        this CTA's segments: (item, tiles) in order, and the tiles' scales, through rings
//   warp 2        codes of the tiles by TMA
//   warp 3        products with K
//   warps 4-11    softmax, two warpgroups; results
//   warps 12-15   K's codes to f16, into tensor memory; queries
//   warps 16-19   V's codes to f16, into shared memory
#pragma once

#include "attend_pages_engine.cuh"

namespace hytopk {
namespace pages {

template <int D_>
struct TCfg {
  static constexpr int D = D_, N = 16;  // N: columns, of the heads
  static constexpr int RB = 2 * D;
  using Geo = tc::Geo<RB>;
  static constexpr int SLOT = 128 * RB;  // f16 V of a tile
  static constexpr int PB = 16384;       // P of a tile: [128 keys][64 heads], whole atoms
  static constexpr int QB = N * RB;
  static constexpr int UNIT = 128 * D;  // codes, K in even units and V in odd ones
  static constexpr int UNITS = D == 128 ? 6 : 8;
  static constexpr int P_OFF = 2 * SLOT;
  static constexpr int Q_OFF = P_OFF + 2 * PB;
  static constexpr int STAGE_OFF = Q_OFF + 2 * QB;
  static constexpr int CONST_OFF = STAGE_OFF + UNITS * UNIT;
  static constexpr int SEG_OFF = CONST_OFF + kConsts * (int)sizeof(TileConst);
  static constexpr int QS_OFF = SEG_OFF + kSegs * (int)sizeof(Seg);  // [2][N] queries' powers of two
  // of a warpgroup: [2][N] -m, factors, d; [4][N] maxima, sums; [2 N + 16] what the other is told
  static constexpr int SOFT = (14 * N + 2 * N + 16) * 4;
  static constexpr int SOFT_OFF = QS_OFF + 2 * N * 4;
  static constexpr int SHARE_OFF = SOFT_OFF + 2 * SOFT;
  static constexpr int BAR_OFF = SHARE_OFF + (int)sizeof(Share);
  static constexpr int SMEM = BAR_OFF + 768 + 1024;
  static constexpr int K_COL = 0, S_COL = 128, O_COL = 256, COLS = 512;  // two each
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static_assert(SEG_OFF % 16 == 0 && SHARE_OFF % 8 == 0 && BAR_OFF % 8 == 0, "alignment");
};
constexpr int kTThreads = 640;
// Registers: 96 a thread at launch; the widening warps keep them.
constexpr int kTRegsLaunch = 96, kTRegsCtl = 64, kTRegsSoft = 112;
static_assert(kTRegsCtl + 2 * kTRegsSoft + 2 * kTRegsLaunch <= 5 * kTRegsLaunch, "register split");

// Two fp32 at a time: (a0, a1) * (b0, b1) + (c0, c1)
__device__ __forceinline__ void madd2(float& a0, float& a1, float b0, float b1, float c0, float c1) {
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %3};\n"
      " mov.b64 z, {%4, %5};\n fma.rn.f32x2 x, x, y, z;\n mov.b64 {%0, %1}, x;\n}\n"
      : "+f"(a0), "+f"(a1)
      : "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}

// 16-byte chunk of heads h .. h + 7 of key r in the P tile
__device__ __forceinline__ uint32_t p_chunk(int r, int h) {
  return (uint32_t)((r >> 3) * 1024 + (r & 7) * 128 + (((h >> 3) ^ (r & 7)) << 4));
}

template <class C>
__global__ void __launch_bounds__(kTThreads, 1)
    k_attend_tokens(const AttendArgs a, const __grid_constant__ CUtensorMap k_map,
                    const __grid_constant__ CUtensorMap v_map) {
  constexpr int D = C::D, N = C::N, UNITS = C::UNITS;
  using Geo = typename C::Geo;
  extern __shared__ __align__(1024) uint8_t smem_dyn[];
  uint8_t* smem = tc::align1024(smem_dyn);
  TileConst* const_s = reinterpret_cast<TileConst*>(smem + C::CONST_OFF);
  Seg* seg_s = reinterpret_cast<Seg*>(smem + C::SEG_OFF);
  float* qs_s = reinterpret_cast<float*>(smem + C::QS_OFF);
  Share* share = reinterpret_cast<Share*>(smem + C::SHARE_OFF);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  uint64_t* k_full = bars;          // [2] of a tile, by its parity: f16 K
  uint64_t* k_empty = k_full + 2;   // [2]
  uint64_t* v_full = k_empty + 2;   // [2] f16 V
  uint64_t* v_empty = v_full + 2;   // [2]
  uint64_t* s_full = v_empty + 2;   // [2] scores
  uint64_t* s_empty = s_full + 2;   // [2]
  uint64_t* p_full = s_empty + 2;   // [2] weights
  uint64_t* pv_done = p_full + 2;   // [2] products with them
  uint64_t* o_full = pv_done + 2;   // a segment's
  uint64_t* o_empty = o_full + 1;
  uint64_t* ml_full = o_empty + 1;  // the second warpgroup's sums
  uint64_t* ml_empty = ml_full + 1;
  uint64_t* q_full = ml_empty + 1;  // [2]
  uint64_t* q_empty = q_full + 2;   // [2]
  uint64_t* seg_full = q_empty + 2;        // [kSegs]
  uint64_t* seg_empty = seg_full + kSegs;  // [kSegs]
  uint64_t* c_full = seg_empty + kSegs;    // [kConsts] scales of a tile
  uint64_t* c_empty = c_full + kConsts;    // [kConsts]
  uint64_t* unit_full = c_empty + kConsts;  // [UNITS] codes
  uint64_t* unit_empty = unit_full + UNITS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(unit_empty + UNITS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* several_s = abort_flag + 1;  // some sequence has several rows
  static_assert((24 + 2 * kSegs + 2 * kConsts + 2 * UNITS) * 8 + 12 <= 768, "barriers");

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(k_full + i, 4);
      tc::mbar_init(k_empty + i, 1);
      tc::mbar_init(v_full + i, 4);
      tc::mbar_init(v_empty + i, 1);
      tc::mbar_init(s_full + i, 1);
      tc::mbar_init(s_empty + i, 4);
      tc::mbar_init(p_full + i, 4);
      tc::mbar_init(pv_done + i, 1);
      tc::mbar_init(q_full + i, 4);
      tc::mbar_init(q_empty + i, 1 + 8);
    }
    tc::mbar_init(o_full, 1);
    tc::mbar_init(o_empty, 4);
    tc::mbar_init(ml_full, 4);
    tc::mbar_init(ml_empty, 4);
    for (int i = 0; i < kSegs; ++i) {
      tc::mbar_init(seg_full + i, 1);
      tc::mbar_init(seg_empty + i, 3 + 16);
    }
    for (int i = 0; i < kConsts; ++i) {
      tc::mbar_init(c_full + i, 1);
      tc::mbar_init(c_empty + i, 4);
    }
    for (int i = 0; i < UNITS; ++i) {
      tc::mbar_init(unit_full + i, 1);
      tc::mbar_init(unit_empty + i, 4);
    }
    *abort_flag = 0;
    *several_s = 0;
    tc::fence_barrier_init();
  }
  if (warp == 0) {
    tc::tmem_alloc(tmem_slot, C::COLS);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  allow_next();
  wait_for_earlier();
  if (find_share<kTThreads>(a, reinterpret_cast<int64_t*>(const_s), share)) *several_s = 1;
  __syncthreads();

  const uint32_t abort_at = tc::smem_u32(tmem_slot + 1);
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_phase(bar, parity, abort_at)) != 0;
  };
  auto arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(bar);
  };
  auto take = [&](int number, Seg& s) -> bool {
    if (!wait(seg_full + number % kSegs, (number / kSegs) & 1)) return false;
    s = seg_s[number % kSegs];
    arrive(seg_empty + number % kSegs);
    return true;
  };
  // A role's walk over the tiles of the segments, in order.
  struct At {
    int hk, row, end, t, t0, t1, number;
    bool ok;
  };
  auto settle = [&](At& c) {  // to the next tile at or after c
    if (c.ok && c.t >= c.t1) {
      Seg s;
      c.ok = take(c.number, s) && !(s.flags & kStop);
      ++c.number;
      c.hk = s.hk;
      c.row = s.row0;
      c.end = s.end;
      c.t = c.t0 = s.t0;
      c.t1 = s.t1;
    }
  };
  auto next = [&](At c) {
    if (c.ok) {
      ++c.t;
      settle(c);
    }
    return c;
  };
  auto begin = [&]() {
    At c{0, 0, 0, 0, 0, 0, 0, true};
    settle(c);
    return c;
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTRegsCtl));
    if (warp == 1) {
      // ---------------- segments ----------------
      // (several rows of a sequence: no segment here, all of it is the next kernel's; a return here
      // and now cost the roles' code 10 % of their speed)
      const int several = *several_s;
      if (a.several) {
        if (blockIdx.x == 0 && lane == 0) *a.several = several;
        if (lane == 0 && several) share->any = 0;
        __syncwarp();
      }
      // The scales of a segment's tiles follow it, up to kConsts tiles ahead of the softmax.
      int number = 0, g = 0;
      segments<D>(a, *share, lane, [&](const Seg& s) {
        if (!wait(seg_empty + number % kSegs, ((number / kSegs) & 1) ^ 1)) return false;
        if (lane == 0) {
          seg_s[number % kSegs] = s;
          tc::mbar_arrive(seg_full + number % kSegs);
        }
        ++number;
        return segment_scales(a, s, lane, [&](int k, float2 group, float ref, uint32_t odd) {
          const int slot = g % kConsts;
          if (!wait(c_empty + slot, ((g / kConsts) & 1) ^ 1)) return false;
          TileConst* out = const_s + slot;
          if (lane >> 3 == k) reinterpret_cast<float2*>(out->group)[lane & 7] = group;
          if (lane == 0) {
            out->ref = ref;
            out->odd = odd;
          }
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(c_full + slot);
          ++g;
          return true;
        });
      });
    } else if (warp == 2) {
      // ---------------- codes of the tiles ----------------
      // They come by TMA, as many rows at a time as a page and a tile share (a page that is not
      // there lies past the pool's end, where rows of zeros are).
      int unit = 0;
      uint32_t used = 0, phases = 0;  // bits of the units' places
      // tile t of a segment, whose pages eight lanes from `first` on have
      auto copy = [&](const CUtensorMap* map, int hk, int t, int page, int first) -> bool {
        const uint32_t bit = 1u << unit;
        if (!wait(unit_empty + unit, (phases & bit) ? 0u : 1u)) return false;
        phases ^= bit;
        used |= bit;
        uint8_t* to = smem + C::STAGE_OFF + unit * C::UNIT;
        if (elect_one()) tc::mbar_expect_tx(unit_full + unit, C::UNIT);
        __syncwarp();
#pragma unroll 1
        for (int r = 0; r < 128; r += a.box) {
          const int pg = __shfl_sync(0xffffffffu, page, first + (r >> 4));
          const int row = (uint32_t)pg < (uint32_t)a.s.N
                              ? (pg << a.shift) + ((t * 128 + r) & (a.s.P - 1))
                              : a.s.N << a.shift;
          if (elect_one()) tc::tma_load_2d(to + r * D, map, unit_full + unit, hk * D, row);
          __syncwarp();
        }
        if (++unit == UNITS) unit = 0;
        return true;
      };
      if (lane == 0) {
        tc::tma_prefetch(&k_map);
        tc::tma_prefetch(&v_map);
      }
      // (what earlier kernels stored is read by the copies' own path)
      asm volatile("fence.proxy.async.global;" ::: "memory");
      Seg s;
      bool ok = true;
#pragma unroll 1
      for (int segs = 0; ok && take(segs, s) && !(s.flags & kStop); ++segs) {
        int page = pages_of(a, lane, s.b, s.t0, s.end), next = -1;
#pragma unroll 1
        for (int t = s.t0; t < s.t1; ++t) {
          const int first = (t - s.t0) % 4 * 8;
          if (first == 0) {  // (the four after these, as early)
            if (t > s.t0) page = next;
            if (t + 4 < s.t1) next = pages_of(a, lane, s.b, t + 4, s.end);
          }
          if (!(ok = copy(&k_map, s.hk, t, page, first) && copy(&v_map, s.hk, t, page, first))) break;
        }
      }
      if (!ok || *abort_flag) {
        // given up: copies in flight land before the CTA ends (a bounded wait)
#pragma unroll 1
        for (int i = 0; i < UNITS; ++i) {
          if (!(used >> i & 1)) continue;
          const uint32_t parity = phases >> i & 1 ? 0u : 1u;  // of the last copy there
          for (int n = 0; n < 100000; ++n)
            if (tc::mbar_try_wait(unit_full + i, parity)) break;
        }
      }
    } else {
      // ---------------- products: with K (warp 3), with V (warp 0) ----------------
      // The state is in uniform registers (what comes from a segment passes a shuffle); one
      // elected lane issues. In one warp the two took 1700 cycles a tile, most of them its
      // own instructions and waits.
      constexpr uint32_t D_HI = (1024u >> 4) | (1u << 14) | (2u << 29);  // 8-row groups, SW128
      constexpr uint32_t LBO_K = 1u << 16, LBO_MN = (16384u >> 4) << 16;
      constexpr uint32_t ID_S = f16_desc(N), ID_O = f16_desc(64) | (1u << 15) | (1u << 16);
      auto low = [](const void* p) { return (tc::smem_u32(p) >> 4) & 0x3FFFu; };
      auto desc = [&](uint32_t lo) { return tc::desc_from_words(lo, D_HI); };
      Seg s;
      int g = 0;  // tiles so far
      bool ok = true;
#pragma unroll 1
      for (int segs = 0; ok && take(segs, s); ++segs) {
        if (__shfl_sync(0xffffffffu, s.flags & kStop, 0)) break;
        const int T = __shfl_sync(0xffffffffu, s.t1 - s.t0, 0);
        if (warp == 3) {
          const int qb = segs & 1;
          const uint32_t bd = (low(smem + C::Q_OFF) + qb * (C::QB >> 4)) | LBO_K;
          if (!(ok = wait(q_full + qb, segs >> 1 & 1))) break;
#pragma unroll 1
          for (int i = 0; i < T; ++i, ++g) {
            const int buf = g & 1, ph = g >> 1 & 1;
            if (!(ok = wait(k_full + buf, ph))) break;
            if (!(ok = wait(s_empty + buf, ph ^ 1))) break;
            if (i == 0) tc::fence_proxy_async_smem();  // (the queries)
            tc::fence_after_sync();
            if (elect_one()) {
#pragma unroll
              for (int j = 0; j < C::RB / 32; ++j)
                mma_ts(tmem + C::S_COL + buf * 64, tmem + C::K_COL + buf * 64 + j * 8,
                       desc(bd + (Geo::step_offset(j, N) >> 4)), ID_S, j > 0 ? 1u : 0u);
              tc::mma_commit(k_empty + buf);
              if (i == T - 1) tc::mma_commit(q_empty + qb);
              tc::mma_commit(s_full + buf);
            }
            __syncwarp();
          }
        } else {
          if (!(ok = wait(o_empty, (segs & 1) ^ 1))) break;
#pragma unroll 1
          for (int i = 0; i < T; ++i, ++g) {
            const int buf = g & 1, ph = g >> 1 & 1;
            if (!(ok = wait(v_full + buf, ph))) break;
            if (!(ok = wait(p_full + buf, ph))) break;
            tc::fence_proxy_async_smem();
            tc::fence_after_sync();
            const uint32_t ad = (low(smem) + buf * (C::SLOT >> 4)) | LBO_MN;
            const uint32_t bd = (low(smem + C::P_OFF) + buf * (C::PB >> 4)) | LBO_MN;
            const uint32_t o = tmem + C::O_COL + buf * 64, add = i < 2 ? 0u : 1u;
            if (elect_one()) {
              // (d = 64 has one atom of 64 columns; the second one that M = 128 takes is what
              // follows in shared memory, and fills lanes that are never read)
#pragma unroll
              for (int j = 0; j < 8; ++j)  // 16 keys
                tc::mma<0>(o, desc(ad + (j * 2048 >> 4)), desc(bd + (j * 2048 >> 4)), ID_O,
                           j > 0 ? 1u : add);
              tc::mma_commit(v_empty + buf);
              if (i == T - 1) tc::mma_commit(o_full);
              tc::mma_commit(pv_done + buf);
            }
            __syncwarp();
          }
        }
      }
    }
  } else if (warp >= 16) {
    // ---------------- V's codes to f16 ----------------
    // A warp takes 32 keys of a tile, CPR lanes a key: two 16-byte chunks of f16 for 16 codes.
    // Lanes of the second 128-byte line of a key write theirs in the other order: eight lanes
    // at a time then meet eight banks.
    constexpr int CPR = D / 16, RPP = 32 / CPR, PASSES = 32 / RPP;
    const int ww = warp - 16, c = lane % CPR, rl = lane / CPR;
    const int flip = (2 * c) >> 3 & 1;
    uint32_t place[2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
      place[e] = tc::smem_u32(smem) + Geo::chunk_offset(ww * 32 + rl, 2 * c + (e ^ flip), 128);
    int unit = 1, g = 0;
    uint32_t phase = 0;
#pragma unroll 1
    for (At at = begin(); at.ok; at = next(at), ++g) {
      if (!wait(unit_full + unit, phase)) break;
      const uint4* from =
          reinterpret_cast<const uint4*>(smem + C::STAGE_OFF + unit * C::UNIT + ww * 32 * D) + lane;
      uint4 x[PASSES];
#pragma unroll
      for (int u = 0; u < PASSES; ++u) x[u] = from[u * 32];
      arrive(unit_empty + unit);
      if ((unit += 2) > UNITS) {
        unit = 1;
        phase ^= 1u;
      }
      const int key = at.t * 128 + ww * 32 + rl;
      if (at.end - at.t * 128 < 128) {  // no row sees what lies past the end
#pragma unroll
        for (int u = 0; u < PASSES; ++u)
          if (key + u * RPP >= at.end) x[u] = make_uint4(0, 0, 0, 0);
      }
      if (!wait(v_empty + (g & 1), ((g >> 1) & 1) ^ 1)) break;
      const uint32_t to = (g & 1) * C::SLOT;
      // (keys RPP apart: the swizzle repeats every 8 keys)
#pragma unroll
      for (int u = 0; u < PASSES; ++u) {
        const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // 8-key groups are 1024 bytes apart, and a half of one flips the chunk's third bit
          const uint32_t p = (RPP == 8 ? place[e] + u * 1024
                                       : (place[e] + (u / 2) * 1024 + (u % 2) * 512) ^ ((u % 2) * 64u)) +
                             to;
          const int h = e ^ flip;
          const uint2 lo = widen(h ? w[2] : w[0]), hi = widen(h ? w[3] : w[1]);
          att::st_shared16(p, make_uint4(lo.x, lo.y, hi.x, hi.y));
        }
      }
      arrive(v_full + (g & 1));
    }
  } else if (warp >= 12) {
    // ---------------- K's codes to f16 ----------------
    // A thread takes a key: its codes lie swizzled (128 or 64 bytes a row), so that eight lanes
    // meet eight banks.
    const int quad = warp & 3, key = quad * 32 + lane;
    const uint32_t k_addr = tmem + ((uint32_t)(quad * 32) << 16) + C::K_COL;
    const int swz = D == 128 ? key & 7 : key >> 1 & 3;
    // An item's queries, N / 4 rows of each warp: to f16, with a power of two out of each row, so
    // that its largest is 2^14 to 2^15; LPR lanes a row, rows that no head has are zeros.
    constexpr int LPR = D / 8, RPI = 32 / LPR;
    const float sign = a.scale < 0.0f ? -1.0f : a.scale == 0.0f ? 0.0f : 1.0f;
    auto queries = [&](int qb, const At& at) {
      const int c = lane % LPR;
      uint8_t* block = smem + C::Q_OFF + qb * C::QB;
      const __nv_bfloat16* from = a.q + (int64_t)at.row * a.q_row + (int64_t)at.hk * a.G * D + c * 8;
#pragma unroll 2
      for (int i = 0; i < N / 4 / RPI; ++i) {
        const int r = quad * (N / 4) + i * RPI + lane / LPR;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (r < a.G) x = ld_after(reinterpret_cast<const uint4*>(from + r * D));
        const uint32_t most2 = __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu),
                                        __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
        uint32_t most = max(most2 << 16, most2 & 0xFFFF0000u);
#pragma unroll
        for (int o = LPR / 2; o; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
        const int ex = max((int)(most >> 23) - 127 - 14, -110);
        const float inv = sign * __int_as_float((127 - ex) << 23);
        const uint32_t y[4] = {x.x, x.y, x.z, x.w};
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float lo = __uint_as_float(y[e] << 16), hi = __uint_as_float(y[e] & 0xFFFF0000u);
          att::mul2(lo, hi, inv, inv);
          h[e] = pack_f16(lo, hi);
        }
        *reinterpret_cast<uint4*>(block + Geo::chunk_offset(r, c, N)) = make_uint4(h[0], h[1], h[2], h[3]);
        if (c == 0) qs_s[qb * N + r] = __int_as_float((ex + 127) << 23);
      }
    };
    int unit = 0, g = 0, items = 0;
    uint32_t phase = 0;
#pragma unroll 1
    for (At at = begin(); at.ok; at = next(at), ++g) {
      if (at.t == at.t0) {
        const int qb = items & 1;
        if (!wait(q_empty + qb, ((items >> 1) & 1) ^ 1)) break;
        queries(qb, at);
        arrive(q_full + qb);
        ++items;
      }
      if (!wait(unit_full + unit, phase)) break;
      const uint8_t* from = smem + C::STAGE_OFF + unit * C::UNIT + key * D;
      uint4 x[D / 16];
#pragma unroll
      for (int i = 0; i < D / 16; ++i) x[i] = *reinterpret_cast<const uint4*>(from + ((i ^ swz) << 4));
      arrive(unit_empty + unit);
      if ((unit += 2) >= UNITS) {
        unit = 0;
        phase ^= 1u;
      }
      if (!wait(k_empty + (g & 1), ((g >> 1) & 1) ^ 1)) break;
      tc::fence_after_sync();
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {  // 32 elements, 16 columns
        uint32_t y[16];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint4 z = x[2 * i + e];
          const uint2 p0 = widen(z.x), p1 = widen(z.y), p2 = widen(z.z), p3 = widen(z.w);
          y[8 * e] = p0.x, y[8 * e + 1] = p0.y, y[8 * e + 2] = p1.x, y[8 * e + 3] = p1.y;
          y[8 * e + 4] = p2.x, y[8 * e + 5] = p2.y, y[8 * e + 6] = p3.x, y[8 * e + 7] = p3.y;
        }
        tmem_store16(k_addr + (g & 1) * 64 + i * 16, y);
      }
      tc::tmem_wait_st();
      tc::fence_before_sync();
      arrive(k_full + (g & 1));
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTRegsSoft));
    // ---------------- softmax: TMEM lane = key ----------------
    // A warpgroup has every other tile, with references and a result of its own, joined at an
    // item's end.
    const int wg = (warp >> 2) - 1, quad = warp & 3, row = quad * 32 + lane;
    const int bar = 1 + wg;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t s_addr = tmem + lane_off + C::S_COL + wg * 64;
    const uint32_t o_addr = tmem + lane_off + C::O_COL + wg * 64;
    float* nm_s = reinterpret_cast<float*>(smem + C::SOFT_OFF + wg * C::SOFT);  // [2][N] -m
    float* f_s = nm_s + 2 * N;                                                 // [2][N]
    float* d_s = f_s + 2 * N;       // [2][N] (see the general kernel's softmax)
    float* quad_s = d_s + 2 * N;    // [4][N] maxima
    float* sum_s = quad_s + 4 * N;  // [4][N]
    float* told_s = sum_s + 4 * N;  // [N] -m, [N] d, and the reference of v's scales
    const int Hq = a.Hkv * a.G;
    int g0 = 0, cur = 0;  // tiles of the segments before; which nm_s counts
    Seg s;
    // The four warps leave together, and tell each other of waits that were given up: a named
    // barrier's vote for all that one tile or result needs.
    auto some_of_us = [&](bool x) { return tc::bar_or(bar, 128, x); };
#pragma unroll 1
    for (int segs = 0;; ++segs) {
      const bool got = take(segs, s);
      if (some_of_us(!got) || (s.flags & kStop)) break;
      const int T = s.t1 - s.t0;
      float l[N];
#pragma unroll
      for (int r = 0; r < N; ++r) l[r] = 0.0f;
      float ref = 1.0f;
      // slow: the slow form, for all that is left of a segment (see the general kernel); unset: some
      // head has no reference, because all scores so far are -inf or of rows that are not there
      bool slow = false, started = false, unset = false, ok = true;
      const float* qs = qs_s + (segs & 1) * N;
#pragma unroll 1
      for (int i = (g0 ^ wg) & 1; i < T; i += 2) {
        const int g = g0 + i;
        const TileConst* tile = const_s + g % kConsts;
        ok = ok && wait(c_full + g % kConsts, (g / kConsts) & 1);
        const float2 k = reinterpret_cast<const float2*>(tile->group)[row >> 4];
        const bool seen = (s.t0 + i) * 128 + row < s.end && !(tile->odd >> (row >> 4) & 1);
        slow |= tile->odd > 0xFFu;
        ok = ok && wait(s_full + wg, g >> 1 & 1);
        tc::fence_after_sync();
        float v[N];
        // s + b - m of all columns; the largest
        auto weights = [&]() -> float {
          const float* nm = nm_s + cur * N;
#pragma unroll
          for (int j = 0; j < N; j += 16) tc::tmem_ld16(s_addr + j, reinterpret_cast<float(&)[16]>(v[j]));
#pragma unroll
          for (int j = 0; j < N; j += 16) tc::tmem_wait_ld(reinterpret_cast<float(&)[16]>(v[j]));
#pragma unroll
          for (int j = 0; j < N; j += 4) {
            float4 c = *reinterpret_cast<const float4*>(qs + j);
            float4 m = *reinterpret_cast<const float4*>(nm + j);
            att::mul2(c.x, c.y, k.x, k.x);
            att::mul2(c.z, c.w, k.x, k.x);
            add2(m.x, m.y, k.y, k.y);
            add2(m.z, m.w, k.y, k.y);
            madd2(v[j], v[j + 1], c.x, c.y, m.x, m.y);
            madd2(v[j + 2], v[j + 3], c.z, c.w, m.z, m.w);
          }
          float m0 = max3(v[0], v[1], v[2]), m1 = max3(v[3], v[4], v[5]);
#pragma unroll
          for (int j = 6; j + 3 < N; j += 4) {
            m0 = max3(m0, v[j], v[j + 1]);
            m1 = max3(m1, v[j + 2], v[j + 3]);
          }
          return fmaxf(max3(m0, v[N - 2], v[N - 1]), m1);
        };
        if (!started) ok = ok && wait(q_full + (segs & 1), segs >> 1 & 1);  // (their powers of two)
        // Maxima over the tile of f(x, column) for all columns, x the score rounded; those of column
        // `lane` % N come back.
        auto tops = [&](auto&& f) -> float {
#pragma unroll 1
          for (int j = 0; j < N; j += 16) {
            float x[16];
            tc::tmem_ld16(s_addr + j, x);
            tc::tmem_wait_ld(x);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              x[e] = f(__fmul_rn(x[e], k.x * qs[j + e]), j + e);
              x[e] = seen && x[e] > -INFINITY ? x[e] : -INFINITY;  // (NaN as well)
            }
            const float top = att::reduce_columns<16, true>(x, lane);
            if (!(lane & 1)) quad_s[quad * N + j + lane / 2] = top;
          }
          some_of_us(false);
          const int r = lane % N;
          return fmaxf(fmaxf(quad_s[r], quad_s[N + r]), fmaxf(quad_s[2 * N + r], quad_s[3 * N + r]));
        };
        // the result so far times f_s
        auto shrink = [&]() {
          const float* f = f_s + cur * N;
          // the last products with this result
          ok = wait(pv_done + wg, (g - 2) >> 1 & 1);
          tc::fence_after_sync();
          if (ok) {
#pragma unroll 1
            for (int j = 0; j < N; j += 8) {
              float o[8];
              att::tmem_load(o_addr + j, o);
#pragma unroll
              for (int e = 0; e < 8; ++e) o[e] *= f[j + e];
              att::tmem_store8(o_addr + j, o);
            }
            tc::tmem_wait_st();
          }
        };
        bool raise = slow || !started || unset;
        if (!raise) raise = weights() > 11.0f && seen;
        if (some_of_us(raise || !ok)) {
          if (some_of_us(!ok)) {
            ok = false;
            break;
          }
          // (all four warps write the same, a lane a column)
          const int r = lane % N;
          float was = started ? nm_s[cur * N + r] : -INFINITY, d = started ? d_s[cur * N + r] : 0.0f;
          if (!slow) {
            // new references where the tile's maxima pass
            const float top = tops([&](float x, int) { return __fadd_rn(x, k.y); });
            const float to = 4.0f - ceilf(fmaxf(top, -att::kLargest));
            const bool none = was == -INFINITY, over = top > -INFINITY && (none || top + was > 11.0f);
            const float now = over ? to : was, f = over && !none ? ex2(to - was) : 1.0f;
            cur ^= 1;
            nm_s[cur * N + r] = now;
            f_s[cur * N + r] = f;
            d_s[cur * N + r] = 0.0f;
            __syncwarp();
            if (__any_sync(0xffffffffu, f != 1.0f)) {
#pragma unroll
              for (int j = 0; j < N; ++j) l[j] *= f_s[cur * N + j];
              shrink();
            }
            unset = __any_sync(0xffffffffu, r < a.G && now == -INFINITY);
            slow = __any_sync(0xffffffffu, now > -INFINITY && fabsf(now) > kFar);
            was = now;
            if (!slow) weights();
          }
          if (slow) {
            // the denominators' reference, then the weights'
            some_of_us(false);  // (the last maxima are read)
            float top = tops([&](float x, int) { return x; });
            const bool none = was == -INFINITY;
            float f = 1.0f, now = was;
            if (top > -INFINITY && (none || top + was > kWide)) {
              now = 4.0f - ceilf(fmaxf(top, -att::kLargest));
              if (!none) {
                f = ex2(now - was);
                d += was - now;
              }
            }
            cur ^= 1;
            nm_s[cur * N + r] = now;
            f_s[cur * N + r] = f;
            __syncwarp();
            const float* nm = nm_s + cur * N;
#pragma unroll
            for (int j = 0; j < N; ++j) l[j] *= f_s[cur * N + j];
            some_of_us(false);
            top = tops([&](float x, int j) { return __fadd_rn(__fadd_rn(x, nm[j]), k.y); });
            f = 1.0f;
            if (top > -INFINITY && (none || top + d > 11.0f)) {
              const float to = 4.0f - ceilf(top);
              if (!none) f = ex2(to - d);
              d = to;
            }
            f_s[cur * N + r] = f;
            d_s[cur * N + r] = d;
            __syncwarp();
            if (__any_sync(0xffffffffu, f != 1.0f)) shrink();
            const float nan = k.y - k.y;  // (NaN of a scale that is none, or 0)
#pragma unroll
            for (int j = 0; j < N; j += 16) {
              float x[16];
              tc::tmem_ld16(s_addr + j, x);
              tc::tmem_wait_ld(x);
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                x[e] = __fadd_rn(__fmul_rn(x[e], k.x * qs[j + e]), nm[j + e]);
                l[j + e] += seen ? ex2(x[e]) + nan : 0.0f;
                v[j + e] = __fadd_rn(__fadd_rn(x[e], k.y), d_s[cur * N + j + e]);
              }
            }
          }
          started = true;
        }
        ref = tile->ref;
        tc::fence_before_sync();
        arrive(s_empty + wg);
        if (lane == 0) tc::mbar_arrive(c_empty + g % kConsts);
        // the weights' place: of the products two tiles before (a wait that was given up is told
        // of in the next vote)
        if (g >= 2 && ok) ok = wait(pv_done + wg, (g - 2) >> 1 & 1);
        const float share_b = slow ? 0.0f : ex2(-k.y);  // (b goes out of the denominators)
        const uint32_t p0 = tc::smem_u32(smem + C::P_OFF + wg * C::PB);
#pragma unroll
        for (int j = 0; j < N; j += 8) {
          uint4 y = make_uint4(0, 0, 0, 0);
          if (seen) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[j + e] = ex2(v[j + e]);
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              float w0 = v[j + e], w1 = v[j + e + 1];
              fma2(w0, w1, share_b, l[j + e], l[j + e + 1]);
              l[j + e] = w0;
              l[j + e + 1] = w1;
            }
            y = make_uint4(pack_f16(v[j], v[j + 1]), pack_f16(v[j + 2], v[j + 3]),
                           pack_f16(v[j + 4], v[j + 5]), pack_f16(v[j + 6], v[j + 7]));
          }
          att::st_shared16(p0 + p_chunk(row, j), y);
        }
        arrive(p_full + wg);
      }
      if (some_of_us(!ok)) break;
      // ---- the result ----
      const bool part = s.part >= 0;
      if (wg == 1) ok = wait(ml_empty, (segs & 1) ^ 1);  // (the last ones are read)
#pragma unroll
      for (int j = 0; j < N; j += 16) {
        const float sum = att::reduce_columns<16, false>(reinterpret_cast<float(&)[16]>(l[j]), lane);
        if (!(lane & 1)) sum_s[quad * N + j + lane / 2] = sum;
      }
      const int r = lane % N;  // a column
      const float nm = started ? nm_s[cur * N + r] : -INFINITY, d = started ? d_s[cur * N + r] : 0.0f;
      arrive(q_empty + (segs & 1));  // (their powers of two)
      if (wg == 1) {
        // the first warpgroup takes this one's sums, references and result along
        if (quad == 0 && lane < N) told_s[r] = nm, told_s[N + r] = d;
        if (quad == 0 && lane == 0) told_s[2 * N] = ref;
        arrive(ml_full);
        if (some_of_us(!ok)) break;
        g0 += T;
        continue;
      }
      ok = wait(ml_full, segs & 1) && wait(o_full, segs & 1);
      if (some_of_us(!ok)) break;
      tc::fence_after_sync();
      // of this lane's column: factors of the results, so that the sum of weights is 1
      auto sum_of = [&](const float* x) { return (x[r] + x[N + r]) + (x[2 * N + r] + x[3 * N + r]); };
      const bool mine = T > 1 || !(g0 & 1), other = T > 1 || (g0 & 1);
      const float* theirs = sum_s + C::SOFT / 4;  // the second warpgroup's
      if (!mine) ref = theirs[6 * N];
      const Factors x = factors(sum_of(sum_s), nm, d, sum_of(theirs), theirs[4 * N + r], theirs[5 * N + r], ref);
      const size_t at = (size_t)s.row0 * Hq + (size_t)s.hk * a.G;  // the first head of out
      const size_t part_at = (size_t)max(s.part, 0) * a.rows;
      if (quad * 32 < D) {
#pragma unroll 1
        for (int j = 0; j < a.G; j += 8) {
          float o[8], z[8];
          if (mine) att::tmem_load(o_addr + j, o);
          if (other) att::tmem_load(o_addr + 64 + j, z);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float a1 = __shfl_sync(0xffffffffu, x.f1, j + e), a2 = __shfl_sync(0xffffffffu, x.f2, j + e);
            float y = 0.0f;
            if (mine) y = o[e] * a1;
            if (other) y += z[e] * a2;
            if (x.odd) y = y * __shfl_sync(0xffffffffu, x.p1, j + e) * __shfl_sync(0xffffffffu, x.p2, j + e);
            if (j + e < a.G) {
              if (part) a.part[(part_at + j + e) * D + row] = y;
              else a.out[(at + j + e) * D + row] = __float2bfloat16_rn(y);
            }
          }
        }
      }
      if (quad == 0 && lane < a.G) {
        if (part) a.ml[part_at + lane] = make_float2(x.sum, x.nm);
        else if (a.lse) a.lse[at + lane] = x.sum == 0.0f ? -INFINITY : (log2f(x.sum) - x.nm) * att::kLn2;
      }
      tc::fence_before_sync();
      arrive(o_empty);
      arrive(ml_empty);
      g0 += T;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag && a.status) atomicOr(a.status, tc::kDevTimeout);
  if (warp == 0) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, C::COLS);
  }
}

// (the parts are joined after the general kernel, or by `join`)
template <class C>
cudaError_t launch_attend_tokens(const AttendArgs& a, int ctas, bool join, cudaStream_t st) {
  auto kernel = k_attend_tokens<C>;
  CUtensorMap k_map, v_map;
  const uint64_t rows = (uint64_t)a.s.N * a.s.P;
  if (!make_tmap_2d(&k_map, a.k, 1, (uint64_t)a.Hkv * C::D, rows, C::D, a.box, C::D) ||
      !make_tmap_2d(&v_map, a.v, 1, (uint64_t)a.Hkv * C::D, rows, C::D, a.box, 0))
    return cudaErrorInvalidValue;
  static unsigned long long opted_in = 0;
  static int regs_ok = 0;
  // setmaxnreg waits for registers that the launch must have brought
  if (!__atomic_load_n(&regs_ok, __ATOMIC_RELAXED)) {
    cudaFuncAttributes fa;
    const cudaError_t e = cudaFuncGetAttributes(&fa, kernel);
    if (e != cudaSuccess) return e;
    if (fa.numRegs < kTRegsLaunch) return cudaErrorLaunchOutOfResources;
    __atomic_store_n(&regs_ok, 1, __ATOMIC_RELAXED);
  }
  const cudaError_t e =
      att::launch_opted_in(reinterpret_cast<const void*>(kernel), C::SMEM, &opted_in, [&] {
        return launch_early(kernel, (unsigned)ctas, kTThreads, C::SMEM, st, 1, a, k_map, v_map);
      });
  if (e != cudaSuccess || !join) return e;
  return launch_early(k_join_parts<C::D>, (unsigned)(ctas * kJoinBlocks), kJoinThreads, 0, st, 1, a,
                      ctas);
}

}  // namespace pages
}  // namespace hytopk
