// attend_pages_tokens.cuh -- attention over a cache in pages for one new row of each sequence
// (hytopk_attend_pages without cu_q), at most 64 heads on a cache head.
//
// An item is a sequence's row and the N heads that share a cache head; N is few, and every key
// is seen by all of them. So the keys are the 128 lanes of the tensor core, and nothing is
// computed for rows that no head uses:
//
//   S^T [128 keys x N]  = K . Q^T      (K from tensor memory, Q from shared memory)
//   O^T [d x N]        += V^T . P^T    (both from shared memory, d and the heads contiguous)
//
// The mathematics, the types and the shares of the work are those of the general kernel
// (attend_pages_engine.cuh): f16 operands, weights 2^(s + b - m) with b of v's scale, m whole
// numbers that are raised when a weight would pass 2^11. Here a thread of the softmax owns a
// key: k's scale, b, and whether the key is seen are its own, the denominators are summed per
// thread and joined at an item's end, and m is agreed on by a vote of the four warps, a tile.
// Keys past the context end have their v replaced by zeros as it is widened, all rows see the
// same ones, so that their NaN codes reach nothing.
//
// What bounds it: memory, and shared memory just behind: of a tile of 128 columns 32 KB come as
// codes and 152 KB pass through shared memory (of 128 bytes a cycle: 1190 cycles; memory's share
// of an SM brings the codes in 1400). In the general kernel those are 224 KB, f16 keys and the
// operands of 128 rows among them; here the keys' f16 form goes to tensor memory.
//
//   warp 0        queries to f16; tensor memory
//   warp 1        this CTA's segments: (item, tiles) in order, through a ring
//   warp 2        pages: codes of the tiles by TMA, their scales through a ring
//   warp 3        products
//   warps 4-7     softmax; results
//   warps 8-11    K's codes to f16, into tensor memory
//   warps 12-15   V's codes to f16, into shared memory
#pragma once

#include "attend_pages_engine.cuh"

namespace hytopk {
namespace pages {

template <int D_, int N_>
struct TCfg {
  static constexpr int D = D_, N = N_;  // N: columns, of the heads
  static constexpr int RB = 2 * D;
  using Geo = tc::Geo<RB>;
  static constexpr int SLOT = 128 * RB;  // f16 V of a tile
  static constexpr int PB = 16384;       // P of a tile: [128 keys][64 heads], whole atoms
  static constexpr int QB = N * RB;
  static constexpr int UNIT = 128 * D;  // codes, K in even units and V in odd ones
  static constexpr int UNITS = D == 128 ? (N == 64 ? 4 : 6) : 8;
  static constexpr int P_OFF = 2 * SLOT;
  static constexpr int Q_OFF = P_OFF + 2 * PB;
  static constexpr int STAGE_OFF = Q_OFF + 2 * QB;
  static constexpr int CONST_OFF = STAGE_OFF + UNITS * UNIT;
  static constexpr int SEG_OFF = CONST_OFF + kConsts * (int)sizeof(TileConst);
  // [2][N] queries' powers of two, -m, factors; [4][N] maxima, sums; [2][4] votes
  static constexpr int QS_OFF = SEG_OFF + kSegs * (int)sizeof(Seg);
  static constexpr int NM_OFF = QS_OFF + 2 * N * 4;
  static constexpr int F_OFF = NM_OFF + 2 * N * 4;
  static constexpr int QUAD_OFF = F_OFF + 2 * N * 4;
  static constexpr int VOTE_OFF = QUAD_OFF + 2 * 4 * N * 4;
  static constexpr int SHARE_OFF = VOTE_OFF + 2 * 4 * 4;
  static constexpr int BAR_OFF = SHARE_OFF + (int)sizeof(Share);
  static constexpr int SMEM = BAR_OFF + 640 + 1024;
  static constexpr int K_COL = 0, S_COL = 128, O_COL = 256, COLS = 512;
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static_assert(SEG_OFF % 16 == 0 && SHARE_OFF % 8 == 0 && BAR_OFF % 8 == 0, "alignment");
  // The scales of a tile are written once its K has a place: K of the tile UNITS / 2 before is
  // widened then, so the products of the tile two before that are done, and the softmax
  // with the one another two before.
  static_assert(UNITS / 2 + 5 < kConsts, "scales");
};
// Registers by role: 128 (64 + 208 + 128 + 112) = 128 a thread at launch.
constexpr int kTRegsCtl = 64, kTRegsSoft = 208, kTRegsK = 128, kTRegsV = 112;
static_assert(kTRegsCtl + kTRegsSoft + kTRegsK + kTRegsV <= 4 * kRegsLaunch, "register split");

// 16-byte chunk of heads h .. h + 7 of key r in the P tile
__device__ __forceinline__ uint32_t p_chunk(int r, int h) {
  return (uint32_t)((r >> 3) * 1024 + (r & 7) * 128 + (((h >> 3) ^ (r & 7)) << 4));
}

template <class C>
__global__ void __launch_bounds__(kThreads, 1)
    k_attend_tokens(const AttendArgs a, const __grid_constant__ CUtensorMap k_map,
                    const __grid_constant__ CUtensorMap v_map) {
  constexpr int D = C::D, N = C::N, UNITS = C::UNITS;
  using Geo = typename C::Geo;
  extern __shared__ __align__(1024) uint8_t smem_dyn[];
  uint8_t* smem = tc::align1024(smem_dyn);
  TileConst* const_s = reinterpret_cast<TileConst*>(smem + C::CONST_OFF);
  Seg* seg_s = reinterpret_cast<Seg*>(smem + C::SEG_OFF);
  float* qs_s = reinterpret_cast<float*>(smem + C::QS_OFF);
  float* nm_s = reinterpret_cast<float*>(smem + C::NM_OFF);
  float* f_s = reinterpret_cast<float*>(smem + C::F_OFF);
  float* quad_s = reinterpret_cast<float*>(smem + C::QUAD_OFF);
  float* sum_s = quad_s + 4 * N;
  volatile int* vote_s = reinterpret_cast<volatile int*>(smem + C::VOTE_OFF);
  Share* share = reinterpret_cast<Share*>(smem + C::SHARE_OFF);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  uint64_t* k_full = bars;          // [2] of a tile, by its parity: f16 K
  uint64_t* k_empty = k_full + 2;   // [2]
  uint64_t* v_full = k_empty + 2;   // [2] f16 V
  uint64_t* v_empty = v_full + 2;   // [2]
  uint64_t* s_full = v_empty + 2;   // [2] scores
  uint64_t* p_full = s_full + 2;    // [2] weights
  uint64_t* pv_done = p_full + 2;   // a tile's products
  uint64_t* o_full = pv_done + 1;   // a segment's
  uint64_t* vote = o_full + 1;      // a tile's vote is in
  uint64_t* meet = vote + 1;        // the softmax warps, elsewhere
  uint64_t* q_full = meet + 1;      // [2]
  uint64_t* q_empty = q_full + 2;   // [2]
  uint64_t* seg_full = q_empty + 2;        // [kSegs]
  uint64_t* seg_empty = seg_full + kSegs;  // [kSegs]
  uint64_t* c_full = seg_empty + kSegs;    // [kConsts] scales of a tile
  uint64_t* unit_full = c_full + kConsts;  // [UNITS] codes
  uint64_t* unit_empty = unit_full + UNITS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(unit_empty + UNITS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  static_assert((20 + 2 * kSegs + kConsts + 2 * UNITS) * 8 + 8 <= 640, "barriers");

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(k_full + i, 4);
      tc::mbar_init(k_empty + i, 1);
      tc::mbar_init(v_full + i, 4);
      tc::mbar_init(v_empty + i, 1);
      tc::mbar_init(s_full + i, 1);
      tc::mbar_init(p_full + i, 4);
      tc::mbar_init(q_full + i, 1);
      tc::mbar_init(q_empty + i, 1 + 4);
    }
    tc::mbar_init(pv_done, 1);
    tc::mbar_init(o_full, 1);
    tc::mbar_init(vote, 4);
    tc::mbar_init(meet, 4);
    for (int i = 0; i < kSegs; ++i) {
      tc::mbar_init(seg_full + i, 1);
      tc::mbar_init(seg_empty + i, 3 + 12);
    }
    for (int i = 0; i < kConsts; ++i) tc::mbar_init(c_full + i, 1);
    for (int i = 0; i < UNITS; ++i) {
      tc::mbar_init(unit_full + i, 1);
      tc::mbar_init(unit_empty + i, 4);
    }
    *abort_flag = 0;
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
  find_share(a, reinterpret_cast<int64_t*>(const_s), share);
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
    int b, hk, end, t, t0, t1, number;
    bool ok;
  };
  auto settle = [&](At& c) {  // to the next tile at or after c
    if (c.ok && c.t >= c.t1) {
      Seg s;
      c.ok = take(c.number, s) && !(s.flags & kStop);
      ++c.number;
      c.b = s.b;
      c.hk = s.hk;
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
    if (warp == 0) {
      // ---------------- queries ----------------
      // Of each segment: to f16, with a power of two out of each row, so that its
      // largest is 2^14 to 2^15; LPR lanes a row, rows that no head has are zeros.
      constexpr int LPR = D / 8, RPI = 32 / LPR;
      const int c = lane % LPR;
      const float sign = a.scale < 0.0f ? -1.0f : a.scale == 0.0f ? 0.0f : 1.0f;
      Seg s;
      int loaded = 0;
#pragma unroll 1
      for (int number = 0; take(number, s) && !(s.flags & kStop); ++number) {
        const int qb = loaded & 1;
        if (!wait(q_empty + qb, ((loaded >> 1) & 1) ^ 1)) break;
        uint8_t* block = smem + C::Q_OFF + qb * C::QB;
        const __nv_bfloat16* from = a.q + (int64_t)s.row0 * a.q_row + (int64_t)s.hk * a.G * D + c * 8;
#pragma unroll 4
        for (int i = 0; i < N / RPI; ++i) {
          const int r = i * RPI + lane / LPR;
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
        arrive(q_full + qb);
        ++loaded;
      }
    } else if (warp == 1) {
      // ---------------- segments ----------------
      int number = 0;
      segments<D>(a, *share, lane, [&](const Seg& s) {
        if (!wait(seg_empty + number % kSegs, ((number / kSegs) & 1) ^ 1)) return false;
        if (lane == 0) {
          seg_s[number % kSegs] = s;
          tc::mbar_arrive(seg_full + number % kSegs);
        }
        ++number;
        return true;
      });
    } else if (warp == 2) {
      // ---------------- codes and scales of the tiles ----------------
      // Lanes 0 .. 7 take a group each: its page and its scales. The codes come by TMA, as many
      // rows at a time as a page and a tile share (a page that is not there lies past the
      // pool's end, where rows of zeros are). The page of the tile after next and the scales
      // of the next one are loaded while this one's go out.
      auto page_of = [&](const At& c) -> int {
        const int key = c.t * 128 + (lane & 7) * 16;
        if (!c.ok || key >= c.end) return -1;
        return ld_after(a.s.table + (size_t)c.b * a.s.columns + (key >> a.shift));
      };
      auto scales_of = [&](const At& c, int page) -> float2 {
        if (page < 0 || page >= a.s.N) return make_float2(0.0f, 0.0f);
        const size_t at = (size_t)page * a.Hkv + c.hk;
        return make_float2(ld_after(a.k_scale + at), ld_after(a.v_scale + at));
      };
      const float c_scale = (a.scale == 0.0f ? 1.0f : fabsf(a.scale)) * att::kLog2e;
      At c0 = begin();
      At c1 = next(c0);
      int page0 = page_of(c0), page1 = page_of(c1);
      float2 sc0 = scales_of(c0, page0);
      int tile = 0, unit = 0;
      uint32_t used = 0, phases = 0;  // bits of the units' places
      float ref = 1.0f, inv_ref = 1.0f;
      bool fresh = true;  // the segment's first tile, whose largest is the reference
      auto copy = [&](const CUtensorMap* map, const At& c, int page) -> bool {
        const uint32_t bit = 1u << unit;
        if (!wait(unit_empty + unit, (phases & bit) ? 0u : 1u)) return false;
        phases ^= bit;
        used |= bit;
        uint8_t* to = smem + C::STAGE_OFF + unit * C::UNIT;
        if (elect_one()) tc::mbar_expect_tx(unit_full + unit, C::UNIT);
        __syncwarp();
#pragma unroll 1
        for (int r = 0; r < 128; r += a.box) {
          const int pg = __shfl_sync(0xffffffffu, page, r >> 4);
          const int row = (uint32_t)pg < (uint32_t)a.s.N
                              ? (pg << a.shift) + ((c.t * 128 + r) & (a.s.P - 1))
                              : a.s.N << a.shift;
          if (elect_one()) tc::tma_load_2d(to + r * D, map, unit_full + unit, c.hk * D, row);
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
      bool ok = true;
#pragma unroll 1
      while (c0.ok) {
        const At c2 = next(c1);
        const int page2 = page_of(c2);
        const float2 sc1 = scales_of(c1, page1);
        if (!(ok = copy(&k_map, c0, page0))) break;
        const bool in = page0 >= 0 && page0 < a.s.N;
        if (page0 != -1 && !in && lane < 8 && a.status) atomicOr(a.status, HYTOPK_DEV_BAD_INDEX);
        const bool k_ok = sc0.x > 0.0f && sc0.x <= att::kLargest;
        const bool v_ok = sc0.y > 0.0f && sc0.y <= att::kLargest;
        if (in && !(k_ok && v_ok) && lane < 8 && a.status) atomicOr(a.status, HYTOPK_DEV_BAD_SCALE);
        if (fresh) {
          float top = in && v_ok ? sc0.y : 0.0f;
#pragma unroll
          for (int o = 4; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          ref = fmaxf(top > 0.0f ? top : 1.0f, 1.17549435e-38f);
          inv_ref = 1.0f / ref;
          fresh = false;
        }
        const float nan = __int_as_float(0x7fc00000);
        const bool past = c0.t * 128 + (lane & 7) * 16 >= c0.end;
        float2 group = make_float2(1.0f, 0.0f);  // (masked keys: any factor will do)
        if (in) {
          group.x = k_ok ? fmaxf(c_scale * sc0.x, 1.17549435e-38f) : nan;
          group.y = v_ok ? fminf(fmaxf(log2f(sc0.y * inv_ref), -100.0f), 100.0f) : nan;
        }
        const uint32_t absent = ~__ballot_sync(0xffffffffu, in || past) & 0xFFu;
        TileConst* out = const_s + tile % kConsts;
        if (lane < 8) reinterpret_cast<float2*>(out->group)[lane] = group;
        if (lane == 0) {
          out->ref = ref;
          out->absent = absent;
        }
        arrive(c_full + tile % kConsts);
        if (!(ok = copy(&v_map, c0, page0))) break;
        ++tile;
        fresh = c1.number != c0.number;
        c0 = c1;
        c1 = c2;
        page0 = page1;
        page1 = page2;
        sc0 = sc1;
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
    } else if (warp == 3) {
      // ---------------- products ----------------
      // The scores of a tile go out before the products of the tile before. A tile's scores
      // take the place of those of the tile two before, whose weights the products waited for.
      constexpr uint32_t D_HI = (1024u >> 4) | (1u << 14) | (2u << 29);  // 8-row groups, SW128
      constexpr uint32_t LBO_K = 1u << 16, LBO_MN = (16384u >> 4) << 16;
      constexpr uint32_t ID_S = f16_desc(N), ID_O = f16_desc(64) | (1u << 15) | (1u << 16);
      auto low = [](const void* p) { return (tc::smem_u32(p) >> 4) & 0x3FFFu; };
      const uint32_t v_lo = low(smem), p_lo = low(smem + C::P_OFF), q_lo = low(smem + C::Q_OFF);
      auto desc = [&](uint32_t lo) { return tc::desc_from_words(lo, D_HI); };
      auto uniform = [&](int x) { return __shfl_sync(0xffffffffu, x, 0); };
      int g = 0, segs = 0;  // tile and segment of the next scores
      auto scores = [&](bool first, bool last) -> bool {
        const int buf = g & 1, qb = segs & 1;
        if (first && !wait(q_full + qb, segs >> 1 & 1)) return false;
        if (!wait(k_full + buf, g >> 1 & 1)) return false;
        tc::fence_proxy_async_smem();  // (the queries)
        tc::fence_after_sync();
        const uint32_t bd = (q_lo + qb * (C::QB >> 4)) | LBO_K;
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < C::RB / 32; ++j)
            mma_ts(tmem + C::S_COL + buf * 64, tmem + C::K_COL + buf * 64 + j * 8,
                   desc(bd + (Geo::step_offset(j, N) >> 4)), ID_S, j > 0 ? 1u : 0u);
          tc::mma_commit(k_empty + buf);
          if (last) tc::mma_commit(q_empty + qb);
          tc::mma_commit(s_full + buf);
        }
        __syncwarp();
        ++g;
        if (last) ++segs;
        return true;
      };
      // of tile i
      auto weighted = [&](int i, bool first, bool last) -> bool {
        const int buf = i & 1;
        if (!wait(v_full + buf, i >> 1 & 1)) return false;
        if (!wait(p_full + buf, i >> 1 & 1)) return false;
        tc::fence_proxy_async_smem();
        tc::fence_after_sync();
        const uint32_t ad = (v_lo + buf * (C::SLOT >> 4)) | LBO_MN;
        const uint32_t bd = (p_lo + buf * (C::PB >> 4)) | LBO_MN;
        const uint32_t add = first ? 0u : 1u;
        if (elect_one()) {
          // (d = 64 has one atom of 64 columns; the second one that M = 128 takes is what
          // follows in shared memory, and fills lanes that are never read)
#pragma unroll
          for (int j = 0; j < 8; ++j)  // 16 keys
            tc::mma<0>(tmem + C::O_COL, desc(ad + (j * 2048 >> 4)), desc(bd + (j * 2048 >> 4)),
                       ID_O, j > 0 ? 1u : add);
          tc::mma_commit(v_empty + buf);
          if (last) tc::mma_commit(o_full);
          tc::mma_commit(pv_done);
        }
        __syncwarp();
        return true;
      };
      At c = begin();
      bool more = uniform(c.ok) != 0;
      bool first = true, last = uniform(c.t + 1 >= c.t1) != 0;
      if (more && scores(first, last)) {
#pragma unroll 1
        for (int i = 0;; ++i) {
          c = next(c);
          more = uniform(c.ok) != 0;
          const bool first1 = uniform(c.t == c.t0) != 0, last1 = uniform(c.t + 1 >= c.t1) != 0;
          if (more && !scores(first1, last1)) break;
          if (!weighted(i, first, last) || !more) break;
          first = first1;
          last = last1;
        }
      }
    }
  } else if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTRegsV));
    // ---------------- V's codes to f16 ----------------
    // A warp takes 32 keys of a tile, CPR lanes a key: two 16-byte chunks of f16 for 16 codes.
    // Lanes of the second 128-byte line of a key write theirs in the other order: eight lanes
    // at a time then meet eight banks.
    constexpr int CPR = D / 16, RPP = 32 / CPR, PASSES = 32 / RPP;
    const int ww = warp - 12, c = lane % CPR, rl = lane / CPR;
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
      if (at.t * 128 + 128 > at.end) {  // no row sees what lies past the end
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
  } else if (warp >= 8) {
    // 128 registers, as at launch
    // ---------------- K's codes to f16 ----------------
    // A thread takes a key: its codes lie swizzled (128 or 64 bytes a row), so that eight lanes
    // meet eight banks.
    const int quad = warp & 3, key = quad * 32 + lane;
    const uint32_t k_addr = tmem + ((uint32_t)(quad * 32) << 16) + C::K_COL;
    const int swz = D == 128 ? key & 7 : key >> 1 & 3;
    int unit = 0, g = 0;
    uint32_t phase = 0;
#pragma unroll 1
    for (At at = begin(); at.ok; at = next(at), ++g) {
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
    const int quad = warp & 3, row = quad * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t s_base = tmem + lane_off + C::S_COL, o_addr = tmem + lane_off + C::O_COL;
    uint8_t* p_at = smem + C::P_OFF;
    const int Hq = a.Hkv * a.G;
    int g = 0, segs = 0;        // tiles and segments so far
    uint32_t met = 0;           // meetings of the four warps so far
    int cur = 0;                // which nm_s counts
    Seg s;
    bool ok = true;
    auto together = [&]() -> bool {
      arrive(meet);
      const bool here = wait(meet, met & 1);
      ++met;
      return here;
    };
#pragma unroll 1
    for (int number = 0; ok && take(number, s) && !(s.flags & kStop); ++number) {
      const size_t at = (size_t)s.row0 * Hq + (size_t)s.hk * a.G;  // the first head of out
      float l[N];
#pragma unroll
      for (int r = 0; r < N; ++r) l[r] = 0.0f;
      float ref = 1.0f;
      bool exact = false;  // some reference is far from 0
      const float* qs = qs_s + (segs & 1) * N;
#pragma unroll 1
      for (int t = s.t0; t < s.t1; ++t, ++g) {
        const TileConst* tile = const_s + g % kConsts;
        if (!(ok = wait(c_full + g % kConsts, (g / kConsts) & 1))) break;
        ref = tile->ref;
        const float2 k = reinterpret_cast<const float2*>(tile->group)[row >> 4];
        const bool seen = t * 128 + row < s.end && !(tile->absent >> (row >> 4) & 1);
        if (!(ok = wait(s_full + (g & 1), g >> 1 & 1))) break;
        tc::fence_after_sync();
        const uint32_t s_addr = s_base + (g & 1) * 64;
        float v[N];
        // s + b - m of all heads; false if some would pass 11
        auto weights = [&]() -> bool {
          const float* nm = nm_s + cur * N;
#pragma unroll
          for (int i = 0; i < N; i += 16) tc::tmem_ld16(s_addr + i, reinterpret_cast<float(&)[16]>(v[i]));
          float top = -INFINITY;
#pragma unroll
          for (int i = 0; i < N; i += 16) {
            tc::tmem_wait_ld(reinterpret_cast<float(&)[16]>(v[i]));
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              const float4 q4 = *reinterpret_cast<const float4*>(qs + i + e);
              const float4 m4 = *reinterpret_cast<const float4*>(nm + i + e);
              const float qv[4] = {q4.x, q4.y, q4.z, q4.w}, mv[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                float& x = v[i + e + j];
                const float c = k.x * qv[j];
                if (exact) x = __fadd_rn(__fadd_rn(__fmul_rn(x, c), k.y), mv[j]);
                else x = __fadd_rn(__fmaf_rn(x, c, mv[j]), k.y);
                top = fmaxf(top, x);
              }
            }
          }
          return !(seen && top > 11.0f);
        };
        bool raise = t == s.t0;
        if (!raise) {
          raise = __any_sync(0xffffffffu, !weights());
          if (lane == 0) vote_s[(g & 1) * 4 + quad] = raise;
          arrive(vote);
          if (!(ok = wait(vote, g & 1))) break;
          int any = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) any |= vote_s[(g & 1) * 4 + i];
          raise = any != 0;
        } else {
          if (!(ok = wait(q_full + (segs & 1), segs >> 1 & 1))) break;  // (their powers of two)
          arrive(vote);
          if (!(ok = wait(vote, g & 1))) break;
        }
        if (raise) {
          // the tile's maxima, a column at a time, and new references where they pass
          const bool start = t == s.t0;
#pragma unroll 1
          for (int i = 0; i < N; i += 16) {
            float x[16];
            tc::tmem_ld16(s_addr + i, x);
            tc::tmem_wait_ld(x);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              x[e] = __fadd_rn(__fmul_rn(x[e], k.x * qs[i + e]), k.y);
              x[e] = seen && x[e] > -INFINITY ? x[e] : -INFINITY;  // (NaN as well)
            }
            const float top = att::reduce_columns<16, true>(x, lane);
            if (!(lane & 1)) quad_s[quad * N + i + lane / 2] = top;
          }
          if (!(ok = together())) break;
          const float* nm0 = nm_s + cur * N;
          cur ^= 1;
          bool some = false, far = false;  // O to be scaled; a reference far from 0
          for (int r = lane; r < N; r += 32) {
            const float top = fmaxf(fmaxf(quad_s[r], quad_s[N + r]), fmaxf(quad_s[2 * N + r], quad_s[3 * N + r]));
            const float was = start ? -INFINITY : nm0[r];
            const float to = 4.0f - ceilf(fmaxf(top, -att::kLargest));
            const bool none = was == -INFINITY, over = top > -INFINITY && (none || top + was > 11.0f);
            const float now = over ? to : was;
            const float f = over && !none ? ex2(to - was) : 1.0f;
            // (all four warps write the same)
            nm_s[cur * N + r] = now;
            f_s[cur * N + r] = f;
            some |= f != 1.0f;
            far |= now > -INFINITY && fabsf(now) > 1048576.0f;
          }
          __syncwarp();
          some = __any_sync(0xffffffffu, some);
          exact = __any_sync(0xffffffffu, far);
          if (some) {
            const float* f = f_s + cur * N;
#pragma unroll
            for (int r = 0; r < N; ++r) l[r] *= f[r];
            if (!(ok = wait(pv_done, (g - 1) & 1))) break;
            tc::fence_after_sync();
#pragma unroll 1
            for (int i = 0; i < N; i += 8) {
              float o[8];
              att::tmem_load(o_addr + i, o);
#pragma unroll
              for (int e = 0; e < 8; ++e) o[e] *= f[i + e];
              att::tmem_store8(o_addr + i, o);
            }
            tc::tmem_wait_st();
          }
          weights();
        }
        const float share_b = ex2(-k.y);  // (b goes out of the denominators)
        const uint32_t p0 = tc::smem_u32(p_at + (g & 1) * C::PB);
#pragma unroll
        for (int i = 0; i < N; i += 8) {
          uint32_t y[4];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float w = seen ? ex2(v[i + e]) : 0.0f;
            l[i + e] += seen ? w * share_b : 0.0f;
            v[i + e] = w;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = pack_f16(v[i + 2 * e], v[i + 2 * e + 1]);
          att::st_shared16(p0 + p_chunk(row, i), make_uint4(y[0], y[1], y[2], y[3]));
        }
        tc::fence_before_sync();
        arrive(p_full + (g & 1));
      }
      if (!ok) break;
      // ---- the result ----
#pragma unroll
      for (int i = 0; i < N; i += 16) {
        const float sum = att::reduce_columns<16, false>(reinterpret_cast<float(&)[16]>(l[i]), lane);
        if (!(lane & 1)) sum_s[quad * N + i + lane / 2] = sum;
      }
      if (!(ok = together())) break;
      if (!(ok = wait(o_full, segs & 1))) break;
      tc::fence_after_sync();
      auto sum_of = [&](int r) { return sum_s[r] + sum_s[N + r] + (sum_s[2 * N + r] + sum_s[3 * N + r]); };
      const bool part = s.part >= 0;
      if (row < D) {
#pragma unroll 1
        for (int i = 0; i < a.G; i += 16) {
          float o[16];
          tc::tmem_ld16(o_addr + i, o);
          tc::tmem_wait_ld(o);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int r = i + e;
            if (r >= a.G) break;
            const float sum = sum_of(r), x = o[e] * (part ? ref : sum == 0.0f ? 0.0f : ref / sum);
            if (part) a.part[((size_t)s.part * a.rows + r) * D + row] = x;
            else a.out[(at + r) * D + row] = __float2bfloat16_rn(x);
          }
        }
      }
      if (row < a.G) {
        const float sum = sum_of(row), m = nm_s[cur * N + row];
        if (part) a.ml[(size_t)s.part * a.rows + row] = make_float2(sum, m);
        else if (a.lse) a.lse[at + row] = sum == 0.0f ? -INFINITY : (log2f(sum) - m) * att::kLn2;
      }
      arrive(q_empty + (segs & 1));  // (their powers of two)
      // (the next sums are written after the next tile's vote, and maxima after another vote)
      ++segs;
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

template <class C>
cudaError_t launch_attend_tokens(const AttendArgs& a, int ctas, cudaStream_t st) {
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
    if (fa.numRegs < kRegsLaunch) return cudaErrorLaunchOutOfResources;
    __atomic_store_n(&regs_ok, 1, __ATOMIC_RELAXED);
  }
  const cudaError_t e =
      att::launch_opted_in(reinterpret_cast<const void*>(kernel), C::SMEM, &opted_in, [&] {
        return launch_early(kernel, (unsigned)ctas, kThreads, C::SMEM, st, 1, a, k_map, v_map);
      });
  if (e != cudaSuccess) return e;
  return launch_early(k_join_parts<C::D>, (unsigned)(ctas * kJoinBlocks), kJoinThreads, 0, st, 1, a,
                      ctas);
}

}  // namespace pages
}  // namespace hytopk
