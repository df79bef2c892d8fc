// attend_backward_engine.cuh -- gradients of the attention over selected rows
// (hytopk_attend_backward), on the tensor cores.
//
// One work item is a query and up to N = 64 of the heads that share a cache
// head; its selected rows are gathered 128 at a time. As in the forward engine
// the rows fill the 128 lanes and the heads are the narrow side. Per tile, with
// P = exp(S - lse) and dS = P (dP - grad . out):
//
//   S^T  [128 rows x N]   = K . Q^T           dP^T [128 rows x N] = V . dO^T
//   dV^T [d x 128 rows]   = dO^T . P^T        (A: M = d contiguous; B: P as
//   dK^T [d x 128 rows]   = Q^T . dS^T         [row][head], K-major)
//   dQ^T [d x N]         += K^T . dS^T        (A: K as gathered, M = d contiguous;
//                                              B: dS as [row][head], N contiguous)
//
// The results are fp32, so P and dS are written as three bf16 parts (24 bits)
// and their products take three terms; the other operands are bf16 as given.
// dQ^T takes the first two parts side by side (N = 128) and adds the third to
// the second's columns.
//
// Measured: 2048 queries of 64 heads, 2048 rows of 128 columns: 1215 us (283 TFLOP/s,
// additions 3.5 TB/s); of 16 heads 840 us (5.1 TB/s); 64 columns 1063 us. Bound by the
// chain of a tile at 64 heads (80 % of the time remains with no row selected; 18000 warp
// instructions), by the additions at 16 (12700). What made it fast: read-out warps of their own
// 1640 -> 1500 us, d along the lanes (whole-line additions) -> 1350, additions predicated
// instead of branched around and addresses of one instruction -> 1250. P and dS come from
// the same code in two passes (the exponentials twice), which needs fewer registers.
//
// A tile's products keep the tensor core busy if a tile's softmax overlaps the
// products of the tile before. The order is
//   dV(g), dK(g), S(g+1) + dP(g+1), dQ(g)
// so that the rows of tile g+1 have the time of dV(g) and dK(g) to arrive (K has
// two buffers and V one: shared memory is full), dV(g) and dK(g) are added to
// global memory while later products run, and P(g+1) is computed under dQ(g).
//
// The tensor core's fp32 additions truncate, so a long chain of them drifts (128
// steps: 2e-6 of the result). dQ^T is read out and added up in global memory
// every kChunk tiles.
//
// dV and dK come out with d along the lanes, so that an addition instruction
// covers 128 consecutive bytes of one row: random rows take 6.4 TB/s of such
// additions, 3.8 TB/s in 32-byte pieces and 3.3 TB/s in 16-byte pieces (measured
// alone, 67 MB of rows). They are the bound: 8 d bytes per selected row and head
// group.
//
//   8 warps       softmax (two warpgroups, each with half of the N head columns)
//   8 warps       read-out: four add dV (and write dQ), four add dK
//   4 warps       producers (cp.async); also the row sums grad . out
//   last warp     MMA issuer, TMEM
#pragma once

#include "attend_engine.cuh"

namespace hytopk {
namespace att {

// N: 16 or 64 head columns; larger groups take several items. (2048 queries of 16 heads:
// 840 us with N = 16, 1065 with N = 64; of 128 heads, two items of 64: 2333 us.)
template <int D_, int N_>
struct BCfg {
  static constexpr int D = D_, N = N_;
  static constexpr int SWARPS = 8;
  static constexpr int HG = N / 2;             // head columns of a warpgroup
  static constexpr int CH = HG < 16 ? HG : 16; // columns at a time
  static constexpr int RB = 2 * D;
  using Geo = tc::Geo<RB>;
  static constexpr int SLOT = 128 * RB;  // K or V tile
  static constexpr int PBYTES = 16384;   // one part of P or dS: 128 rows x 64 heads
  static constexpr int QBYTES = N * RB;
  static constexpr int PWARPS = 4;
  static constexpr int PROD_WARP = SWARPS + 8;
  static constexpr int MMA_WARP = PROD_WARP + PWARPS;
  static constexpr int THREADS = (MMA_WARP + 1) * 32;
  static constexpr int K_OFF = 0;                 // two buffers
  static constexpr int V_OFF = 2 * SLOT;
  static constexpr int P_OFF = 3 * SLOT;          // three parts
  static constexpr int S_OFF = P_OFF + 3 * PBYTES;
  static constexpr int Q_OFF = S_OFF + 3 * PBYTES;
  static constexpr int G_OFF = Q_OFF + QBYTES;    // gradient rows
  static constexpr int MISC_OFF = G_OFF + QBYTES;
  static constexpr int MISC = 4 * N * 4 + 256;    // -lse, -grad . out [2][N]; barriers
  // d = 64 has one 64-column atom; the second one that M = 128 takes is what
  // follows in shared memory (for the gradient rows: this pad), and fills
  // accumulator lanes never read
  static constexpr int PAD = D == 64 ? QBYTES : 0;
  static constexpr int SMEM = MISC_OFF + MISC + PAD + 1024;
  // TMEM columns
  static constexpr int S_COL = 0, DP_COL = N, DV_COL = 128, DK_COL = 256, DQ_COL = 384;
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static_assert(2 * N <= 128, "TMEM columns");
};

__device__ __forceinline__ void red_add(float* p, float v) {
  asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" ::"l"(p), "f"(v) : "memory");
}
// the same if row >= 0, without a branch
__device__ __forceinline__ void red_add_if(int row, void* p, float v) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ge.s32 p, %2, 0;\n @p red.relaxed.gpu.global.add.f32 [%0], %1;\n}\n" ::"l"(p),
      "f"(v), "r"(row)
      : "memory");
}

// The three bf16 parts of W weights of a row, to the three part buffers.
template <int W>
__device__ __forceinline__ void store_parts(uint8_t* dst, int row, int c0, float (&v)[W]) {
#pragma unroll
  for (int part = 0; part < 3; ++part) {
#pragma unroll
    for (int u = 0; u < W; u += 8) {
      uint32_t x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = pack_bf16(v[u + 2 * e], v[u + 2 * e + 1]);
        if (part < 2) take_bf16(x[e], v[u + 2 * e], v[u + 2 * e + 1]);
      }
      *reinterpret_cast<uint4*>(dst + part * 16384 + p_offset(row, c0 + u)) =
          make_uint4(x[0], x[1], x[2], x[3]);
    }
  }
}

// SPLIT: CTAs share an item (an instance of its own: the others are 1 to 2 % faster
// without it). PART: an item may have fewer than N heads (likewise: 64 heads 1215 us without
// it, 1238 with).
template <class C, bool OUT_F32, bool SPLIT, bool PART>
__global__ void __launch_bounds__(C::THREADS, 1) k_attend_backward(const Args a, const Plan pl) {
  constexpr int D = C::D, N = C::N, HG = C::HG, CH = C::CH;
  using Geo = typename C::Geo;
  extern __shared__ __align__(1024) uint8_t smem_dyn[];
  uint8_t* smem = tc::align1024(smem_dyn);
  float* nl_s = reinterpret_cast<float*>(smem + C::MISC_OFF);  // [2][N] -lse (log2)
  float* nd_s = nl_s + 2 * N;                                  // [2][N] -grad . out
  uint64_t* bars = reinterpret_cast<uint64_t*>(nd_s + 2 * N);
  uint64_t* k_full = bars;
  uint64_t* k_empty = bars + 2;
  uint64_t* v_full = bars + 4;
  uint64_t* v_empty = bars + 5;
  uint64_t* q_full = bars + 6;
  uint64_t* q_empty = bars + 7;
  uint64_t* s_full = bars + 8;
  uint64_t* s_empty = bars + 9;
  uint64_t* p_full = bars + 10;
  uint64_t* ds_full = bars + 11;
  uint64_t* ds_empty = bars + 12;
  uint64_t* dv_full = bars + 13;
  uint64_t* dv_empty = bars + 14;
  uint64_t* dk_full = bars + 15;
  uint64_t* dk_empty = bars + 16;
  uint64_t* dq_full = bars + 17;
  uint64_t* dq_empty = bars + 18;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 19);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(k_full + i, C::PWARPS * 32);
      tc::mbar_init(k_empty + i, 1);
    }
    tc::mbar_init(v_full, C::PWARPS * 32);
    tc::mbar_init(q_full, C::PWARPS);
    uint64_t* by_mma[] = {v_empty, q_empty, s_full, ds_empty, dv_full, dk_full, dq_full};
    for (uint64_t* b : by_mma) tc::mbar_init(b, 1);
    uint64_t* by_softmax[] = {s_empty, p_full, ds_full};
    for (uint64_t* b : by_softmax) tc::mbar_init(b, C::SWARPS);
    uint64_t* by_read[] = {dv_empty, dk_empty, dq_empty};
    for (uint64_t* b : by_read) tc::mbar_init(b, 4);
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
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  allow_next();
  wait_for_earlier();

  // items of this CTA: first, first + stride, ...; its tiles of each: [tile0, tile0 + ntile)
  const int first = SPLIT ? (int)blockIdx.x / pl.splits : (int)blockIdx.x;
  const int rank = SPLIT ? (int)blockIdx.x % pl.splits : 0;
  const int n_mine = pl.items > first ? (pl.items - 1 - first) / pl.stride + 1 : 0;
  const int tile0 = SPLIT ? (int)((int64_t)pl.tiles * rank / pl.splits) : 0;
  const int ntile = SPLIT ? (int)((int64_t)pl.tiles * (rank + 1) / pl.splits) - tile0 : pl.tiles;
  const int total = n_mine * ntile;
  const int Hq = a.Hkv * a.G;
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
  const int left = a.k_top - tile0 * 128;
  const int32_t* idx = a.idx + tile0 * 128;
  auto entry_of = [&](int t, int j) -> int {  // of this CTA's share
    return j < left ? ld_after(idx + (size_t)t * a.k_top + j) : -1;
  };
  auto row_of = [&](int e) -> int { return e >= a.L || e < 0 ? -1 : e; };

  if (warp >= C::PROD_WARP && warp < C::MMA_WARP) {
    // ---------------- producers ----------------
    const int tid = threadIdx.x - C::PROD_WARP * 32;
    const int pw = warp - C::PROD_WARP;
    constexpr int CPR = C::RB / 16;              // 8 or 16
    constexpr int RPP = 32 / CPR;
    constexpr int PASSES = 32 / RPP;
    constexpr int SHIFT = CPR == 16 ? 4 : 3;
    // The item's query and gradient rows (zero beyond its heads), its -lse and
    // its row sums grad . out (padded heads: weights of zero).
    auto load_query = [&](int qi, const Walk& w) -> bool {
      const int h0 = first_head(w), nh = head_count(w);
      const size_t at = (size_t)w.t * Hq + h0;
      const __nv_bfloat16* grad = static_cast<const __nv_bfloat16*>(a.grad) + at * D;
      float* nl = nl_s + (qi & 1) * N;
      float* nd = nd_s + (qi & 1) * N;
      constexpr int EL = D / 32;  // elements of a row per lane
#pragma unroll 4
      for (int h = pw; h < N; h += C::PWARPS) {
        float sum = 0.0f;
        if (h < nh) {
#pragma unroll
          for (int e = 0; e < EL; ++e) {
            const size_t i = (size_t)h * D + e * 32 + lane;
            const float o = OUT_F32 ? ld_after(static_cast<const float*>(a.out) + at * D + i)
                                    : __bfloat162float(static_cast<const __nv_bfloat16*>(a.out)[at * D + i]);
            sum = __fmaf_rn(__bfloat162float(grad[i]), o, sum);
          }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) {
          const float lse = h < nh ? ld_after(a.lse + at + h) : -INFINITY;
          nd[h] = -sum;
          nl[h] = lse == -INFINITY ? -INFINITY : -lse * kLog2e;
        }
      }
      const bool ok = wait_bar(q_empty, (qi & 1) ^ 1, abort_flag, a.status);
      if (!__all_sync(0xffffffffu, ok)) return false;
      const uint8_t* qsrc = static_cast<const uint8_t*>(a.q) +
                            ((size_t)w.t * a.q_row + (size_t)h0 * D) * 2;
      constexpr int PER = N * CPR / (C::PWARPS * 32);
      constexpr int U = PER < 4 ? PER : 4;
#pragma unroll 1
      for (int p = 0; p < PER; p += U) {
        uint4 v[U], x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int f = (p + u) * C::PWARPS * 32 + tid;
          v[u] = x[u] = make_uint4(0, 0, 0, 0);
          if (f / CPR < nh) {
            v[u] = ld_after(reinterpret_cast<const uint4*>(qsrc) + f);
            x[u] = ld_after(reinterpret_cast<const uint4*>(grad) + f);
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int f = (p + u) * C::PWARPS * 32 + tid;
          const uint32_t off = Geo::chunk_offset(f / CPR, f % CPR, N);
          *reinterpret_cast<uint4*>(smem + C::Q_OFF + off) = v[u];
          *reinterpret_cast<uint4*>(smem + C::G_OFF + off) = x[u];
        }
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(q_full);
      return true;
    };
    Walk w = start, wn = w;
    int qi = 0;
    bool ok = true;
    int e_next = total > 0 ? entry_of(w.t, tid) : -1;
#pragma unroll 1
    for (int g = 0; g < total && ok; ++g, w = wn) {
      const int s_own = row_of(e_next);
      int rows[PASSES];
#pragma unroll
      for (int p = 0; p < PASSES; ++p)
        rows[p] = __shfl_sync(0xffffffffu, s_own, p * RPP + (lane >> SHIFT));
      if (g + 1 < total) {
        walk_next(wn);
        e_next = entry_of(wn.t, wn.i * 128 + tid);
      }
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv) {
        uint64_t* empty = kv ? v_empty : k_empty + (g & 1);
        uint64_t* full = kv ? v_full : k_full + (g & 1);
        const uint32_t parity = kv ? (g & 1) ^ 1 : ((g >> 1) & 1) ^ 1;
        ok = __all_sync(0xffffffffu, wait_bar(empty, parity, abort_flag, a.status));
        if (!ok) break;
        const uint32_t dst = tc::smem_u32(smem + (kv ? C::V_OFF : C::K_OFF + (g & 1) * C::SLOT));
        const int c = lane & ((1 << SHIFT) - 1);
        const uint8_t* base = static_cast<const uint8_t*>(kv ? a.v : a.k) + (size_t)w.hk * C::RB + c * 16;
        const int64_t row_bytes = (kv ? a.v_row : a.k_row) * 2;
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
          const int s = rows[p];
          cp_async16(dst + Geo::chunk_offset(pw * 32 + p * RPP + (lane >> SHIFT), c, 128),
                     base + (s >= 0 ? s * row_bytes : 0), s >= 0);
        }
        cp_async_arrive(full);
      }
      if (ok && w.i == 0 && !load_query(qi++, w)) break;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == C::MMA_WARP) {
    // ---------------- MMA issuer (whole warp, one elected lane issues) ----------------
    constexpr uint32_t ID_S = tc::instr_desc(0, 128, N);
    constexpr uint32_t ID_DV = tc::instr_desc(0, 128, 128) | (1u << 15);
    constexpr uint32_t ID_DQ2 = tc::instr_desc(0, 128, 128) | (1u << 15) | (1u << 16);
    constexpr uint32_t ID_DQ1 = tc::instr_desc(0, 128, 64) | (1u << 15) | (1u << 16);
    constexpr uint32_t D_HI = (1024u >> 4) | (1u << 14) | (2u << 29);
    constexpr uint32_t LBO_K = 1u << 16, LBO_MN = (16384u >> 4) << 16;
    constexpr uint32_t LBO_Q = ((uint32_t)(N * 128) >> 4) << 16;
    auto low = [](const void* p) { return (tc::smem_u32(p) >> 4) & 0x3FFFu; };
    auto desc = [&](uint32_t lo) { return tc::desc_from_words(lo, D_HI); };
    const uint32_t k_lo = low(smem + C::K_OFF), v_lo = low(smem + C::V_OFF);
    const uint32_t p_lo = low(smem + C::P_OFF), s_lo = low(smem + C::S_OFF);
    const uint32_t q_lo = low(smem + C::Q_OFF), g_lo = low(smem + C::G_OFF);
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, wait_bar(bar, parity, abort_flag, a.status)) != 0;
    };
    int si = 0, sq = 0;  // tile of its item and item of the next scores
    auto scores = [&](int g) -> bool {
      if (si == 0 && !wait(q_full, sq & 1)) return false;
      if (!wait(k_full + (g & 1), (g >> 1) & 1)) return false;
      if (!wait(v_full, g & 1)) return false;
      if (!wait(s_empty, (g & 1) ^ 1)) return false;
      tc::fence_proxy_async_smem();
      tc::fence_after_sync();
      const uint32_t ka = (k_lo + (g & 1) * (C::SLOT >> 4)) | LBO_K;
      if (elect_one()) {
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
          tc::mma<0>(tmem + C::S_COL, desc(ka + (Geo::step_offset(j, 128) >> 4)),
                     desc((q_lo | LBO_K) + (Geo::step_offset(j, N) >> 4)), ID_S, j > 0 ? 1u : 0u);
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
          tc::mma<0>(tmem + C::DP_COL, desc((v_lo | LBO_K) + (Geo::step_offset(j, 128) >> 4)),
                     desc((g_lo | LBO_K) + (Geo::step_offset(j, N) >> 4)), ID_S, j > 0 ? 1u : 0u);
        tc::mma_commit(s_full);
        tc::mma_commit(v_empty);
      }
      __syncwarp();
      if (++si == ntile) {
        si = 0;
        ++sq;
      }
      return true;
    };
    // D [d x 128 rows] = sum over the parts of A ([head][d]) . B (K-major, [row][head])
    auto rows_product = [&](uint32_t col, uint32_t a_lo, uint32_t b_lo) {
#pragma unroll
      for (int part = 0; part < 3; ++part)
#pragma unroll
        for (int s = 0; s < N / 16; ++s)
          tc::mma<0>(tmem + col, desc((a_lo | LBO_Q) + ((s * 2048) >> 4)),
                     desc((b_lo | LBO_K) + ((part * C::PBYTES + s * 32) >> 4)), ID_DV,
                     (part > 0 || s > 0) ? 1u : 0u);
    };
    int i = -1, nq = 0;  // tile of its item; chunks of dQ begun
    bool ok = true;
#pragma unroll 1
    for (int g = -1; g < total && ok; ++g) {
      const bool last = i == ntile - 1;
      if (g >= 0) {
#pragma unroll 1
        for (int k = 0; k < 2 && ok; ++k) {  // dV, dK
          ok = wait(k ? dk_empty : dv_empty, (g & 1) ^ 1) && wait(k ? ds_full : p_full, g & 1);
          if (!ok) break;
          tc::fence_proxy_async_smem();
          tc::fence_after_sync();
          if (elect_one()) {
            rows_product(k ? C::DK_COL : C::DV_COL, k ? q_lo : g_lo, k ? s_lo : p_lo);
            tc::mma_commit(k ? dk_full : dv_full);
            if (k && last) tc::mma_commit(q_empty);
          }
          __syncwarp();
        }
      }
      // the next tile's scores, then this one's dQ; the next item's scores wait for
      // its queries, so they come after dQ
#pragma unroll 1
      for (int k = 0; k < 2 && ok; ++k) {
        if ((k == 0) != (last && g >= 0)) {
          if (g + 1 < total) ok = scores(g + 1);
        } else if (g >= 0) {
          const bool begin = i % kChunk == 0, end = i % kChunk == kChunk - 1 || last;
          if (begin && !(ok = wait(dq_empty, (nq++ & 1) ^ 1))) break;
          const uint32_t ka = (k_lo + (g & 1) * (C::SLOT >> 4)) | LBO_MN;
          if (elect_one()) {
#pragma unroll
            for (int s = 0; s < 8; ++s)  // 16 rows each
              tc::mma<0>(tmem + C::DQ_COL, desc(ka + ((s * 2048) >> 4)),
                         desc((s_lo | LBO_MN) + ((s * 2048) >> 4)), ID_DQ2,
                         (!begin || s > 0) ? 1u : 0u);
#pragma unroll
            for (int s = 0; s < 8; ++s)
              tc::mma<0>(tmem + C::DQ_COL + 64, desc(ka + ((s * 2048) >> 4)),
                         desc((s_lo | LBO_MN) + ((2 * C::PBYTES + s * 2048) >> 4)), ID_DQ1, 1u);
            tc::mma_commit(ds_empty);
            tc::mma_commit(k_empty + (g & 1));
            if (end) tc::mma_commit(dq_full);
          }
          __syncwarp();
        }
      }
      if (++i == ntile) i = 0;
    }
  } else if (warp < C::SWARPS) {
    // ---------------- softmax: TMEM lane = selected row ----------------
    const int wg = warp >> 2, quad = warp & 3;
    const int row = quad * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const int c0 = wg * HG;
    const float c_scale = a.scale * kLog2e;
    auto arrive = [&](uint64_t* bar) {
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar);
    };
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, wait_bar(bar, parity, abort_flag, a.status)) != 0;
    };
    Walk w = start;
    int i = 0, qi = 0, heads = 0;  // tile of its item, item, its heads from c0 on
    bool ok = true;
    int e_next = total > 0 ? entry_of(w.t, row) : -1;
#pragma unroll 1
    for (int g = 0; g < total; ++g) {
      if (PART && i == 0) heads = head_count(w) - c0;
      const bool valid = row_of(e_next) >= 0;
      if (e_next != -1 && !valid && wg == 0 && a.status) atomicOr(a.status, HYTOPK_DEV_BAD_INDEX);
      if (g + 1 < total) {
        walk_next(w);
        e_next = entry_of(w.t, w.i * 128 + row);
      }
      if (i == 0 && !wait(q_full, qi & 1)) break;
      if (!wait(s_full, g & 1)) break;
      tc::fence_after_sync();
      const float* nl = nl_s + (qi & 1) * N + c0;
      const float* nd = nd_s + (qi & 1) * N + c0;
      // pass 0: P, once its last reader, the dV of the tile before, is done;
      // pass 1: dS, once the dQ of the tile before is
#pragma unroll 1
      for (int pass = 0; pass < 2 && ok; ++pass) {
        if (g > 0) ok = wait(pass ? ds_empty : dv_full, (g - 1) & 1);
        uint8_t* dst = smem + (pass ? C::S_OFF : C::P_OFF);
#pragma unroll 1
        for (int cc = 0; cc < HG; cc += CH) {
          float p[CH];
          tmem_load(tmem + lane_off + C::S_COL + c0 + cc, p);
#pragma unroll
          for (int u = 0; u < CH; u += 2) {
            fma2(p[u], p[u + 1], c_scale, nl[cc + u], nl[cc + u + 1]);
            p[u] = valid ? ex2(p[u]) : 0.0f;
            p[u + 1] = valid ? ex2(p[u + 1]) : 0.0f;
          }
          if (pass) {
            float dp[CH];
            tmem_load(tmem + lane_off + C::DP_COL + c0 + cc, dp);
#pragma unroll
            for (int u = 0; u < CH; u += 2) {
              add2(dp[u], dp[u + 1], nd[cc + u], nd[cc + u + 1]);
              mul2(dp[u], dp[u + 1], a.scale, a.scale);  // here, so that dQ and dK come out scaled
              mul2(dp[u], dp[u + 1], p[u], p[u + 1]);
              p[u] = valid ? dp[u] : 0.0f;  // (0 x NaN of a gradient is none of this row's)
              p[u + 1] = valid ? dp[u + 1] : 0.0f;
            }
          }
          // of heads past the group's: their rows are zeros, but 0 times a key that is not
          // finite is not
          if (PART && cc + CH > heads) {
#pragma unroll
            for (int u = 0; u < CH; ++u) p[u] = cc + u < heads ? p[u] : 0.0f;
          }
          store_parts<CH>(dst, row, c0 + cc, p);
        }
        if (pass) {
          // scores and the item's sums are read: both may be replaced
          tc::fence_before_sync();
          arrive(s_empty);
        }
        arrive(pass ? ds_full : p_full);
      }
      if (!ok) break;
      if (++i == ntile) {
        i = 0;
        ++qi;
      }
    }
  } else if (warp < C::PROD_WARP) {
    // ---------------- read-out: TMEM lane = d ----------------
    const int quad = warp & 3;
    const int row = quad * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    auto arrive = [&](uint64_t* bar) {
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar);
    };
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      const bool ok = __all_sync(0xffffffffu, wait_bar(bar, parity, abort_flag, a.status)) != 0;
      tc::fence_after_sync();
      return ok;
    };
    const bool is_dk = warp >= C::SWARPS + 4;
    uint64_t* full = is_dk ? dk_full : dv_full;
    uint64_t* empty = is_dk ? dk_empty : dv_empty;
    const uint32_t addr = tmem + lane_off + (is_dk ? C::DK_COL : C::DV_COL);
    const uint32_t stride = (uint32_t)a.Hkv * D * 4;  // bytes of a row of dk and dv
    Walk w = start, wf = start;
    int nq = 0;
    int e_next = total > 0 ? entry_of(w.t, lane) : -1;  // of the next 32 rows
#pragma unroll 1
    for (int g = 0; g < total; ++g) {
      walk_next(wf);
      if (!wait(full, g & 1)) break;
      uint8_t* dst = reinterpret_cast<uint8_t*>((is_dk ? a.dk : a.dv) + (size_t)w.hk * D + row);
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        const int s = row_of(e_next);
        if (q < 3) e_next = entry_of(w.t, w.i * 128 + 32 * (q + 1) + lane);
        else if (g + 1 < total) e_next = entry_of(wf.t, wf.i * 128 + lane);
        if (quad * 32 < D) {
          float x[32];
          tmem_load(addr + 32 * q, x);
#pragma unroll
          for (int b = 0; b < 32; b += 8) {
            int r[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) r[u] = __shfl_sync(0xffffffffu, s, b + u);
#pragma unroll
            for (int u = 0; u < 8; ++u)  // 32 x 32 + 64 bits: one instruction an address
              red_add_if(r[u], dst + (uint64_t)(uint32_t)r[u] * stride, x[b + u]);
          }
        }
      }
      arrive(empty);
      if (!is_dk && (w.i % kChunk == kChunk - 1 || w.i == ntile - 1)) {
        // dQ^T of the chunk, the parts' two column blocks summed
        if (!wait(dq_full, nq++ & 1)) break;
        const int nh = head_count(w);
        float* dst = a.dq + ((size_t)w.t * Hq + first_head(w)) * D + row;
        if (quad * 32 < D) {
#pragma unroll 1
          for (int cc = 0; cc < nh; cc += 16) {
            float x[16], y[16];
            tmem_load(tmem + lane_off + C::DQ_COL + cc, x);
            tmem_load(tmem + lane_off + C::DQ_COL + 64 + cc, y);
#pragma unroll
            for (int u = 0; u < 16; ++u) {
              if (cc + u < nh) {
                const float v = x[u] + y[u];
                if (!SPLIT && w.i < kChunk) dst[(size_t)(cc + u) * D] = v;
                else red_add(dst + (size_t)(cc + u) * D, v);  // after this thread's own store
              }
            }
          }
        }
        arrive(dq_empty);
      }
      w = wf;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == C::MMA_WARP) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

template <class C, bool OUT_F32>
cudaError_t launch_backward(const Args& a, int sms, cudaStream_t st) {
  static unsigned long long opted_in[4] = {0, 0, 0, 0};
  Plan pl{};
  pl.blocks = (a.G + C::N - 1) / C::N;
  pl.heads = (a.G + pl.blocks - 1) / pl.blocks;
  pl.tiles = (a.k_top + 127) / 128;
  pl.items = a.n * a.Hkv * pl.blocks;
  pl.stride = pl.items < sms ? pl.items : sms;
  // Few items: CTAs share an item's tiles, as many as there are multiprocessors for; each
  // adds its part of dQ to zeros. (64 queries of 64 heads, 2048 rows: 101 -> 63 us.)
  pl.splits = sms / pl.items < 1 ? 1 : sms / pl.items < pl.tiles ? sms / pl.items : pl.tiles;
  pl.sb = pl.stride % pl.blocks;
  pl.sh = pl.stride / pl.blocks % a.Hkv;
  pl.st = pl.stride / pl.blocks / a.Hkv;
  const bool split = pl.splits > 1, part = C::N == 16 || pl.blocks * C::N != a.G;
  auto kernel = split ? k_attend_backward<C, OUT_F32, true, true> : k_attend_backward<C, OUT_F32, false, true>;
  if constexpr (C::N != 16)  // (of 16 heads 836 and 840 us: one instance)
    if (!part)
      kernel = split ? k_attend_backward<C, OUT_F32, true, false> : k_attend_backward<C, OUT_F32, false, false>;
  const size_t rows = a.zero ? (size_t)a.L * a.Hkv * C::D : 0;
  const size_t own = split ? (size_t)a.n * a.Hkv * a.G * C::D : 0;
  const cudaError_t e = launch_zero(a.dk, a.dv, rows, a.dq, own, sms, st);
  if (e != cudaSuccess) return e;
  return launch_opted_in(reinterpret_cast<const void*>(kernel), C::SMEM, opted_in + 2 * part + split, [&] {
    return launch_early(kernel, pl.stride * pl.splits, C::THREADS, C::SMEM, st, 1, a, pl);
  });
}

}  // namespace att
}  // namespace hytopk
