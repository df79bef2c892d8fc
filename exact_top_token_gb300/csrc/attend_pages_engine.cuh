// attend_pages_engine.cuh -- attention over a cache in pages on the tensor cores
// (hytopk_attend_pages).
//
// An item is a cache head and up to 256 of the (token, head) rows that read it: tokens
// neighbour in one sequence, so that they share keys. Keys are taken 128 at a time (a
// tile); the rows are the 128 lanes of the tensor core, two blocks of them:
//
//   S [128 rows x 128 keys]  = Q . K^T    (both from shared memory, K-major)
//   O [128 rows x d]        += P . V      (P from tensor memory, where it takes S's place)
//
// so a thread of the softmax owns a row: its maximum and sum need no other lane. Items of
// more than a block of rows (A) give each of the two warpgroups a block, and both use every
// tile; smaller ones, single tokens above all (B), give both warpgroups the same rows and
// every other tile each, and the two results are joined in tensor memory.
//
// e4m3 codes are widened to f16, which holds every e4m3 value. The page scales never touch
// them: sixteen neighbouring keys lie in one page (a group), so k's scale is a factor of a
// group's scores, and v's, as b = log2(v_scale / reference), a summand of its exponents. The
// weights 2^(s + b - m) are what is rounded to f16 and multiplied with the codes; their sum
// over a group times 2^-b is the group's share of the softmax's denominator. m is at least the
// largest s + b of an item's first tile less 4, and is raised, with O and the tile's
// weights so far scaled, when a weight would pass 2^11. So the largest weight is above 2^3, f16
// keeps 11 bits down to 2^-14, and a weight below that, less than 2^-17 of the largest product
// with v's scale, has an error of 2^-25, less than 2^-28 of it. m is a whole number, so that
// s + (b - m) is rounded once. Queries are taken to f16 with a power of two out of each row.
//
// That is the quick form. Scales of v that lie 2^60 and more from the reference, or scores so far
// from 0 that b is lost beside m, take a slow one from there to the segment's end: denominators
// have a reference m' of their own, the largest s or so, and weights are 2^(((s - m') + b) + d).
// It reads the scores three times: 64 rows 183 -> 309 us where all tiles take it, a prompt of 8192
// 527 -> 1085. Results of parts are kept divided by their denominators, so that no product of a
// scale and a weight passes the range of fp32.
//
// A masked weight is 0 whatever the score is, but 0 times a NaN code of v is not: in the
// tiles that hold keys some row does not see, NaN codes of v are replaced by 0 and, by column,
// the first key that has one is kept; the rows that see it become NaN there at the end.
//
// The work of a call is only known on the device (contexts and their new rows). Every CTA
// adds it up, in units of a tile's time, and takes an equal share of it in order, tile by
// tile: an item that lies in several shares leaves parts in the workspace, each with its sum,
// and a second kernel joins them. The result does not depend on timing. A row of a page holds
// all cache heads, so neighbouring CTAs take the same places of different heads: read by
// themselves, pieces of 128 bytes 1 KB apart come at 4.1 TB/s, whole rows at 5.4.
//
//   warp 0        tensor memory
//   warp 1        this CTA's segments: (item, tiles) in order, and the tiles' scales, through rings
//   warp 2        codes of the tiles by TMA
//   warp 3        products
//   warps 4-11    softmax, two warpgroups; queries; results
//   warps 12-15   codes to f16, as they land, into the ring of operands
//
// What bounds it: a prompt of 8192 tokens (32 heads of 128 on 4) takes 555 us, 990 TFLOP/s. A
// tile of two blocks takes 4200 cycles: its products alone 2048, shared memory for them, the
// codes and their f16 form 2560, the softmax 2300 on the same schedulers, and a warpgroup's
// softmax waits for its own products. At 560 us, weights handed over by halves of a tile, with
// scores by halves (649) or whole (600), two more softmax warpgroups (593), twice the widening
// warps (573) and a sum in place of the maximum (573) were slower. One token of 64 heads on one
// cache head over 2^20 keys takes 88 us, 3.05 TB/s: 2300 cycles a tile, 1750 of them shared
// memory's for operands of 128 rows, half of which no head uses. Where a sequence has one token
// and few heads share a cache head, attend_pages_tokens.cuh is faster.
#pragma once

#include "attend_engine.cuh"
#include "attend_pages.h"
#include "launch.h"

namespace hytopk {
namespace pages {

using att::add2;
using att::elect_one;
using att::ex2;
using att::fma2;
using att::max3;

constexpr int kOverhead = 8;   // of an item, in the units below
constexpr int kSegs = 8;       // ring of segments
constexpr int kConsts = 16;    // ring of the tiles' scales
constexpr int kThreads = 512;
constexpr int kBlock = 4;      // groups of 16 keys that the softmax takes at a time
// The quick form of the softmax has one reference m for weights and denominators: |b| may be up to
// kWide in it (of 2^60, 2^11 and 2^31 keys fp32 holds the product), and |m| up to kFar, where
// b - m is rounded by 2^-13 at most and v's scale by 8.5e-5 (bf16 results by 2e-3 and more).
constexpr float kWide = 60.0f, kFar = 4096.0f;
// Registers: 128 a thread at launch, then by role: 128 (64 + 2 * 184 + 80) = 65536.
constexpr int kRegsLaunch = 128, kRegsCtl = 64, kRegsSoft = 184, kRegsWide = 80;
static_assert(kRegsCtl + 2 * kRegsSoft + kRegsWide <= 4 * kRegsLaunch, "register split");

// A segment: tiles [t0, t1) of an item.
struct Seg {
  int b, hk, row0, tokens;  // sequence, cache head, first row of q, tokens
  int p0, end;              // position of the first token; keys of the last one
  int t0, t1;
  int flags, part;          // part: its number, -1: the whole item
};
enum : int { kStop = 1, kSmall = 2, kStarts = 4, kEnds = 8 };

struct TileConst {
  float4 group[4];  // of two groups: factor of the scores, b
  float ref;        // reference of v's scales
  uint32_t odd;     // bits of the groups: 0 on: rows that are not there, 8 on: b past kWide
  uint32_t pad[2];
};

template <int D_>
struct PCfg {
  static constexpr int D = D_;
  static constexpr int RB = 2 * D;
  using Geo = tc::Geo<RB>;
  static constexpr int SLOT = 128 * RB;
  static constexpr int NS = D == 128 ? 4 : 8;  // even: K in even slots, V in odd ones
  // V of a later item is written while results of item i are awaited: with V of item
  // i + 1 held back, up to V of item i + NS / 2.
  static constexpr int NANS = NS / 2 + 2;  // items whose NaN columns are kept
  // Codes on their way, a unit K or V of a tile. For d = 128 shared memory holds one beside
  // large items; small ones, which wait for memory rather than for the tensor core, have
  // two more in the place of the second block of queries.
  static constexpr int UNIT = 128 * D;
  static constexpr int UNITS = D == 128 ? 1 : 6;
  static constexpr bool SHARED = D == 128;
  static constexpr int SMALL_UNITS = SHARED ? UNITS + SLOT / UNIT : UNITS;
  static constexpr int Q_OFF = NS * SLOT;
  static constexpr int STAGE_OFF = Q_OFF + 2 * SLOT;
  static constexpr int NAN_OFF = STAGE_OFF + UNITS * UNIT;
  static constexpr int CONST_OFF = NAN_OFF + NANS * 2 * D * 4;
  static constexpr int SEG_OFF = CONST_OFF + kConsts * (int)sizeof(TileConst);
  static constexpr int ML_OFF = SEG_OFF + kSegs * (int)sizeof(Seg);
  static constexpr int QS_OFF = ML_OFF + 128 * 12;
  static constexpr int EPI_OFF = (QS_OFF + 2 * 128 * 4 + 15) / 16 * 16;  // [8 warps][1 KB]
  static constexpr int BAR_OFF = EPI_OFF + 8 * 1024;
  static constexpr int SMEM = BAR_OFF + 896 + 1024;
  static constexpr int S_COL = 0, O_COL = 256, COLS = 512;
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static_assert(NS % 2 == 0, "K in even slots, V in odd ones");
};

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// four codes to four f16
__device__ __forceinline__ uint2 widen(uint32_t codes) {
  uint2 r;
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n"
      " cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
      : "=r"(r.x), "=r"(r.y)
      : "r"(codes));
  return r;
}
// bytes that are NaN codes, as 0x80 each
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

// two f16 products
__device__ __forceinline__ uint32_t mul_f16(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void tmem_load8(uint32_t addr, uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_store8(uint32_t addr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(
                   addr),
               "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16};" ::"r"(addr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem], f16
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(add)
      : "memory");
}
// f16 operands, fp32 sums, M = 128
__host__ __device__ constexpr uint32_t f16_desc(int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
}

// ---- the work of a call ---------------------------------------------------------------

// sum of floor((a j + b) / m) over j < n; a, b >= 0 (lattice points under a line, by the steps of
// Euclid's algorithm)
static __device__ __noinline__ int64_t floor_sum(int64_t n, int64_t m, int64_t a, int64_t b) {
  int64_t sum = 0;
  while (n > 0) {
    if (a >= m) {
      sum += n * (n - 1) / 2 * (a / m);
      a %= m;
    }
    if (b >= m) {
      sum += n * (b / m);
      b %= m;
    }
    const int64_t y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y % m;
    const int64_t t = m;
    m = a;
    a = t;
  }
  return sum;
}

// A sequence's items for one cache head: blocks of `per` = 2 * tokens tokens.
struct Work {
  int m, start, per, count;  // start: position of the first token (may be negative)

  __device__ Work(const AttendArgs& a, const Seq& q)
      : m(q.m), start(q.length - q.m), per(2 * a.tokens), count((q.m + per - 1) / per) {}
  __device__ int tokens_of(int i) const { return min(per, m - i * per); }
  __device__ int tiles_of(int i) const {
    const int last = start + i * per + tokens_of(i) - 1;
    return last < 0 ? 0 : (last >> 7) + 1;
  }
  // a tile of a large item takes twice a small one's time
  __device__ int unit_of(int i) const { return 2 * tokens_of(i) > per ? 2 : 1; }
  __device__ int64_t weight_of(int i) const {
    return kOverhead + (int64_t)unit_of(i) * tiles_of(i);
  }
  // weight of the items before i
  __device__ __noinline__ int64_t before(int i) const {
    if (i <= 0) return 0;
    if (i == count) return before(i - 1) + weight_of(i - 1);
    // whole items: floor((start + (j + 1) per - 1) / 128) + 1 tiles from the first that has any
    const int first = start >= 0 ? 0 : max((1 - start + per - 1) / per - 1, 0);
    int64_t w = (int64_t)kOverhead * i;
    if (i > first)
      w += 2 * (floor_sum(i - first, 128, per, (int64_t)start + (int64_t)(first + 1) * per - 1) +
                (i - first));
    return w;
  }
};

// CTA c belongs to group c % groups, which has the heads h groups + c % groups; shares are numbered
// group by group. Where a share begins: item `i` of the group's head `h` of sequence `b`, and
// its first unit, all in units of the group's work.
struct Share {
  int64_t lo, hi, at;
  int b, h, i, any;
};
__device__ __forceinline__ int share_number(const AttendArgs& a) {
  return (int)(blockIdx.x % a.groups * (gridDim.x / a.groups) + blockIdx.x / a.groups);
}

template <int THREADS, typename T>
__device__ __forceinline__ T scan(T x, T* warps, T& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T s = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  __syncthreads();
  if (lane == 31) warps[warp] = s;
  __syncthreads();
  T before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += warps[w];
    total += warps[w];
  }
  return before + s - x;
}

// All threads; the result is in `share` (shared memory) after the next barrier. `warps`: a
// number for each warp. Whether this thread saw a sequence with several rows.
template <int THREADS>
__device__ __forceinline__ bool find_share(const AttendArgs& a, int64_t* warps, Share* share) {
  const int heads = a.Hkv / a.groups;
  int64_t mine = 0, kept = 0, total;
  bool several = false;
  for (int b = threadIdx.x; b < a.s.B; b += THREADS) {
    const Seq q = seq_of(a.s, a.n, b);
    several |= q.m > 1;
    if (q.bad && blockIdx.x == 0 && a.status) atomicOr(a.status, HYTOPK_DEV_BAD_POSITION);
    if (q.m > 0) {
      const Work w(a, q);
      kept = w.before(w.count) * heads;
      mine += kept;
    }
  }
  int64_t at = scan<THREADS>(mine, warps, total);
  const int64_t shares = gridDim.x / a.groups, number = blockIdx.x / a.groups;
  const int64_t lo = total * number / shares, hi = total * (number + 1) / shares;
  if (threadIdx.x == 0) {
    share->lo = lo;
    share->hi = hi;
    share->any = 0;
  }
  __syncthreads();
  if (lo == hi) return several;
  int64_t base = 0;
  for (int b0 = 0; b0 < a.s.B; b0 += THREADS) {
    const int b = b0 + threadIdx.x;
    int64_t all = mine;  // one pass: as it was
    if (a.s.B > THREADS) {
      all = 0;
      if (b < a.s.B) {
        const Seq q = seq_of(a.s, a.n, b);
        if (q.m > 0) {
          const Work w(a, q);
          all = w.before(w.count) * heads;
        }
      }
      at = base + scan<THREADS>(all, warps, total);
    }
    if (all > 0 && lo >= at && lo < at + all) {
      const Work w(a, seq_of(a.s, a.n, b));
      const int64_t head = all / heads;
      const int h = (int)((lo - at) / head);
      const int64_t in = lo - at - h * head;
      int i = 0, j = w.count;  // before(i) <= in < before(j)
      while (j - i > 1) {
        const int mid = (i + j) / 2;
        if (w.before(mid) <= in) i = mid;
        else j = mid;
      }
      share->b = b;
      share->h = h;
      share->i = i;
      share->at = at + h * head + w.before(i);
      share->any = 1;
    }
    base += total;
  }
  return several;
}

// A CTA's segments in order, to push(segment), which tells whether to go on, and a last one with
// kStop; the records of its parts (kStop there: there is such a part). One warp. Items whose
// rows see nothing get their results here: roles look ahead to a segment's successors, so
// any number of segments without a tile between two others would fill the ring.
template <int D, class Push>
__device__ __forceinline__ void segments(const AttendArgs& a, const Share& share, int lane, Push push) {
  const Share sh = share;
  const int place = 2 * share_number(a), heads = a.Hkv / a.groups;
  int4 rec0 = make_int4(0, 0, 0, 0), rec1 = rec0;  // of an item begun before; begun here
  bool ok = true;
  if (sh.any) {
    int b = sh.b, h = sh.h, i = sh.i;
    int64_t at = sh.at;
    Seq q = seq_of(a.s, a.n, b);
#pragma unroll 1
    while (ok && at < sh.hi) {
      const int hk = h * a.groups + (int)(blockIdx.x % a.groups);
      const Work w(a, q);
      const int T = w.tiles_of(i), unit = w.unit_of(i);
      // tiles whose first unit lies in [lo, hi)
      auto tile_at = [&](int64_t u) -> int {
        const int64_t x = u - at - kOverhead;
        return x <= 0 ? 0 : (int)min((int64_t)T, unit == 2 ? (x + 1) >> 1 : x);
      };
      const int t0 = tile_at(sh.lo), t1 = tile_at(sh.hi);
      if (T == 0 && at >= sh.lo) {
        const int tokens = w.tokens_of(i);
#pragma unroll 1
        for (int t = 0; t < tokens; ++t) {
          const size_t head = (size_t)(q.row0 + i * w.per + t) * (a.Hkv * a.G) + hk * a.G;
          for (int e = lane; e < a.G * (D / 8); e += 32)
            reinterpret_cast<uint4*>(a.out + head * D)[e] = make_uint4(0, 0, 0, 0);
          for (int e = lane; a.lse && e < a.G; e += 32) a.lse[head + e] = -INFINITY;
        }
      }
      if (t0 < t1) {
        Seg s;
        s.b = b;
        s.hk = hk;
        s.row0 = q.row0 + i * w.per;
        s.tokens = w.tokens_of(i);
        s.p0 = w.start + i * w.per;
        s.end = max(s.p0 + s.tokens, 0);
        s.t0 = t0;
        s.t1 = t1;
        s.flags = (unit == 1 ? kSmall : 0) | (t0 == 0 ? kStarts : 0) | (t1 == T ? kEnds : 0);
        s.part = -1;
        if ((s.flags & (kStarts | kEnds)) != (kStarts | kEnds)) {
          const int4 r = make_int4(s.flags | kStop, s.row0, s.tokens, s.hk);
          s.part = place + (t0 == 0 ? 1 : 0);
          if (t0 == 0) rec1 = r;
          else rec0 = r;
        }
        ok = push(s);
      }
      at += w.weight_of(i);
      if (++i == w.count) {
        i = 0;
        if (++h == heads) {
          h = 0;
          do {
            if (++b >= a.s.B) break;
            q = seq_of(a.s, a.n, b);
          } while (q.m == 0);
          if (b >= a.s.B) break;
        }
      }
    }
  }
  if (lane == 0) {
    a.record[place] = rec0;
    a.record[place + 1] = rec1;
  }
  Seg s{};
  s.flags = kStop;
  if (ok) push(s);
}

// Pages of four tiles from t on, a lane a group of 16 keys; -1: none there.
__device__ __forceinline__ int pages_of(const AttendArgs& a, int lane, int b, int t, int end) {
  const uint32_t key = (uint32_t)t * 128 + lane * 16;  // (may pass 2^31)
  return key < (uint32_t)end ? ld_after(a.s.table + (size_t)b * a.s.columns + (key >> a.shift)) : -1;
}

// A segment's scales, four tiles at a time: put(k, group, ref, absent) for its tiles in order, of
// which the lanes from 8 k on have the groups (odd: their bits); put tells whether to go on. One warp.
template <class Put>
__device__ __forceinline__ bool segment_scales(const AttendArgs& a, const Seg& s, int lane, Put put) {
  const float c_scale = (a.scale == 0.0f ? 1.0f : fabsf(a.scale)) * att::kLog2e;
  float ref = 1.0f;
#pragma unroll 1
  for (int t = s.t0; t < s.t1; t += 4) {
    const int page = pages_of(a, lane, s.b, t, s.end);
    const bool in = page >= 0 && page < a.s.N, past = (uint32_t)t * 128 + lane * 16 >= (uint32_t)s.end;
    float2 sc = make_float2(0.0f, 0.0f);
    if (in) {
      const size_t at = (size_t)page * a.Hkv + s.hk;
      sc = make_float2(ld_after(a.k_scale + at), ld_after(a.v_scale + at));
    }
    if (page != -1 && !in && a.status) atomicOr(a.status, HYTOPK_DEV_BAD_INDEX);
    const bool k_ok = sc.x > 0.0f && sc.x <= att::kLargest;
    const bool v_ok = sc.y > 0.0f && sc.y <= att::kLargest;
    if (in && !(k_ok && v_ok) && a.status) atomicOr(a.status, HYTOPK_DEV_BAD_SCALE);
    if (t == s.t0) {  // the largest of a segment's first tile is the reference
      float top = lane < 8 && in && v_ok ? sc.y : 0.0f;
#pragma unroll
      for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      ref = fmaxf(top > 0.0f ? top : 1.0f, 1.17549435e-38f);
    }
    const float nan = __int_as_float(0x7fc00000);
    float2 group = make_float2(1.0f, 0.0f);  // (masked keys: any factor will do)
    if (in) {
      group.x = k_ok ? fmaxf(c_scale * sc.x, 1.17549435e-38f) : nan;
      const float ratio = sc.y * (1.0f / ref);  // (may pass the range of fp32)
      group.y = !v_ok ? nan
                : ratio > 1e-30f && ratio < 1e30f ? log2f(ratio) : log2f(sc.y) - log2f(ref);
    }
    const uint32_t absent = ~__ballot_sync(0xffffffffu, in || past);
    const uint32_t wide = __ballot_sync(0xffffffffu, fabsf(group.y) > kWide);
#pragma unroll 1
    for (int k = 0; k < 4 && t + k < s.t1; ++k)
      if (!put(k, group, ref, (absent >> (8 * k) & 0xFFu) | (wide >> (8 * k) & 0xFFu) << 8)) return false;
  }
  return true;
}

// Two sums with references of their own (-m' of the denominators l, d more of the weights; nm = -inf:
// nothing so far) as one: sum, nm, and what the results with the weights are multiplied with
// for softmax times v: f1, f2, or, where these could pass the range of fp32 somewhere in the warp
// (`odd`), f1, f2 and the powers of two p1, p2 on top.
struct Factors {
  float sum, nm, f1, f2, p1, p2;
  bool odd;
};
__device__ __forceinline__ Factors factors(float l, float nm, float d, float l2, float nm2, float d2,
                                           float ref) {
  Factors r;
  const bool one = nm > -INFINITY, two = nm2 > -INFINITY;
  const float both = fminf(one ? nm : INFINITY, two ? nm2 : INFINITY);
  r.nm = one || two ? both : -INFINITY;
  r.sum = l * (one ? ex2(both - nm) : 0.0f) + l2 * (two ? ex2(both - nm2) : 0.0f);
  // powers of two of the weights, beside ref
  const float a1 = one ? (both - nm) - d : -INFINITY, a2 = two ? (both - nm2) - d2 : -INFINITY;
  const float most = one || two ? fmaxf(a1, a2) : 0.0f;
  const int e = (int)(__float_as_uint(ref) >> 23) - 127;
  r.odd = __any_sync(0xffffffffu, fabsf(most) > kWide || abs(e) > (int)kWide);
  const float norm = (r.odd ? 1.0f : ref) / r.sum, shift = r.odd ? most : 0.0f;
  r.f1 = r.sum == 0.0f ? 0.0f : one ? ex2(a1 - shift) * norm : 0.0f * norm;
  r.f2 = r.sum == 0.0f ? 0.0f : two ? ex2(a2 - shift) * norm : 0.0f * norm;
  const float all = e + most, half = floorf(0.5f * all);
  r.p1 = ex2(half) * (ref * __uint_as_float((uint32_t)(127 - min(e, 126)) << 23)) * (e > 126 ? 0.5f : 1.0f);
  r.p2 = ex2(all - half);
  return r;
}

// ---- the kernel -------------------------------------------------------------------------

// Wait for a phase of `bar`; gives up (false, abort flag) when another role has, or after
// kTries tests of at most 2 us each. As few instructions as that takes: the code of all
// roles shares one instruction cache, and there are forty waits. (The status bit is set at
// the kernel's end.)
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, uint32_t abort_at) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b32 n, f;\n mov.b32 n, 0;\n"
      "W_:\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n @p bra D_;\n"
      " ld.volatile.shared.b32 f, [%4];\n add.u32 n, n, 1;\n setp.ne.b32 q, f, 0;\n"
      " setp.gt.or.u32 q, n, %5, q;\n @!q bra W_;\n st.volatile.shared.b32 [%4], 1;\n"
      "D_:\n selp.b32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(tc::smem_u32(bar)), "r"(parity), "r"(tc::kSuspendHintNs), "r"(abort_at), "n"(att::kTries)
      : "memory");
  return ok != 0;
}

// SECOND: launched behind the kernel of single rows, for calls that this one found not to be its
// own. An instance of its own, because the return at the top costs the others 1 to 2 %.
template <class C, bool SECOND>
__global__ void __launch_bounds__(kThreads, 1)
    k_attend_pages(const AttendArgs a, const __grid_constant__ CUtensorMap k_map,
                   const __grid_constant__ CUtensorMap v_map) {
  constexpr int D = C::D, NS = C::NS;
  using Geo = typename C::Geo;
  extern __shared__ __align__(1024) uint8_t smem_dyn[];
  uint8_t* smem = tc::align1024(smem_dyn);
  int* nan_s = reinterpret_cast<int*>(smem + C::NAN_OFF);  // [NANS][2][D] first key
  TileConst* const_s = reinterpret_cast<TileConst*>(smem + C::CONST_OFF);
  Seg* seg_s = reinterpret_cast<Seg*>(smem + C::SEG_OFF);
  float2* ml_s = reinterpret_cast<float2*>(smem + C::ML_OFF);  // [128] of the second warpgroup: l, nm
  float* d_s = reinterpret_cast<float*>(ml_s + 128);           // [128] its d
  float* qs_s = reinterpret_cast<float*>(smem + C::QS_OFF);  // [2][128]
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  uint64_t* full = bars;              // [NS] operands of a tile
  uint64_t* empty = full + NS;
  uint64_t* s_full = empty + NS;      // [2] scores of a warpgroup
  uint64_t* p_full = s_full + 2;      // [2] its weights
  uint64_t* pv_done = p_full + 2;     // [2] its products
  uint64_t* q_full = pv_done + 2;
  uint64_t* q_empty = q_full + 1;
  uint64_t* o_empty = q_empty + 1;
  uint64_t* ml_full = o_empty + 1;    // the second warpgroup's sums (small items)
  uint64_t* ml_empty = ml_full + 1;
  uint64_t* seg_full = ml_empty + 1;  // [kSegs]
  uint64_t* seg_empty = seg_full + kSegs;
  uint64_t* c_full = seg_empty + kSegs;       // [kConsts] scales of a tile
  uint64_t* c_empty = c_full + kConsts;       // [kConsts]
  uint64_t* unit_full = c_empty + kConsts;    // [SMALL_UNITS] codes
  uint64_t* unit_empty = unit_full + C::SMALL_UNITS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(unit_empty + C::SMALL_UNITS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  // [NANS][2]: some column of an item is NaN; softmax warps that are done with them
  uint32_t* nan_any = tmem_slot + 2;
  uint32_t* nan_done = nan_any + 2 * C::NANS;
  Share* share = reinterpret_cast<Share*>(ml_s);           // (before anything else is there)
  int64_t* scan_s = reinterpret_cast<int64_t*>(const_s);

  if (SECOND) {
    allow_next();
    wait_for_earlier();
    if (!ld_after(a.several)) return;
  }
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      tc::mbar_init(full + i, 4);
      tc::mbar_init(empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(s_full + i, 1);
      tc::mbar_init(p_full + i, 4);
      tc::mbar_init(pv_done + i, 1);
    }
    tc::mbar_init(q_full, 8);
    tc::mbar_init(q_empty, 1);
    tc::mbar_init(o_empty, 8);
    tc::mbar_init(ml_full, 4);
    tc::mbar_init(ml_empty, 4);
    for (int i = 0; i < kSegs; ++i) {
      tc::mbar_init(seg_full + i, 1);
      tc::mbar_init(seg_empty + i, 1 + 1 + 8 + 4);
    }
    for (int i = 0; i < kConsts; ++i) {
      tc::mbar_init(c_full + i, 1);
      tc::mbar_init(c_empty + i, 8);
    }
    for (int i = 0; i < C::SMALL_UNITS; ++i) {
      tc::mbar_init(unit_full + i, 1);
      tc::mbar_init(unit_empty + i, 4);
    }
    *abort_flag = 0;
    tc::fence_barrier_init();
  }
  for (int i = threadIdx.x; i < C::NANS * 2 * D; i += kThreads) nan_s[i] = INT32_MAX;
  if (threadIdx.x < C::NANS * 4) nan_any[threadIdx.x] = 0;  // (and nan_done)
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
  find_share<kThreads>(a, scan_s, share);
  __syncthreads();

  const uint32_t abort_at = tc::smem_u32(tmem_slot + 1);
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_phase(bar, parity, abort_at)) != 0;
  };
  // The number-th segment, taken out of the ring (each role, in order); false after a failed
  // wait.
  auto take = [&](int number, Seg& s) -> bool {
    if (!wait(seg_full + number % kSegs, (number / kSegs) & 1)) return false;
    s = seg_s[number % kSegs];
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(seg_empty + number % kSegs);
    return true;
  };
  auto unit_at = [&](int i) -> uint8_t* {
    return smem + (i < C::UNITS ? C::STAGE_OFF + i * C::UNIT
                                : C::Q_OFF + C::SLOT + (i - C::UNITS) * C::UNIT);
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsCtl));
    if (warp == 1) {
      // ---------------- segments ----------------
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
      // there lies past the pool's end, where rows of zeros are); eight copies for each tile,
      // issued by a lane each, took 2500 cycles of it.
      bool was_large = false;
      int unit = 0;
      uint32_t used = 0, phases = 0;  // bits of the units' places
      // tile t of a segment, whose pages eight lanes from `first` on have
      auto copy = [&](const CUtensorMap* map, const Seg& s, int t, int page, int first) -> bool {
        const uint32_t bit = 1u << unit;
        if (!wait(unit_empty + unit, (phases & bit) ? 0u : 1u)) return false;
        phases ^= bit;
        used |= bit;
        uint8_t* to = unit_at(unit);
        if (elect_one()) tc::mbar_expect_tx(unit_full + unit, C::UNIT);
        __syncwarp();
#pragma unroll 1
        for (int r = 0; r < 128; r += a.box) {
          const int pg = __shfl_sync(0xffffffffu, page, first + (r >> 4));
          const int row = (uint32_t)pg < (uint32_t)a.s.N ? (pg << a.shift) + ((t * 128 + r) & (a.s.P - 1))
                                                         : a.s.N << a.shift;
          if (elect_one()) tc::tma_load_2d(to + r * D, map, unit_full + unit, s.hk * D, row);
          __syncwarp();
        }
        unit = unit + 1 < (s.flags & kSmall ? C::SMALL_UNITS : C::UNITS) ? unit + 1 : 0;
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
        const bool small = s.flags & kSmall;
        if (C::SHARED && small == was_large) unit = 0;
        // (the last large item's queries lie in the place of a small one's codes)
        if (C::SHARED && small && was_large && !(ok = wait(q_empty, (segs - 1) & 1))) break;
        was_large = !small;
        int page = pages_of(a, lane, s.b, s.t0, s.end), next = -1;
#pragma unroll 1
        for (int t = s.t0; t < s.t1; ++t) {
          const int first = (t - s.t0) % 4 * 8;
          if (first == 0) {  // (the four after these, as early)
            if (t > s.t0) page = next;
            if (t + 4 < s.t1) next = pages_of(a, lane, s.b, t + 4, s.end);
          }
          if (!(ok = copy(&k_map, s, t, page, first) && copy(&v_map, s, t, page, first))) break;
        }
      }
      if (!ok || *abort_flag) {
        // given up: copies in flight land before the CTA ends (a bounded wait)
#pragma unroll 1
        for (int i = 0; i < C::SMALL_UNITS; ++i) {
          if (!(used >> i & 1)) continue;
          const uint32_t parity = phases >> i & 1 ? 0u : 1u;  // of the last copy there
          for (int n = 0; n < 100000; ++n)
            if (tc::mbar_try_wait(unit_full + i, parity)) break;
        }
      }
    } else if (warp == 3) {
      // ---------------- MMA issuer ----------------
      // The whole warp waits and keeps the state, all of it in uniform registers (numbers
      // of a segment come through a shuffle, so that the compiler knows): descriptors that
      // pass through vector registers cost 100 cycles a product. One elected lane issues.
      constexpr uint32_t D_HI = (1024u >> 4) | (1u << 14) | (2u << 29);  // 8-row groups, SW128
      constexpr uint32_t LBO_K = 1u << 16, LBO_MN = (16384u >> 4) << 16;
      constexpr uint32_t ID_S = f16_desc(128), ID_O = f16_desc(D) | (1u << 16);
      const uint32_t ring_lo = (tc::smem_u32(smem) >> 4) & 0x3FFFu;
      const uint32_t q_lo = (tc::smem_u32(smem + C::Q_OFF) >> 4) & 0x3FFFu;
      auto desc = [&](uint32_t lo) { return tc::desc_from_words(lo, D_HI); };
      // Slots of the next K and V, whose tiles are taken in the order of the ring.
      struct At {
        int slot;
        uint32_t phase;
      };
      At k{0, 0}, v{1, 0};
      auto step = [&](At& x) {
        x.slot += 2;
        if (x.slot >= NS) {
          x.slot -= NS;
          x.phase ^= 1u;
        }
      };
      auto landed = [&](const At& x) {
        const bool ok = wait(full + x.slot, x.phase);
        tc::fence_proxy_async_smem();  // of all that was stored into the ring
        return ok;
      };
      uint32_t p_phase = 0;  // bits: of the weights of each warpgroup
      uint32_t odd = 0;      // segments with tiles so far, modulo 2
      Seg s;
      bool ok = true;
#pragma unroll 1
      for (int number = 0; ok && take(number, s) && !(s.flags & kStop); ++number) {
        const int T = __shfl_sync(0xffffffffu, s.t1 - s.t0, 0);
        const bool small = __shfl_sync(0xffffffffu, s.flags & kSmall, 0) != 0;
        // Step i is warpgroup i % 2's: the products of its tile, then the scores of its next
        // one (which take the place of the weights). Of a large item both have every tile,
        // of a small one every other.
        const int N = small ? T : 2 * T;
        if (!(ok = wait(q_full, odd))) break;
#pragma unroll 1
        for (int i = -2; i < N; ++i) {
          const int w = i & 1;
          const bool first = small || w == 0, last = small || w == 1;  // with this K or V
          if (i >= 0) {
            if (!(ok = wait(p_full + w, p_phase >> w & 1u))) break;
            p_phase ^= 1u << w;
            if (i == 0 && !(ok = wait(o_empty, odd ^ 1u))) break;
            if (first && !(ok = landed(v))) break;
            tc::fence_after_sync();
            const uint32_t bd = (ring_lo + v.slot * (C::SLOT >> 4)) | LBO_MN;
            const uint32_t add = i >= 2 ? 1u : 0u;
            if (elect_one()) {
#pragma unroll
              for (int j = 0; j < 8; ++j)  // 16 keys
                mma_ts(tmem + C::O_COL + w * D, tmem + C::S_COL + w * 128 + j * 8,
                       desc(bd + (j * 2048 >> 4)), ID_O, j > 0 ? 1u : add);
              // (what the softmax waits for is committed last: nothing arrives after a CTA's end)
              if (last) tc::mma_commit(empty + v.slot);
              tc::mma_commit(pv_done + w);
            }
            __syncwarp();
            if (last) step(v);
          }
          if (i + 2 < N) {
            if (first && !(ok = landed(k))) break;
            tc::fence_after_sync();
            const uint32_t ad = (q_lo + (small ? 0 : w) * (C::SLOT >> 4)) | LBO_K;
            const uint32_t bd = (ring_lo + k.slot * (C::SLOT >> 4)) | LBO_K;
            if (elect_one()) {
#pragma unroll
              for (int j = 0; j < C::RB / 32; ++j)
                tc::mma<0>(tmem + C::S_COL + w * 128, desc(ad + (Geo::step_offset(j, 128) >> 4)),
                           desc(bd + (Geo::step_offset(j, 128) >> 4)), ID_S, j > 0 ? 1u : 0u);
              if (last) tc::mma_commit(empty + k.slot);
              if (i + 3 == N) tc::mma_commit(q_empty);
              tc::mma_commit(s_full + w);
            }
            __syncwarp();
            if (last) step(k);
          }
        }
        odd ^= 1u;
      }
    }
  } else if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsWide));
    // ---------------- codes to f16 ----------------
    // A warp takes 32 rows of a tile as they land, CPR lanes a row.
    constexpr int CPR = D / 16, RPP = 32 / CPR, PASSES = 32 / RPP;
    const int ww = warp - 12, c = lane % CPR, rl = lane / CPR;
    // Two 16-byte chunks of f16 for 16 codes. Lanes of the second 128-byte line of a row
    // write theirs in the other order: eight lanes at a time then meet eight banks.
    const int flip = (2 * c) >> 3 & 1;
    uint32_t place[2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
      place[e] = tc::smem_u32(smem) + Geo::chunk_offset(ww * 32 + rl, 2 * c + (e ^ flip), 128);
    int unit = 0, slot = 0;
    uint32_t phases = 0, phase = 1;
    bool large = false;
    // The next unit's codes into the next slot of the ring, whose row `key0` + ... some row of
    // the item may not see (`partly`). (The MMA issuer makes them visible to the tensor core.)
    auto spread = [&](bool partly, int key0, int end, int nans) -> bool {
      const uint32_t bit = 1u << unit;
      if (!wait(unit_full + unit, (phases & bit) ? 1u : 0u)) return false;
      phases ^= bit;
      const uint4* from = reinterpret_cast<const uint4*>(unit_at(unit) + ww * 32 * D) + lane;
      uint4 x[PASSES];
#pragma unroll
      for (int u = 0; u < PASSES; ++u) x[u] = from[u * 32];
      uint32_t found = 0;
      if (partly) {
#pragma unroll
        for (int u = 0; u < PASSES; ++u)
          found |= nan_codes(x[u].x) | nan_codes(x[u].y) | nan_codes(x[u].z) | nan_codes(x[u].w);
      }
      const bool odd = __any_sync(0xffffffffu, found != 0);  // (and all have read the unit)
      if (lane == 0) tc::mbar_arrive(unit_empty + unit);
      unit = unit + 1 < (large ? C::UNITS : C::SMALL_UNITS) ? unit + 1 : 0;
      if (!wait(empty + slot, phase)) return false;
      // (rows RPP apart: the swizzle repeats every 8 rows)
#pragma unroll
      for (int u = 0; u < PASSES; ++u) {
        const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // 8-row groups are 1024 bytes apart, and a half of one flips the chunk's third bit
          const uint32_t at = (RPP == 8 ? place[e] + u * 1024
                                        : (place[e] + (u / 2) * 1024 + (u % 2) * 512) ^
                                              ((u % 2) * 64u)) +
                              slot * C::SLOT;
          const int h = e ^ flip;
          const uint2 lo = widen(h ? w[2] : w[0]), hi = widen(h ? w[3] : w[1]);
          att::st_shared16(at, make_uint4(lo.x, lo.y, hi.x, hi.y));
        }
      }
      if (odd) {
        // NaN codes are replaced by 0 where they went, and their keys kept by column for the
        // rows that see them
        int* first = nan_s + nans * 2 * D + c * 16;
#pragma unroll 1
        for (int u = 0; u < PASSES * 16; ++u) {
          const int e = u % 16, r = ww * 32 + u / 16 * RPP + rl, key = key0 + u / 16 * RPP;
          uint16_t* h = reinterpret_cast<uint16_t*>(smem + slot * C::SLOT +
                                                    Geo::chunk_offset(r, 2 * c + e / 8, 128)) + e % 8;
          if ((*h & 0x7FFFu) <= 0x7C00u) continue;
          *h = 0;
          if (key >= end) continue;
          // a softmax warpgroup's own, which it clears once all products with the item are
          // done (of a small item the second one writes no result, and may not even wait for V)
          atomicMin(first + e, key);
          nan_any[nans * 2] = 1;
          if (!large) continue;
          atomicMin(first + D + e, key);
          nan_any[nans * 2 + 1] = 1;
        }
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(full + slot);
      if (++slot == NS) {
        slot = 0;
        phase ^= 1u;
      }
      return true;
    };
    Seg s;
    bool ok = true, first = true;
    int item = 0;  // of the NaN columns
#pragma unroll 1
    for (int number = 0; ok && take(number, s) && !(s.flags & kStop); ++number) {
      const bool now = !(s.flags & kSmall);
      if (C::SHARED && (first || now != large)) unit = 0;
      large = now;
      first = false;
#pragma unroll 1
      for (int u = 2 * s.t0; ok && u < 2 * s.t1; ++u) {  // K, V, K, V, ...
        const int key = (u >> 1) * 128;
        ok = spread((u & 1) && key + 127 > s.p0, key + ww * 32 + rl, s.end, item);
      }
      item = (item + 1) % C::NANS;
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
    // ---------------- softmax: TMEM lane = row ----------------
    // What bounds a tile is how fast instructions come: a tile as straight code took 2200
    // cycles here for 560 instructions, and slowed the other roles, a second copy of the
    // widening warps' loop alone 1.4 times. So all that runs per tile is a short loop.
    const int w = (warp >> 2) - 1, quad = warp & 3, row = quad * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t s_addr = tmem + lane_off + C::S_COL + w * 128;
    const uint32_t o_addr = tmem + lane_off + C::O_COL + w * D;
    const int my_token = row / a.G, my_head = row % a.G, Hq = a.Hkv * a.G;
    const float sign = a.scale < 0.0f ? -1.0f : a.scale == 0.0f ? 0.0f : 1.0f;
    // of a segment: this row's token
    auto token_of = [&](const Seg& s) {
      return my_token + (s.flags & kSmall ? 0 : w * a.tokens);
    };
    auto is_there = [&](const Seg& s) { return my_token < a.tokens && token_of(s) < s.tokens; };
    uint32_t loaded = 0;  // segments whose queries were taken
    // The queries of a segment into shared memory, and there to f16; `qs` is what was taken out
    // of this row's, a power of two, so that the largest is 2^14 to 2^15. They are copied in
    // whole lines, LPR lanes a row, all at once, and converted by the rows' threads. A small
    // item has one block of rows, the first warpgroup's, and the second is told `qs`.
    auto queries = [&](const Seg& s, float& qs) -> bool {
      constexpr int LPR = D / 8, RPI = 32 / LPR;  // lanes of a row, rows at a time
      const bool small = s.flags & kSmall;
      if (!wait(q_empty, (loaded & 1) ^ 1)) return false;
      float* told = qs_s + (loaded & 1) * 128 + row;
      if (!small || w == 0) {
        uint8_t* block = smem + C::Q_OFF + w * C::SLOT;
        const int c = lane % LPR;
        const int64_t at = (int64_t)(s.row0 + token_of(s)) * a.q_row + (int64_t)(s.hk * a.G + my_head) * D;
        const bool there = is_there(s);
#pragma unroll 4
        for (int i = 0; i < 32 / RPI; ++i) {
          const int r = i * RPI + lane / LPR;
          const int64_t from = __shfl_sync(0xffffffffu, at, r);
          const bool on = __shfl_sync(0xffffffffu, (int)there, r) != 0;
          att::cp_async16(tc::smem_u32(block) + Geo::chunk_offset(quad * 32 + r, c, 128),
                          a.q + (on ? from : 0) + c * 8, on);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        qs = 1.0f;
        if (__any_sync(0xffffffffu, there)) {  // (rows of zeros are the same in both types)
          uint32_t most2 = 0;  // two magnitudes' bits, each its own maximum
#pragma unroll 8
          for (int i = 0; i < LPR; ++i) {
            const uint4 x = *reinterpret_cast<const uint4*>(block + Geo::chunk_offset(row, i, 128));
            most2 = __vmaxu2(most2, __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu),
                                             __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu)));
          }
          const uint32_t most = max(most2 << 16, most2 & 0xFFFF0000u);
          const int ex = max((int)(most >> 23) - 127 - 14, -110);
          const float inv = sign * __int_as_float((127 - ex) << 23);
          qs = __int_as_float((ex + 127) << 23);
#pragma unroll 4
          for (int i = 0; i < LPR; ++i) {
            uint4* place = reinterpret_cast<uint4*>(block + Geo::chunk_offset(row, i, 128));
            const uint4 x = *place;
            const uint32_t y[4] = {x.x, x.y, x.z, x.w};
            uint32_t h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float lo = __uint_as_float(y[e] << 16), hi = __uint_as_float(y[e] & 0xFFFF0000u);
              att::mul2(lo, hi, inv, inv);
              h[e] = pack_f16(lo, hi);
            }
            *place = make_uint4(h[0], h[1], h[2], h[3]);
          }
        }
        if (small) *told = qs;
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(q_full);
      if (small && w == 1) {
        if (!wait(q_full, loaded & 1)) return false;
        qs = *reinterpret_cast<volatile float*>(told);
      }
      ++loaded;
      return true;
    };
    uint32_t cnt = 0;  // tiles of this warpgroup so far
    int tile0 = 0;     // tiles of the segments before
    int segs = 0, smalls = 0;
    uint32_t cnt0 = 0;   // the first warpgroup's
    bool dirty = false;  // codes of a small item may lie in the second block of queries
    Seg s{};             // (nothing yet: no token, no tile)
    float qs = 1.0f;
#pragma unroll 1
    for (int number = 0;; ++number) {
      const bool small = s.flags & kSmall;
      const int T = s.t1 - s.t0, step = small ? 2 : 1;
      const bool there = is_there(s);
      const int p = there ? s.p0 + token_of(s) : -1;  // the row's position
      const bool warp_there = __any_sync(0xffffffffu, there);
      const int p_first = s.p0 + (small ? 0 : w * a.tokens);  // the least position
      // nm: -m of the denominators, d: by how much -m of the weights is more (0 in the quick form)
      float nm = -INFINITY, d = 0.0f, l = 0.0f, ref = 1.0f;
      bool ok = true, slow = false;
      int mine = 0;  // tiles of this segment so far
#pragma unroll 1
      for (int t = s.t0 + (small ? w : 0); t < s.t1; t += step, ++mine, ++cnt) {
        // the tile's scales, before its scores are there
        const int number_c = tile0 + t - s.t0;
        const TileConst* tile = const_s + number_c % kConsts;
        if (!(ok = wait(c_full + number_c % kConsts, (number_c / kConsts) & 1))) break;
        ref = tile->ref;
        const uint32_t absent = tile->odd & 0xFFu;
        slow |= tile->odd > 0xFFu;
        if (!(ok = wait(s_full + w, cnt & 1))) break;
        tc::fence_after_sync();
        if (warp_there) {
          const int seen = p - t * 128;  // the tile's keys up to this one
          // (uniform in the warp) some key is not seen by some row, or not there
          const bool masked = t * 128 + 127 > p_first || absent != 0;
          auto upto = [&](int g) { return absent >> g & 1 ? -1 : seen - 16 * g; };
          // O and the tile's weights so far, those of `done` blocks, times 2^-by
          auto shrink = [&](float by, int done) -> bool {
            const float f = ex2(-by);
            // (f16 has no 2^-25, but weights that it leaves something of: in two steps)
            const float f_once = ex2(-fminf(by, 14.0f)), f_more = ex2(fminf(by, 14.0f) - by);
            const uint32_t f2 = pack_f16(f_once, f_once), f3 = pack_f16(f_more, f_more);
            tc::tmem_wait_st();
#pragma unroll 1
            for (int i = 0; i < 16 * done; i += 8) {
              uint32_t y[8];
              tmem_load8(s_addr + i, y);
#pragma unroll
              for (int e = 0; e < 8; ++e) y[e] = mul_f16(mul_f16(y[e], f2), f3);
              tmem_store8(s_addr + i, y);
            }
            if (mine > 0) {
              if (!wait(pv_done + w, (cnt - 1) & 1)) return false;
              tc::fence_after_sync();
#pragma unroll 1
              for (int i = 0; i < D; i += 8) {
                float o[8];
                att::tmem_load(o_addr + i, o);
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] *= f;
                att::tmem_store8(o_addr + i, o);
              }
            }
            tc::tmem_wait_st();
            return true;
          };
          // the largest of 16 scores as they are, masked
          auto largest = [&](int g, float (&v)[16]) -> float {
            tc::tmem_ld16(s_addr + 16 * g, v);
            tc::tmem_wait_ld(v);
            if (masked) {
              const int last = upto(g);
#pragma unroll
              for (int j = 0; j < 16; ++j) v[j] = j <= last ? v[j] : -INFINITY;
            }
            float m0 = max3(v[0], v[1], v[2]);
#pragma unroll
            for (int j = 3; j < 15; j += 2) m0 = max3(m0, v[j], v[j + 1]);
            return fmaxf(m0, v[15]);
          };
          if (!slow && __any_sync(0xffffffffu, there && !(fabsf(nm) <= kFar))) {
            // rows without a reference (the item's first tile): the maximum of the whole tile first
            float top = -INFINITY;
#pragma unroll 1
            for (int g = 0; g < 8; ++g) {
              float v[16];
              const float2 k = reinterpret_cast<const float2*>(tile->group)[g];
              top = fmaxf(top, __fadd_rn(__fmul_rn(largest(g, v), k.x * qs), k.y));
            }
            if (there && top > -INFINITY && nm == -INFINITY) nm = 4.0f - ceilf(fmaxf(top, -att::kLargest));
            slow = __any_sync(0xffffffffu, there && fabsf(nm) > kFar && nm > -INFINITY);
          }
          int from = 0;  // the group that the slow form begins with
          if (!slow) {
#pragma unroll 1
            for (int i = 0; i < 8; i += kBlock) {  // groups
              float v[kBlock / 2][32], c[kBlock], kb[kBlock];
#pragma unroll
              for (int h = 0; h < kBlock / 2; ++h) tc::tmem_ld32(s_addr + 16 * i + 32 * h, v[h]);
#pragma unroll
              for (int h = 0; h < kBlock / 2; ++h) {
                const float4 k = tile->group[i / 2 + h];
                c[2 * h] = k.x * qs;
                kb[2 * h] = k.y + nm;
                c[2 * h + 1] = k.z * qs;
                kb[2 * h + 1] = k.w + nm;
              }
#pragma unroll
              for (int h = 0; h < kBlock / 2; ++h) tc::tmem_wait_ld(v[h]);
              float most[kBlock];
#pragma unroll
              for (int g = 0; g < kBlock; ++g) {
                float* x = v[g / 2] + g % 2 * 16;
#pragma unroll
                for (int j = 0; j < 16; j += 2) fma2(x[j], x[j + 1], c[g], kb[g], kb[g]);
                if (masked) {
                  const int last = upto(i + g);
#pragma unroll
                  for (int j = 0; j < 16; ++j) x[j] = j <= last ? x[j] : -INFINITY;
                }
                float m0 = max3(x[0], x[1], x[2]), m1 = max3(x[3], x[4], x[5]);
                m0 = max3(m0, x[6], x[7]);
                m1 = max3(m1, x[8], x[9]);
                m0 = max3(m0, x[10], x[11]);
                m1 = max3(m1, x[12], x[13]);
                most[g] = fmaxf(max3(m0, x[14], x[15]), m1);
              }
              float top = most[0];
#pragma unroll
              for (int g = 1; g + 1 < kBlock; g += 2) top = max3(top, most[g], most[g + 1]);
              top = fmaxf(top, most[kBlock - 1]);
              // (what was added to a group's scores is taken out of its sum)
#pragma unroll
              for (int g = 0; g < kBlock; ++g) kb[g] = nm - kb[g];
              if (__any_sync(0xffffffffu, there && top > 11.0f)) {
                // m by `by` more (whole numbers); where that is so much that nothing so far counts,
                // from here on as if nothing had been, and slowly
                slow = __any_sync(0xffffffffu, there && top > kFar);
                const float by = !there || !(top > (slow ? kFar : 11.0f)) ? 0.0f
                                 : slow ? INFINITY : ceilf(top) - 4.0f;
                l *= ex2(-by);
                nm -= by;
                if (!(ok = shrink(by, i / 2))) break;
                if (slow) {
                  from = i;
                  break;
                }
#pragma unroll
                for (int j = 0; j < 16 * kBlock; ++j) v[j / 32][j % 32] -= by;
              }
#pragma unroll
              for (int h = 0; h < kBlock / 2; ++h) {
                uint32_t y[16];
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                  float* x = v[h] + 16 * g;
                  float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
                  for (int j = 0; j < 16; j += 2) {
                    x[j] = ex2(x[j]);
                    x[j + 1] = ex2(x[j + 1]);
                    add2(s0, s1, x[j], x[j + 1]);
                    y[8 * g + j / 2] = pack_f16(x[j], x[j + 1]);
                  }
                  // (a row without a score so far has nm = -inf and no weights)
                  const float sum = s0 + s1, share = sum * ex2(kb[2 * h + g]);
                  l += sum != 0.0f ? share : 0.0f;
                }
                tmem_store16(s_addr + 8 * i + 16 * h, y);
              }
            }
            if (!ok) break;
          }
          if (slow) {
            // The slow form, for all that is left of a segment: scores far from 0, where b would be
            // rounded away beside m, or b so far apart that no m would do for weights and
            // denominators both. x = s rounded as the maximum was; denominators sum 2^(x - m') with
            // m' of their own, weights are 2^(((x - m') + b) + d).
            const bool none = nm == -INFINITY;
            float by = 0.0f;
#pragma unroll 1
            for (int pass = 0; pass < 2; ++pass) {
              float top = -INFINITY;
#pragma unroll 1
              for (int g = from; g < 8; ++g) {
                float v[16];
                const float2 k = reinterpret_cast<const float2*>(tile->group)[g];
                const float x = __fmul_rn(largest(g, v), k.x * qs);
                top = fmaxf(top, pass ? __fadd_rn(__fadd_rn(x, nm), k.y) : x);
              }
              if (there && top > -INFINITY && (none || top + (pass ? d : nm) > (pass ? 11.0f : kWide))) {
                const float to = 4.0f - ceilf(fmaxf(top, -att::kLargest));
                if (pass) {
                  if (!none) by = d - to;
                  d = to;
                } else {
                  if (!none) {
                    l *= ex2(to - nm);
                    d += nm - to;
                  }
                  nm = to;
                }
              }
              __syncwarp();
            }
            if (__any_sync(0xffffffffu, by != 0.0f) && !(ok = shrink(by, from / 2))) break;
#pragma unroll 1
            for (int g = from; g < 8; ++g) {
              float v[16];
              tc::tmem_ld16(s_addr + 16 * g, v);
              tc::tmem_wait_ld(v);
              const float2 k = reinterpret_cast<const float2*>(tile->group)[g];
              const int last = masked ? upto(g) : 15;
              const float c = k.x * qs, nan = k.y - k.y;  // (NaN of a scale that is none, or 0)
              float sum = 0.0f;
              uint32_t y[8];
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const float x = __fadd_rn(__fmul_rn(v[j], c), nm), u = ex2(x) + nan;
                sum += j <= last ? u : 0.0f;
                v[j] = j <= last ? ex2(__fadd_rn(__fadd_rn(x, k.y), d)) : 0.0f;
                if (j & 1) y[j / 2] = pack_f16(v[j - 1], v[j]);
              }
              l += sum;
              tmem_store8(s_addr + 8 * g, y);
            }
          }
          tc::tmem_wait_st();
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(p_full + w);
        if (lane < (small ? 2 : 1)) tc::mbar_arrive(c_empty + number_c % kConsts);
      }
      if (!ok) break;
      if (T > 0) {
        cnt0 += small ? (T + 1) / 2 : T;
        dirty = C::SHARED && small;
      }
      // The next segment's queries, and this one's result: the queries first, so that the next
      // scores are made while the result goes out; but where the queries take the place of
      // codes, all products first.
      Seg next;
      float qs_next = 1.0f;
      const bool more = take(number, next) && !(next.flags & kStop);
      const bool late = more && dirty && !(next.flags & kSmall);
#pragma unroll 1
      for (int pass = 0; ok && pass < 2; ++pass) {
        if ((pass == 0) != late) {
          if (!more) continue;
          if (late) {
            // (own products are done; the first warpgroup's wait for these queries to go on)
            if (w == 1 && !(ok = wait(pv_done, (cnt0 - 1) & 1))) break;
            dirty = false;
          }
          ok = queries(next, qs_next);
          continue;
        }
        const int token = token_of(s), head = s.hk * a.G + my_head;
        const size_t q_at = (size_t)(s.row0 + token);
        if (T == 0) continue;  // (nothing yet)
        tile0 += T;
        // ---- the result ----
        if (mine > 0) {
          if (!(ok = wait(pv_done + w, (cnt - 1) & 1))) break;
          tc::fence_after_sync();
        }
        float l2 = 0.0f, nm2 = -INFINITY, d2 = 0.0f;  // the other warpgroup's
        const bool other = small && T > 1;
        if (small) {
          if (w == 1) {
            if (!(ok = wait(ml_empty, (smalls & 1) ^ 1))) break;
            ml_s[row] = make_float2(l, nm);
            d_s[row] = d;
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(ml_full);
          } else {
            if (!(ok = wait(ml_full, smalls & 1))) break;
            tc::fence_after_sync();
            const float2 x = ml_s[row];
            l2 = x.x;
            nm2 = x.y;
            d2 = d_s[row];
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(ml_empty);
          }
          ++smalls;
        }
        int* nans = nan_s + ((segs % C::NANS) * 2 + w) * D;
        uint32_t* any = nan_any + segs % C::NANS * 2 + w;
        const bool nan_here = *reinterpret_cast<volatile uint32_t*>(any) != 0;
        if (warp_there && !(small && w == 1)) {
          const Factors x = factors(l, nm, d, l2, nm2, d2, ref);
          const float f1 = x.f1, f2 = x.f2, sum = x.sum;
          const bool part = s.part >= 0;
          const int r = w * 128 + row;
          float* to_part = a.part + ((size_t)max(s.part, 0) * a.rows + r) * D;
          const uint64_t to_out = there ? (q_at * Hq + head) * D : 0;
          uint8_t* stage = smem + C::EPI_OFF + (warp - 4) * 1024;
#pragma unroll 1
          for (int i = 0; i < D; i += 32) {
            float o[32];
            tc::tmem_ld32(o_addr + i, o);
            tc::tmem_wait_ld(o);
#pragma unroll
            for (int e = 0; e < 32; e += 2) att::mul2(o[e], o[e + 1], f1, f1);
            if (other) {
              float z[32];
              tc::tmem_ld32(o_addr + D + i, z);
              tc::tmem_wait_ld(z);
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                fma2(z[e], z[e + 1], f2, o[e], o[e + 1]);
                o[e] = z[e];
                o[e + 1] = z[e + 1];
              }
            }
            if (x.odd) {
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = o[e] * x.p1 * x.p2;
            }
            if (part) {
              if (there) {
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                  *reinterpret_cast<float4*>(to_part + i + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                if (nan_here) {
#pragma unroll 1
                  for (int e = i; e < i + 32; ++e)
                    if (nans[e] <= p) to_part[e] = __int_as_float(0x7fc00000);
                }
              }
              __syncwarp();
              continue;
            }
            // 16 rows at a time through shared memory, so that four lanes write 64 bytes of a
            // row (a lane a row, every store met 32 lines: 8100 cycles an item of 256 rows)
            uint32_t y[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] = att::pack_bf16(o[2 * e], o[2 * e + 1]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              __syncwarp();
              if (lane >> 4 == h) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  *reinterpret_cast<uint4*>(stage + (lane & 15) * 64 + ((e ^ (lane >> 1 & 3)) << 4)) =
                      make_uint4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
                if (nan_here) {
#pragma unroll 1
                  for (int e = 0; e < 32; ++e)
                    if (nans[i + e] <= p)
                      *reinterpret_cast<uint16_t*>(stage + (lane & 15) * 64 +
                                                   (((e >> 3) ^ (lane >> 1 & 3)) << 4) + (e & 7) * 2) = 0x7FC0;
                }
              }
              __syncwarp();
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int rr = e * 8 + lane / 4, cc = lane & 3;
                const uint64_t to = __shfl_sync(0xffffffffu, to_out, h * 16 + rr);
                const bool on = __shfl_sync(0xffffffffu, (int)there, h * 16 + rr) != 0;
                const uint4 z = *reinterpret_cast<const uint4*>(stage + rr * 64 + ((cc ^ (rr >> 1 & 3)) << 4));
                if (on) *reinterpret_cast<uint4*>(a.out + to + i + cc * 8) = z;
              }
            }
          }
          if (there) {
            if (part) a.ml[(size_t)s.part * a.rows + r] = make_float2(sum, x.nm);
            else if (a.lse) a.lse[q_at * Hq + head] = sum == 0.0f ? -INFINITY : (log2f(sum) - x.nm) * att::kLn2;
          }
        }
        if (nan_here) {
          // the last of the warpgroup's warps clears them
          __syncwarp();
          uint32_t before = 0;
          if (lane == 0) before = atomicAdd(nan_done + segs % C::NANS * 2 + w, 1u);
          if (__shfl_sync(0xffffffffu, before, 0) == 3) {
            for (int i = lane; i < D; i += 32) nans[i] = INT32_MAX;
            if (lane == 0) {
              *any = 0;
              nan_done[segs % C::NANS * 2 + w] = 0;
            }
          }
        }
        // Eight arrivals: of a small item all are the first warpgroup's, which reads both
        // results (the second may have no tile and be an item ahead).
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0 && !(small && w == 1)) {
          tc::mbar_arrive(o_empty);
          if (small) tc::mbar_arrive(o_empty);
        }
        ++segs;
      }
      if (!ok || !more) break;
      s = next;
      qs = qs_next;
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

// ---- joining the parts ------------------------------------------------------------------

constexpr int kJoinThreads = 256;

// Parts of an item: number 2c + 1 of the share c where it starts, then 2c' + 0 of the shares after
// it, up to the one that ends it (shares between may hold none of it). Many parts or few rows: a block
// a row, its warps sharing the parts; else eight lanes a row, 32 rows a block. Every block finds out
// what there is to join, from all shares' records, and takes every gridDim.x-th of it. (A warp a
// row took 37 sequences of up to 256 rows 129 us instead of 116; blocks for the rows that each
// share might start, 4864 of them, one token 18.7 instead of 16.)
constexpr int kJoinBlocks = 8;  // for each share

template <int D>
__global__ void __launch_bounds__(kJoinThreads) k_join_parts(const AttendArgs a, int ctas) {
  allow_next();
  wait_for_earlier();
  constexpr int WARPS = kJoinThreads / 32, V = D / 32, WORDS = kJoinThreads / 32;
  static_assert(kMaxCtas <= kJoinThreads, "a thread a share");
  __shared__ uint32_t held_s[WORDS], ends_s[WORDS];  // shares that hold a part begun before; ends
  __shared__ int4 first_s[kMaxCtas];                 // what starts there and does not end
  __shared__ int before_s[kJoinThreads + 1];         // blocks' worth of rows in the shares before
  __shared__ int sums_s[WARPS];
  __shared__ float4 acc_s[WARPS][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int4 first0 = make_int4(0, 0, 0, 0);
  int flags0 = 0;
  if (tid < ctas) {
    first0 = ld_after(a.record + 2 * tid + 1);
    flags0 = ld_after(&a.record[2 * tid].x);
    first_s[tid] = first0;
  }
  const uint32_t some = __ballot_sync(0xffffffffu, (flags0 & kStop) != 0);
  const uint32_t end = __ballot_sync(0xffffffffu, (flags0 & kStop) && (flags0 & kEnds));
  if (lane == 0) {
    held_s[warp] = some;
    ends_s[warp] = end;
  }
  __syncthreads();
  auto last_of = [&](int c) -> int {  // the share after c that ends what starts there
    uint32_t word = ends_s[c / 32] & ~((2u << (c % 32)) - 1u);
    int w = c / 32;
    while (!word && ++w < WORDS) word = ends_s[w];
    return word ? w * 32 + __ffs(word) - 1 : ctas - 1;
  };
  // a row is a block's
  auto alone = [](int rows, int count) { return count > 8 || rows <= 16; };
  auto units_of = [&](const int4& f, int count) {  // of a block each
    const int rows = f.z * a.G;
    return !(f.x & kStop) ? 0 : alone(rows, count) ? rows : (rows + 4 * WARPS - 1) / (4 * WARPS);
  };
  {
    int sum = tid < ctas ? units_of(first0, last_of(tid) - tid) : 0;
    const int mine = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    if (lane == 31) sums_s[warp] = sum;
    __syncthreads();
    int base = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w)
      if (w < warp) base += sums_s[w];
    before_s[tid] = base + sum - mine;
    if (tid == kJoinThreads - 1) before_s[kJoinThreads] = base + sum;
    __syncthreads();
  }
  const int Hq = a.Hkv * a.G;
#pragma unroll 1
  for (int at = blockIdx.x; at < before_s[kJoinThreads]; at += gridDim.x) {
    int c = 0;  // the share that has it
#pragma unroll
    for (int step = kJoinThreads / 2; step; step >>= 1)
      if (before_s[c + step] <= at) c += step;
    const int u = at - before_s[c];
    const int4 first = first_s[c];
    const int count = last_of(c) - c;  // shares after c
    auto part_of = [&](int i) -> int {  // i-th share from c on; -1: no part
      if (i == 0) return 2 * c + 1;
      return held_s[(c + i) / 32] >> ((c + i) % 32) & 1 ? 2 * (c + i) : -1;
    };
    const int rows = first.z * a.G;
    const bool small = first.x & kSmall, wide = alone(rows, count);
    const int x = wide ? u : (u * WARPS + warp) * 4 + lane / 8;  // row of the item
    const int token = x / a.G, head = x % a.G;
    const int half = small || token < a.tokens ? 0 : 1;
    const size_t r = half * 128 + (token - half * a.tokens) * a.G + head;
    const size_t to = (size_t)(first.y + token) * Hq + first.w * a.G + head;
    float top = INFINITY, sum = 0.0f;  // top: the least -m; sum: the denominator there
    // (a part without rows counts nothing, but what is NaN in it does)
    auto count_in = [&](float s, float nm) {
      const float t = fminf(top, nm > -INFINITY ? nm : INFINITY);
      sum = (top < INFINITY ? sum * ex2(t - top) : sum) + (nm > -INFINITY ? s * ex2(t - nm) : s);
      top = t;
    };
    auto join_lanes = [&](int lanes) {
      for (int i = lanes / 2; i; i >>= 1) {
        const float s = __shfl_xor_sync(0xffffffffu, sum, i), t = __shfl_xor_sync(0xffffffffu, top, i);
        count_in(s, t < INFINITY ? t : -INFINITY);
      }
    };
    // What a part's result, which is softmax times v of its keys alone, counts, as two factors: little
    // of a large v may be more than all of a small one.
    auto weight_of = [&](float2 m) {
      if (!(m.x > 0.0f)) return make_float2(m.x, 1.0f);  // (0 or NaN)
      auto exponent = [](float x) { return (int)(__float_as_uint(x) >> 23); };
      auto fraction = [](float x) { return __uint_as_float((__float_as_uint(x) & 0x7FFFFFu) | 0x3F800000u); };
      const float all = top - m.y + (float)(exponent(m.x) - exponent(sum)), half = floorf(0.5f * all);
      return make_float2(fraction(m.x) / fraction(sum) * ex2(half), ex2(all - half));
    };
    auto log_sum = [&]() { return sum == 0.0f ? -INFINITY : (log2f(sum) - top) * att::kLn2; };
    if (!wide) {
      const bool on = x < rows;
      const size_t row = on ? r : 0;
      const int l = lane & 7;  // columns 4 l + 32 c
      float4 o[D / 32];
#pragma unroll
      for (int e = 0; e < D / 32; ++e) o[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int i = l; i <= count; i += 8) {
        const int part = part_of(i);
        if (part < 0) continue;
        const float2 m = ld_after(a.ml + part * (size_t)a.rows + row);
        count_in(m.x, m.y);
      }
      join_lanes(8);
#pragma unroll 2
      for (int i = 0; i <= count; ++i) {
        const int part = part_of(i);
        if (part < 0) continue;
        const float2 m = ld_after(a.ml + part * (size_t)a.rows + row);
        const float4* y = reinterpret_cast<const float4*>(a.part + (part * (size_t)a.rows + row) * D) + l;
        float4 z[D / 32];
#pragma unroll
        for (int e = 0; e < D / 32; ++e) z[e] = ld_after(y + 8 * e);
        const float2 f = weight_of(m);
        auto add = [&](float& to, float from) { to += from == 0.0f ? 0.0f : from * f.x * f.y; };
#pragma unroll
        for (int e = 0; e < D / 32; ++e) {
          add(o[e].x, z[e].x);
          add(o[e].y, z[e].y);
          add(o[e].z, z[e].z);
          add(o[e].w, z[e].w);
        }
      }
      if (!on) continue;
#pragma unroll
      for (int e = 0; e < D / 32; ++e)
        *reinterpret_cast<uint2*>(a.out + to * D + 32 * e + 4 * l) =
            make_uint2(att::pack_bf16(o[e].x, o[e].y), att::pack_bf16(o[e].z, o[e].w));
      if (a.lse && l == 0) a.lse[to] = log_sum();
      continue;
    }
    float o[V];
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = 0.0f;
    for (int i = lane; i <= count; i += 32) {
      const int part = part_of(i);
      if (part < 0) continue;
      const float2 m = ld_after(a.ml + part * (size_t)a.rows + r);
      count_in(m.x, m.y);
    }
    join_lanes(32);
#pragma unroll 8
    for (int i = warp; i <= count; i += WARPS) {
      const int part = part_of(i);
      if (part < 0) continue;
      const float2 m = ld_after(a.ml + part * (size_t)a.rows + r);
      const float* y = a.part + (part * (size_t)a.rows + r) * D + lane * V;
      float z[V];
      if constexpr (V == 4) {
        const float4 t = ld_after(reinterpret_cast<const float4*>(y));
        z[0] = t.x, z[1] = t.y, z[2] = t.z, z[3] = t.w;
      } else {
        const float2 t = ld_after(reinterpret_cast<const float2*>(y));
        z[0] = t.x, z[1] = t.y;
      }
      const float2 f = weight_of(m);
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] += z[e] == 0.0f ? 0.0f : z[e] * f.x * f.y;
    }
    __syncthreads();
    acc_s[warp][lane] = make_float4(o[0], o[1], V > 2 ? o[V - 2] : 0.0f, V > 2 ? o[V - 1] : 0.0f);
    __syncthreads();
    if (warp) continue;
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = 0.0f;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) {
      const float4 t = acc_s[i][lane];
      o[0] += t.x;
      o[1] += t.y;
      if constexpr (V > 2) {
        o[2] += t.z;
        o[3] += t.w;
      }
    }
    if constexpr (V == 4)
      *reinterpret_cast<uint2*>(a.out + to * D + lane * V) =
          make_uint2(att::pack_bf16(o[0], o[1]), att::pack_bf16(o[2], o[3]));
    else
      *reinterpret_cast<uint32_t*>(a.out + to * D + lane * V) = att::pack_bf16(o[0], o[1]);
    if (a.lse && lane == 0) a.lse[to] = log_sum();
  }
}

template <class C, bool SECOND>
cudaError_t launch_attend_pages(const AttendArgs& a, int ctas, cudaStream_t st) {
  auto kernel = k_attend_pages<C, SECOND>;
  // rows of one head of a pool [N P rows, Hkv d]
  CUtensorMap k_map, v_map;
  const uint64_t rows = (uint64_t)a.s.N * a.s.P;
  if (!make_tmap_2d(&k_map, a.k, 1, (uint64_t)a.Hkv * C::D, rows, C::D, a.box, 0) ||
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
