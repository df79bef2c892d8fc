// page_pool.cu -- the pool of a cache in pages: sequences forked, freed and grown, the pool
// compacted (hytopk_page_fork, _free, _grow, _compact), and pages copied (hytopk_page_copy).
//
// refs[p] counts the table entries that hold page p, so a fork copies only numbers, and a
// page is copied when a sequence grows into one that others hold. Everything is decided on
// the device in a fixed order (no result depends on which CTA comes first), so a step needs
// no host and can be captured into a graph.
#include "common.cuh"
#include "early.cuh"
#include "launch.h"
#include "pages.h"

namespace hytopk {
namespace pages {
namespace {

constexpr int kMostPages = 1 << 30;  // of a pool: page numbers a few thousand past its end are ints

struct Pool {
  int32_t* table;
  int32_t* lengths;
  int32_t* refs;
  int B, columns, N, P;
  uint32_t* status;
};

__device__ __forceinline__ void flag(uint32_t* status, uint32_t bit) {
  if (status) atomicOr(status, bit);
}
__device__ __forceinline__ int pages_of(int length, int P) { return (int)(((unsigned)length + P - 1) / P); }
// 0 <= length <= columns * P (columns * P < 2^31)
__device__ __forceinline__ bool fits(const Pool& a, int length) {
  return length >= 0 && length <= a.columns * a.P;
}

// Exclusive prefix sum of one value a thread; `total` is the block's.
template <int THREADS, typename T>
__device__ __forceinline__ T block_scan(T x, T* warps, T& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T s = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  __syncthreads();  // (of the scan before)
  if (lane == 31) warps[warp] = s;
  __syncthreads();
  if (warp == 0) {
    T w = lane < THREADS / 32 ? warps[lane] : T(0);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    if (lane < THREADS / 32) warps[lane] = w;
  }
  __syncthreads();
  total = warps[THREADS / 32 - 1];
  return s - x + (warp ? warps[warp - 1] : T(0));
}

// ---- fork and free: a CTA a sequence, a thread an entry of its row ----------------------

constexpr int kRowThreads = 128;

__global__ void __launch_bounds__(kRowThreads) k_fork(const Pool a, const int32_t* src,
                                                      const int32_t* dst, int count) {
  allow_next();
  wait_for_earlier();
  const int i = blockIdx.x, s = ld_after(src + i), d = ld_after(dst + i);
  if (s == -1 || d == -1) return;
  bool bad = s < 0 || s >= a.B || d < 0 || d >= a.B;
  for (int j = threadIdx.x; j < count; j += kRowThreads) {
    const int other = ld_after(dst + j);
    bad |= (j < i && other == d) || other == s;
  }
  // (only a CTA that passes these reads its sequences' state: nobody else changes it)
  bad = __syncthreads_or(bad);
  int length = 0;
  if (!bad) {
    length = ld_after(a.lengths + s);
    bad = !fits(a, length) || ld_after(a.lengths + d) != 0;
    length = bad ? 0 : length;
  }
  bool wrong = bad;
  const int held = pages_of(length, a.P);
  for (int j = threadIdx.x; j < held; j += kRowThreads) {
    int p = ld_after(a.table + (size_t)s * a.columns + j);
    if (p >= 0 && p < a.N) {
      atomicAdd(a.refs + p, 1);
    } else {
      wrong |= p != -1;
      p = -1;
    }
    a.table[(size_t)d * a.columns + j] = p;
  }
  __syncthreads();
  if (threadIdx.x == 0 && !bad) a.lengths[d] = length;
  if (wrong) flag(a.status, HYTOPK_DEV_BAD_INDEX);
}

__global__ void __launch_bounds__(kRowThreads) k_free(const Pool a, const int32_t* rows) {
  allow_next();
  wait_for_earlier();
  const int i = blockIdx.x, b = ld_after(rows + i);
  if (b == -1) return;
  if (b < 0 || b >= a.B) {
    if (threadIdx.x == 0) flag(a.status, HYTOPK_DEV_BAD_INDEX);
    return;
  }
  bool again = false;
  for (int j = threadIdx.x; j < i; j += kRowThreads) again |= ld_after(rows + j) == b;
  if (__syncthreads_or(again)) return;
  int length = ld_after(a.lengths + b);
  bool wrong = !fits(a, length);
  if (wrong) length = length < 0 ? 0 : a.columns * a.P;
  const int held = pages_of(length, a.P);
  for (int j = threadIdx.x; j < held; j += kRowThreads) {
    int32_t* entry = a.table + (size_t)b * a.columns + j;
    const int p = ld_after(entry);
    *entry = -1;
    if (p == -1) continue;
    if (p < 0 || p >= a.N) {
      wrong = true;
    } else if (atomicSub(a.refs + p, 1) <= 0) {
      atomicAdd(a.refs + p, 1);
      wrong = true;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) a.lengths[b] = 0;
  if (wrong) flag(a.status, HYTOPK_DEV_BAD_INDEX);
}

// ---- grow: one CTA ------------------------------------------------------------------

constexpr int kGrowThreads = 1024;

// fresh: [2 N] workspace, the free pages that are given out, ascending. Between the phases
// src_out holds a sequence's flags and need, dst_out its last page, then its first place in
// `fresh`.
__global__ void __launch_bounds__(kGrowThreads) k_grow(const Pool a, const int32_t* add,
                                                       int32_t* src_out, int32_t* dst_out,
                                                       int32_t* fresh) {
  allow_next();
  wait_for_earlier();
  __shared__ long long warps[kGrowThreads / 32];
  __shared__ int warps4[kGrowThreads / 32];
  const int tid = threadIdx.x;
  struct Row {
    int had, have, last;
    bool ok, open;
  };
  auto row_of = [&](int b) {
    const int length = ld_after(a.lengths + b), more = ld_after(add + b);
    Row r{0, 0, -1, fits(a, length) && more >= 0 && more <= a.columns * a.P - length, false};
    if (!r.ok) return r;
    r.had = pages_of(length, a.P);
    r.have = pages_of(length + more, a.P);
    if (more > 0 && length % a.P) {
      r.last = ld_after(a.table + (size_t)b * a.columns + r.had - 1);
      r.open = r.last >= 0 && r.last < a.N;
    }
    return r;
  };
  // the partly filled pages that sequences of this call grow into; of each, how many do (in
  // `fresh`, for now) and the last of them (every sequence looking at all others took 10 us of
  // 512)
  int32_t* most = fresh + a.N;
  for (int b = tid; b < a.B; b += kGrowThreads) {
    const Row r = row_of(b);
    dst_out[b] = r.open ? r.last : -1;
    if (r.open) {
      fresh[r.last] = 0;
      most[r.last] = -1;
    }
  }
  __syncthreads();
  for (int b = tid; b < a.B; b += kGrowThreads) {
    const int p = dst_out[b];
    if (p < 0) continue;
    atomicAdd(fresh + p, 1);
    atomicMax(most + p, b);
  }
  __syncthreads();
  // who needs another page for it: all holders but the last, if all of them grow, else all
  for (int b = tid; b < a.B; b += kGrowThreads) {
    const int p = dst_out[b];
    int away = 0;
    if (p >= 0) {
      const int holders = ld_after(a.refs + p);
      away = holders > 1 && (__ldcg(most + p) > b || __ldcg(fresh + p) != holders);
    }
    src_out[b] = away;
  }
  __syncthreads();
  // needs and places
  long long base = 0;
  for (int b0 = 0; b0 < a.B; b0 += kGrowThreads) {
    const int b = b0 + tid;
    Row r{0, 0, -1, false, false};
    if (b < a.B) r = row_of(b);
    const int away = b < a.B ? src_out[b] : 0, need = r.ok ? r.have - r.had + away : 0;
    long long total;
    const long long at = base + block_scan<kGrowThreads>((long long)need, warps, total);
    if (b < a.B) {
      src_out[b] = r.ok ? need * 2 + away : -1;
      dst_out[b] = (int)(at <= a.N ? at : (long long)a.N + 1);  // (N + 1: past every free page)
    }
    base += total;
  }
  const int wanted = (int)(base < a.N ? base : (long long)a.N);
  // the lowest-numbered free pages, four of a thread at a time
  int found = 0;
  const bool vec = (reinterpret_cast<uintptr_t>(a.refs) & 15) == 0;
  for (int p0 = 0; p0 < a.N && found < wanted; p0 += 4 * kGrowThreads) {
    const int p = p0 + 4 * tid;
    int4 v = make_int4(1, 1, 1, 1);
    if (vec && p + 3 < a.N) {
      v = ld_after(reinterpret_cast<const int4*>(a.refs + p));
    } else {
      if (p < a.N) v.x = ld_after(a.refs + p);
      if (p + 1 < a.N) v.y = ld_after(a.refs + p + 1);
      if (p + 2 < a.N) v.z = ld_after(a.refs + p + 2);
      if (p + 3 < a.N) v.w = ld_after(a.refs + p + 3);
    }
    const bool f[4] = {v.x == 0, v.y == 0, v.z == 0, v.w == 0};
    int total;
    int at = found + block_scan<kGrowThreads>((int)f[0] + f[1] + f[2] + f[3], warps4, total);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (f[i]) {
        if (at < wanted) fresh[at] = p + i;
        ++at;
      }
    found += total;
  }
  __syncthreads();
  // a warp a sequence
  for (int b = tid >> 5; b < a.B; b += kGrowThreads / 32) {
    const int lane = tid & 31, state = src_out[b], at = dst_out[b];
    const Row r = row_of(b);
    const int away = state & 1, need = state >> 1;
    const bool granted = state >= 0 && (long long)at + need <= found;
    const int grown = granted ? ld_after(a.lengths + b) + ld_after(add + b) : 0;
    __syncwarp();  // (all lanes have read the sequence's state)
    if (granted) {
      for (int j = lane; j < need; j += 32) {
        const int p = fresh[at + j];
        a.table[(size_t)b * a.columns + r.had - away + j] = p;
        a.refs[p] = 1;
        if (away && j == 0) {
          src_out[b] = r.last;
          dst_out[b] = p;
          atomicSub(a.refs + r.last, 1);
        }
      }
      if (lane == 0) a.lengths[b] = grown;
    } else if (lane == 0) {
      flag(a.status, state >= 0 || fits(a, ld_after(a.lengths + b)) && ld_after(add + b) >= 0
                         ? HYTOPK_DEV_NO_PAGE
                         : HYTOPK_DEV_BAD_INDEX);
    }
    if (lane == 0 && !(granted && away)) src_out[b] = dst_out[b] = -1;
  }
}

// ---- compact ------------------------------------------------------------------------
// Three launches: pages in use by chunks; every chunk's movers and holes with their ranks
// (of a hole p below K: p minus the pages in use below it); refs and the table. A small pool
// and table are one CTA's, in one launch.

constexpr int kChunkThreads = 256, kPer = 16, kChunk = kChunkThreads * kPer;

struct Compact {
  int32_t* src;
  int32_t* dst;
  int32_t* rank;   // [N] of a mover, -1 of any other page from K on
  int32_t* count;  // [chunks] pages in use, [chunks] K
};

__device__ __forceinline__ int live_of(const Pool& a, int p0, uint32_t& mask) {
  mask = 0;
  if (p0 + kPer <= a.N && !(reinterpret_cast<uintptr_t>(a.refs) & 15)) {
#pragma unroll
    for (int i = 0; i < kPer; i += 4) {
      const int4 v = ld_after(reinterpret_cast<const int4*>(a.refs + p0 + i));
      mask |= ((v.x > 0) | (v.y > 0) << 1 | (v.z > 0) << 2 | (v.w > 0) << 3) << i;
    }
    return __popc(mask);
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (p0 + i < a.N && ld_after(a.refs + p0 + i) > 0) mask |= 1u << i;
  return __popc(mask);
}
// of them, those below K
__device__ __forceinline__ int live_below(int p0, uint32_t mask, int K) {
  const int cut = K - p0;
  return __popc(cut <= 0 ? 0u : cut >= kPer ? mask : mask & ((1u << cut) - 1u));
}
// Movers and holes of a thread's pages; `seen` are in use before them, `low` below K.
__device__ __forceinline__ void rank_pages(const Pool& a, const Compact& c, int p0, uint32_t mask, int K,
                                           int seen, int low) {
#pragma unroll 1
  for (int i = 0; i < kPer && p0 + i < a.N; ++i) {
    const int p = p0 + i;
    const bool live = mask >> i & 1;
    if (p >= K) {
      c.rank[p] = live ? seen - low : -1;
      if (live) c.src[seen - low] = p;
    } else if (!live) {
      c.dst[p - seen] = p;
    }
    seen += live;
  }
}
// refs and the table, every step-th from i0 on
__device__ __forceinline__ void move_pages(const Pool& a, const Compact& c, int K, int64_t i0,
                                           int64_t step) {
  for (int64_t r = i0; r < a.N / 2; r += step) {
    const int s = ld_after(c.src + r);
    if (s < 0) break;
    const int d = ld_after(c.dst + r);
    a.refs[d] = ld_after(a.refs + s);
    a.refs[s] = 0;
  }
  const int64_t entries = (int64_t)a.B * a.columns;
  bool wrong = false;
  for (int64_t e = i0; e < entries; e += step) {
    const int b = (int)(e / a.columns), j = (int)(e - (int64_t)b * a.columns);
    const int p = ld_after(a.table + e), length = ld_after(a.lengths + b);
    const int most = a.columns * a.P;
    wrong |= length < 0 || length > most;
    if (p == -1 || j >= pages_of(min(max(length, 0), most), a.P)) continue;
    if (p < 0 || p >= a.N) {
      wrong = true;
    } else if (p >= K) {
      const int r = ld_after(c.rank + p);
      if (r >= 0) a.table[e] = ld_after(c.dst + r);
      else wrong = true;  // an entry whose page counts as free
    }
  }
  if (wrong) flag(a.status, HYTOPK_DEV_BAD_INDEX);
}

// One launch instead of three: 6.3 us of the host instead of 12.3, and of the GPU 4.3 instead of
// 7.9 for 512 pages and 224 entries of the table, but 9.0 instead of 7.2 for 1000 and 16384, 12.2
// instead of 9.9 for 8192 of both: taken up to 4096 of both.
constexpr int kOneThreads = 1024, kOnePages = 4096, kOneEntries = 4096;
static_assert(kOnePages <= kOneThreads * kPer, "a thread's pages");

__global__ void __launch_bounds__(kOneThreads) k_compact_one(const Pool a, const Compact c) {
  allow_next();
  wait_for_earlier();
  __shared__ int warps[kOneThreads / 32];
  const int tid = threadIdx.x, p0 = tid * kPer, moves = a.N / 2 > 0 ? a.N / 2 : 1;
  for (int r = tid; r < moves; r += kOneThreads) c.src[r] = c.dst[r] = -1;
  uint32_t mask;
  int K, low;
  const int seen = block_scan<kOneThreads>(live_of(a, p0, mask), warps, K);
  block_scan<kOneThreads>(live_below(p0, mask, K), warps, low);
  rank_pages(a, c, p0, mask, K, seen, low);
  __syncthreads();
  move_pages(a, c, K, tid, kOneThreads);
}

__global__ void __launch_bounds__(kChunkThreads) k_compact_count(const Pool a, const Compact c) {
  allow_next();
  wait_for_earlier();
  __shared__ int warps[kChunkThreads / 32];
  uint32_t mask;
  int total;
  block_scan<kChunkThreads>(live_of(a, blockIdx.x * kChunk + threadIdx.x * kPer, mask), warps, total);
  if (threadIdx.x == 0) c.count[blockIdx.x] = total;
  const int moves = a.N / 2 > 0 ? a.N / 2 : 1;
  for (int r = blockIdx.x * kChunkThreads + threadIdx.x; r < moves; r += gridDim.x * kChunkThreads)
    c.src[r] = c.dst[r] = -1;
}

__global__ void __launch_bounds__(kChunkThreads) k_compact_rank(const Pool a, const Compact c) {
  allow_next();
  wait_for_earlier();
  __shared__ int warps[kChunkThreads / 32];
  const int chunks = gridDim.x, tid = threadIdx.x;
  int all = 0, before = 0;
  for (int i = tid; i < chunks; i += kChunkThreads) {
    const int n = ld_after(c.count + i);
    all += n;
    if (i < (int)blockIdx.x) before += n;
  }
  int K, base, low;
  block_scan<kChunkThreads>(all, warps, K);
  block_scan<kChunkThreads>(before, warps, base);
  // pages in use below K: whole chunks, and K's own up to it
  const int at_k = K / kChunk;
  int below = 0;
  for (int i = tid; i < chunks && i < at_k; i += kChunkThreads) below += ld_after(c.count + i);
  uint32_t mask;
  const int q0 = at_k * kChunk + tid * kPer;
  live_of(a, q0, mask);
  below += live_below(q0, mask, K);
  block_scan<kChunkThreads>(below, warps, low);
  const int p0 = blockIdx.x * kChunk + tid * kPer;
  const int mine = live_of(a, p0, mask);
  int total;
  rank_pages(a, c, p0, mask, K, base + block_scan<kChunkThreads>(mine, warps, total), low);
  if (blockIdx.x == 0 && tid == 0) c.count[chunks] = K;
}

__global__ void __launch_bounds__(kChunkThreads) k_compact_move(const Pool a, const Compact c,
                                                                int chunks) {
  allow_next();
  wait_for_earlier();
  move_pages(a, c, ld_after(c.count + chunks), (int64_t)blockIdx.x * kChunkThreads + threadIdx.x,
             (int64_t)gridDim.x * kChunkThreads);
}

// ---- copies -------------------------------------------------------------------------
// A CTA takes 16 KB of a page at a time, so that 4 loads of 16 bytes a thread are in
// flight; it looks at 32 list entries at once, because most of a compaction's are -1.

constexpr int kCopyThreads = 256, kCopyLoads = 4;
constexpr int64_t kPiece = kCopyThreads * kCopyLoads * 16;

struct Copy {
  uint8_t* pages[2];
  float* scale[2];
  int N, H, count;
  int64_t bytes;
  int pieces, pools;
  const int32_t* src;
  const int32_t* dst;
  uint32_t* status;
};

__global__ void __launch_bounds__(kCopyThreads) k_copy(const Copy a) {
  allow_next();
  wait_for_earlier();
  const int lane = threadIdx.x & 31;
  // blocks (piece, pool) of an entry are neighbours
  const unsigned per = (unsigned)a.pieces * a.pools, part = blockIdx.x % per;
  const int pool = (int)(part / a.pieces), piece = (int)(part % a.pieces);
  const int step = (int)(gridDim.x / per);
  const int64_t at = piece * kPiece + (int64_t)threadIdx.x * 16;
#pragma unroll 1
  for (int64_t i0 = blockIdx.x / per; i0 < a.count; i0 += 32 * (int64_t)step) {
    const int64_t mine = i0 + (int64_t)lane * step;
    int s = -1, d = -1;
    if (mine < a.count) {
      s = ld_after(a.src + mine);
      d = ld_after(a.dst + mine);
    }
    bool some = s != -1 && d != -1;
    if (some && (s < 0 || s >= a.N || d < 0 || d >= a.N)) {
      if (threadIdx.x < 32 && part == 0) flag(a.status, HYTOPK_DEV_BAD_INDEX);
      some = false;
    }
    uint32_t todo = __ballot_sync(0xffffffffu, some && s != d);
    while (todo) {
      const int l = __ffs(todo) - 1;
      todo &= todo - 1;
      const int from = __shfl_sync(0xffffffffu, s, l), to = __shfl_sync(0xffffffffu, d, l);
      const uint8_t* x = a.pages[pool] + from * a.bytes;
      uint8_t* y = a.pages[pool] + to * a.bytes;
      uint4 v[kCopyLoads];
#pragma unroll
      for (int u = 0; u < kCopyLoads; ++u) {
        const int64_t o = at + u * (kCopyThreads * 16);
        if (o < a.bytes) v[u] = ld_after(reinterpret_cast<const uint4*>(x + o));
      }
#pragma unroll
      for (int u = 0; u < kCopyLoads; ++u) {
        const int64_t o = at + u * (kCopyThreads * 16);
        if (o < a.bytes) *reinterpret_cast<uint4*>(y + o) = v[u];
      }
      if (piece == 0)
        for (int h = threadIdx.x; h < a.H; h += kCopyThreads)
          a.scale[pool][(size_t)to * a.H + h] = ld_after(a.scale[pool] + (size_t)from * a.H + h);
    }
  }
}

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

hytopk_status check_pool(const void* table, const void* lengths, const void* refs, int B,
                         int columns, int N, int P) {
  if (B < 0 || columns < 1 || N < 1) return HYTOPK_INVALID_ARG;
  if (!page_rows_ok(P) || (int64_t)columns * P >= (int64_t)1 << 31 || N > kMostPages)
    return HYTOPK_UNSUPPORTED;
  if (!refs || (B > 0 && (!table || !lengths))) return HYTOPK_INVALID_ARG;
  if (!aligned(table, 4) || !aligned(lengths, 4) || !aligned(refs, 4)) return HYTOPK_MISALIGNED;
  return HYTOPK_OK;
}

hytopk_status of(cudaError_t e) { return e == cudaSuccess ? HYTOPK_OK : HYTOPK_CUDA_ERROR; }

int chunks_of(int N) { return (int)(((int64_t)N + kChunk - 1) / kChunk); }

}  // namespace
}  // namespace pages
}  // namespace hytopk

using namespace hytopk;
using namespace hytopk::pages;

extern "C" hytopk_status hytopk_page_fork(int32_t* table, int32_t* lengths, int32_t* refs, int B,
                                          int columns, int N, int P, const int32_t* src,
                                          const int32_t* dst, int count, uint32_t* dev_status,
                                          cudaStream_t stream) {
  const hytopk_status s = check_pool(table, lengths, refs, B, columns, N, P);
  if (s != HYTOPK_OK) return s;
  if (count < 0) return HYTOPK_INVALID_ARG;
  if (count == 0) return HYTOPK_OK;
  if (!src || !dst) return HYTOPK_INVALID_ARG;
  if (!aligned(src, 4) || !aligned(dst, 4)) return HYTOPK_MISALIGNED;
  const Pool a{table, lengths, refs, B, columns, N, P, dev_status};
  return of(launch_early(k_fork, (unsigned)count, kRowThreads, 0, stream, 1, a, src, dst, count));
}

extern "C" hytopk_status hytopk_page_free(int32_t* table, int32_t* lengths, int32_t* refs, int B,
                                          int columns, int N, int P, const int32_t* rows,
                                          int count, uint32_t* dev_status, cudaStream_t stream) {
  const hytopk_status s = check_pool(table, lengths, refs, B, columns, N, P);
  if (s != HYTOPK_OK) return s;
  if (count < 0) return HYTOPK_INVALID_ARG;
  if (count == 0) return HYTOPK_OK;
  if (!rows) return HYTOPK_INVALID_ARG;
  if (!aligned(rows, 4)) return HYTOPK_MISALIGNED;
  const Pool a{table, lengths, refs, B, columns, N, P, dev_status};
  return of(launch_early(k_free, (unsigned)count, kRowThreads, 0, stream, 1, a, rows));
}

extern "C" size_t hytopk_page_workspace_size(int N) {
  if (N < 1 || N > kMostPages) return 0;
  return (2 * (size_t)N + chunks_of(N) + 1) * sizeof(int32_t) / 256 * 256 + 256;
}

extern "C" hytopk_status hytopk_page_grow(int32_t* table, int32_t* lengths, int32_t* refs, int B,
                                          int columns, int N, int P, const int32_t* add,
                                          int32_t* src_out, int32_t* dst_out, void* workspace,
                                          size_t workspace_bytes, uint32_t* dev_status,
                                          cudaStream_t stream) {
  const hytopk_status s = check_pool(table, lengths, refs, B, columns, N, P);
  if (s != HYTOPK_OK) return s;
  if (B == 0) return HYTOPK_OK;
  if (!add || !src_out || !dst_out || !workspace) return HYTOPK_INVALID_ARG;
  if (workspace_bytes < hytopk_page_workspace_size(N)) return HYTOPK_WORKSPACE_TOO_SMALL;
  if (!aligned(add, 4) || !aligned(src_out, 4) || !aligned(dst_out, 4) || !aligned(workspace, 256))
    return HYTOPK_MISALIGNED;
  const Pool a{table, lengths, refs, B, columns, N, P, dev_status};
  return of(launch_early(k_grow, 1, kGrowThreads, 0, stream, 1, a, add, src_out, dst_out,
                         static_cast<int32_t*>(workspace)));
}

extern "C" hytopk_status hytopk_page_compact(int32_t* table, const int32_t* lengths, int32_t* refs,
                                             int B, int columns, int N, int P, int32_t* src_out,
                                             int32_t* dst_out, void* workspace,
                                             size_t workspace_bytes, uint32_t* dev_status,
                                             cudaStream_t stream) {
  const hytopk_status s = check_pool(table, lengths, refs, B, columns, N, P);
  if (s != HYTOPK_OK) return s;
  if (!src_out || !dst_out || !workspace) return HYTOPK_INVALID_ARG;
  if (workspace_bytes < hytopk_page_workspace_size(N)) return HYTOPK_WORKSPACE_TOO_SMALL;
  if (!aligned(src_out, 4) || !aligned(dst_out, 4) || !aligned(workspace, 256))
    return HYTOPK_MISALIGNED;
  const Pool a{table, const_cast<int32_t*>(lengths), refs, B, columns, N, P, dev_status};
  const int chunks = chunks_of(N);
  int32_t* ws = static_cast<int32_t*>(workspace);
  const Compact c{src_out, dst_out, ws, ws + N};
  if (N <= kOnePages && (int64_t)B * columns <= kOneEntries)
    return of(launch_early(k_compact_one, 1, kOneThreads, 0, stream, 1, a, c));
  cudaError_t e = launch_early(k_compact_count, (unsigned)chunks, kChunkThreads, 0, stream, 1, a, c);
  if (e == cudaSuccess)
    e = launch_early(k_compact_rank, (unsigned)chunks, kChunkThreads, 0, stream, 1, a, c);
  if (e == cudaSuccess) {
    const int64_t most = (int64_t)B * columns > N / 2 ? (int64_t)B * columns : N / 2;
    const int64_t blocks = (most + kChunkThreads - 1) / kChunkThreads, cap = 4 * (int64_t)num_sms();
    e = launch_early(k_compact_move, (unsigned)(blocks < 1 ? 1 : blocks < cap ? blocks : cap),
                     kChunkThreads, 0, stream, 1, a, c, chunks);
  }
  return of(e);
}

extern "C" hytopk_status hytopk_page_copy(void* k_pages, float* k_scale, void* v_pages,
                                          float* v_scale, int N, int64_t page_bytes, int H,
                                          const int32_t* src, const int32_t* dst, int count,
                                          uint32_t* dev_status, cudaStream_t stream) {
  if (N < 1 || H < 1 || page_bytes < 1 || count < 0) return HYTOPK_INVALID_ARG;
  if (page_bytes % 16 || page_bytes > (int64_t)1 << 31) return HYTOPK_UNSUPPORTED;
  if (count == 0) return HYTOPK_OK;
  if (!k_pages || !k_scale || (v_pages != nullptr) != (v_scale != nullptr) || !src || !dst)
    return HYTOPK_INVALID_ARG;
  if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(k_scale, 4) ||
      !aligned(v_scale, 4) || !aligned(src, 4) || !aligned(dst, 4))
    return HYTOPK_MISALIGNED;
  Copy a{};
  a.pages[0] = static_cast<uint8_t*>(k_pages);
  a.pages[1] = static_cast<uint8_t*>(v_pages);
  a.scale[0] = k_scale;
  a.scale[1] = v_scale;
  a.N = N;
  a.H = H;
  a.count = count;
  a.bytes = page_bytes;
  a.pieces = (int)((page_bytes + kPiece - 1) / kPiece);
  a.pools = v_pages ? 2 : 1;
  a.src = src;
  a.dst = dst;
  a.status = dev_status;
  // whole entries to a row of blocks, as many as keep every SM busy
  const int64_t per = (int64_t)a.pieces * a.pools;
  int64_t rows = (int64_t)num_sms() * 8 / per;
  rows = rows < 1 ? 1 : rows > count ? count : rows;
  return of(launch_early(k_copy, (unsigned)(rows * per), kCopyThreads, 0, stream, 1, a));
}
