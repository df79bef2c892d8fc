// cache.cu -- rotary positions (hytopk_rope) and cache rows: quantised as they
// are written, with the rotation fused in (hytopk_cache_write), and read back
// (hytopk_cache_read). All three move each row once. Measured, of 6.8 TB/s for a plain
// copy: rotation of 8192 x 64 x 128 bf16 42.9 us (6.3 TB/s), of 30011 x 8 x 128 fp32
// 41.7 us (5.9); read of 262144 x 8 x 128 e4m3 as bf16 130 us (6.3), all bound by memory;
// write of 65521 x 8 x 128 bf16, rotated, as e4m3 58.3 us (3.5), bound by instructions, and
// of 200000 x 1 x 128, half rotated, 37 us (2.1), most of it the angles that no head
// shares. Of a few rows each takes its launch.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "launch.h"
#include "early.cuh"
#include "rope.cuh"

namespace hytopk {
namespace {

struct RowArgs {
  const void* x;
  int64_t x_row, x_head;
  void* out;
  int64_t out_row, out_head;
  float* scale;  // e4m3 output: [L, H]
  const int32_t* slots;
  const int32_t* positions;
  const float* inv_freq;
  int n, H, d, L;
  int rot, first, interleaved, inverse;
  float mscale;
  uint32_t* status;
};

__device__ __forceinline__ float load_elem(const float* p) { return *p; }
__device__ __forceinline__ float load_elem(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// ---- any d: one (row, head) per warp, its values in shared memory -----------------
// Kept for head widths other than 64, 128 and 256 (the kernels below need a
// power of two of 16-byte chunks in a row). Elements are taken one by one and angles anew
// for every head: rotation of 43690 x 8 x 192 bf16, 64 columns rotated, 121 us (2.2 TB/s).
constexpr int kWarps = 4;

template <typename T>
__device__ __forceinline__ void load_rotated(const RowArgs& a, int t, int h, float* row, int lane) {
  const T* x = static_cast<const T*>(a.x) + (size_t)t * a.x_row + (size_t)h * a.x_head;
  for (int j = lane; j < a.d; j += 32) row[j] = load_elem(x + j);
  __syncwarp();
  if (!a.positions) return;
  const int pos = a.positions[t];
  const bool bad = pos < 0 || pos >= kMaxPosition;
  if (bad && lane == 0 && a.status) atomicOr(a.status, HYTOPK_DEV_BAD_POSITION);
  for (int i = lane; i < a.rot / 2; i += 32) {
    const int j1 = a.first + (a.interleaved ? 2 * i : i);
    const int j2 = a.interleaved ? j1 + 1 : j1 + a.rot / 2;
    float c, s;
    rope_turn((float)pos, a.inv_freq[i], c, s);
    c *= a.mscale;
    s *= a.inverse ? -a.mscale : a.mscale;
    if (bad) c = s = __int_as_float(0x7fc00000);
    const float x1 = row[j1], x2 = row[j2];
    row[j1] = x1 * c - x2 * s;
    row[j2] = x1 * s + x2 * c;
  }
  __syncwarp();
}

// Rows of other widths than 64, 128 and 256: a warp a row, through shared memory.
template <typename T>
__global__ void __launch_bounds__(32 * kWarps) k_rope(const RowArgs a) {
  allow_next();
  wait_for_earlier();
  extern __shared__ float rows[];
  const int lane = threadIdx.x & 31;
  float* row = rows + (threadIdx.x >> 5) * a.d;
  const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (item >= (int64_t)a.n * a.H) return;
  const int t = (int)(item / a.H), h = (int)(item % a.H);
  load_rotated<T>(a, t, h, row, lane);
  T* y = static_cast<T*>(a.out) + (size_t)t * a.out_row + (size_t)h * a.out_head;
  for (int j = lane; j < a.d; j += 32) y[j] = (T)row[j];
}

template <typename T, bool E4M3>
__global__ void __launch_bounds__(32 * kWarps) k_cache_write(const RowArgs a) {
  allow_next();
  wait_for_earlier();
  extern __shared__ float rows[];
  const int lane = threadIdx.x & 31;
  float* row = rows + (threadIdx.x >> 5) * a.d;
  const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (item >= (int64_t)a.n * a.H) return;
  const int t = (int)(item / a.H), h = (int)(item % a.H);
  const int slot = a.slots ? a.slots[t] : t;
  if (slot < 0 || slot >= a.L) {
    if (slot != -1 && lane == 0 && a.status) atomicOr(a.status, HYTOPK_DEV_BAD_INDEX);
    return;
  }
  load_rotated<T>(a, t, h, row, lane);
  const size_t at = ((size_t)slot * a.H + h) * a.d;
  if constexpr (!E4M3) {
    for (int j = lane; j < a.d; j += 32)
      static_cast<__nv_bfloat16*>(a.out)[at + j] = __float2bfloat16_rn(row[j]);
  } else {
    float amax = 0.0f;
    bool bad = false;
    for (int j = lane; j < a.d; j += 32) {
      const float v = fabsf(row[j]);
      if (v <= 3.402823466e38f) amax = fmaxf(amax, v);
      else bad = true;
    }
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (bad && a.status) atomicOr(a.status, HYTOPK_DEV_NONFINITE);
    const float scale = amax > 0.0f ? fmaxf(__fdiv_rn(amax, 448.0f), 1.17549435e-38f) : 1.0f;
    for (int j = lane; j < a.d; j += 32) {
      const float v = __fdiv_rn(row[j], scale);
      uint8_t code = __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
      if (!(fabsf(row[j]) <= 3.402823466e38f)) code = 0x7F;
      static_cast<uint8_t*>(a.out)[at + j] = code;
    }
    if (lane == 0) a.scale[(size_t)slot * a.H + h] = scale;
  }
}

// ---- d = 64, 128, 256: a row in d / 8 lanes ---------------------------------------
// Lane j of a row's group holds columns 8j .. 8j + 7. Bound by memory: a row is
// read once and written once. What is computed per token, cos and sin of its
// rot / 2 angles, is shared by all the rows of a block through shared memory,
// and computed while the rows' loads are in flight; the other half of a pair of
// the half layout comes from its lane by shuffles.
constexpr int kFastThreads = 256;
constexpr int kIter = 4;  // rows per group: 4 x 16 bytes (bf16) in flight per thread

template <typename T>
__device__ __forceinline__ void load8(const T* p, uint32_t (&raw)[sizeof(T) * 2]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  raw[0] = a.x, raw[1] = a.y, raw[2] = a.z, raw[3] = a.w;
  if constexpr (sizeof(T) == 4) {
    const uint4 b = *(reinterpret_cast<const uint4*>(p) + 1);
    raw[4] = b.x, raw[5] = b.y, raw[6] = b.z, raw[7] = b.w;
  }
}
template <int W>
__device__ __forceinline__ void unpack8(const uint32_t (&raw)[W], float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < W; ++i) {
    if constexpr (W == 8) {
      v[i] = __uint_as_float(raw[i]);
    } else {
      v[2 * i] = __uint_as_float(raw[i] << 16);
      v[2 * i + 1] = __uint_as_float(raw[i] & 0xFFFF0000u);
    }
  }
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
  if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(p) = make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]),
                                              bf16x2(v[4], v[5]), bf16x2(v[6], v[7]));
  }
}
// two values as e4m3 codes, round to nearest even, saturating
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two quotients y / -scale from ninv = -1 / scale: q = y ninv, then q + (y + q scale) ninv.
__device__ __forceinline__ void quotient2(float y0, float y1, float scale, float ninv, float& c0,
                                          float& c1) {
  asm("{\n .reg .b64 y, s, n, q, e;\n mov.b64 y, {%2, %3};\n mov.b64 s, {%4, %4};\n"
      " mov.b64 n, {%5, %5};\n mul.rn.f32x2 q, y, n;\n fma.rn.f32x2 e, q, s, y;\n"
      " fma.rn.f32x2 q, e, n, q;\n mov.b64 {%0, %1}, q;\n}\n"
      : "=f"(c0), "=f"(c1)
      : "f"(y0), "f"(y1), "f"(scale), "f"(ninv));
}

__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Rows whose largest magnitude lies between these bits (1e-18 and 2^127) divide by a
// reciprocal.
constexpr uint32_t kTinyRow = 0x219392EFu, kHugeRow = 0x7F000000u;

// MODE 0: rotated rows; 1: into bf16 cache rows; 2: into e4m3 cache rows.
// V: neighbouring 8-column vectors a lane holds. Quantising is bound by its
// instructions (360 a lane of 16 elements: 163 rotation and angles, the rest loads,
// magnitudes, exact quotients (24) and codes); with V = 2 half the lanes share a row's
// scale, addresses and magnitude steps (8 heads x 65521 rows: 83 -> 68 us). A block takes
// kIter rows a group, so that the loads of several rows are in flight and their angles are
// computed once; four blocks an SM 68 -> 65.6 us (64 registers, and 76 bytes a thread that
// spill); quotients two at a time 62.5; coherent loads of slots and positions 57.9.
template <typename T, int D, int MODE, int V>
__global__ void __launch_bounds__(kFastThreads, 4) k_rows(const RowArgs a) {
  allow_next();
  wait_for_earlier();
  constexpr int GL = D / (8 * V), GROUPS = kFastThreads / GL, W = sizeof(T) * 2;
  extern __shared__ float4 table4[];
  float* table = reinterpret_cast<float*>(table4);  // [tokens][cos rot/2 | sin rot/2]
  const int j = threadIdx.x % GL, group = threadIdx.x / GL;
  // (n H < 2^31: row numbers are 32 bits, and a division is 20 instructions, not 100)
  const unsigned rows = (unsigned)a.n * a.H;
  const unsigned row0 = blockIdx.x * (unsigned)(GROUPS * kIter);
  // Rows are (t, h) in order; a group's are GROUPS apart.
  unsigned row = row0 + group;
  const int dt = GROUPS / a.H, dh = GROUPS - dt * a.H;
  int t = (int)(row / (unsigned)a.H), h = (int)row - t * a.H;
  const int t0 = (int)(row0 / (unsigned)a.H);
  // steps of the source pointer: to the group's next row, and back by H heads and on
  // by a token where the heads run over
  const int64_t x_step = dt * a.x_row + dh * a.x_head, x_wrap = a.x_row - a.H * a.x_head;
  const T* x = static_cast<const T*>(a.x) + t * a.x_row + h * a.x_head + j * (8 * V);
  uint32_t raw[kIter][V][W];
  int ts[kIter], hs[kIter], slot[kIter];
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    ts[i] = min(t, a.n - 1);
    hs[i] = h;
    slot[i] = -1;
    if (row < rows) {
      slot[i] = t;
      if (MODE != 0 && a.slots) slot[i] = ld_after(a.slots + t);
#pragma unroll
      for (int u = 0; u < V; ++u) load8(x + 8 * u, raw[i][u]);
    }
    row += GROUPS;
    t += dt;
    h += dh;
    x += x_step;
    if (h >= a.H) {
      h -= a.H;
      ++t;
      x += x_wrap;
    }
  }
  const int half = a.rot / 2;
  if (a.positions) {
    const unsigned last = min(row0 + GROUPS * kIter, rows) - 1;
    const int tokens = (int)(last / (unsigned)a.H) - t0 + 1;
    const float m_sin = a.inverse ? -a.mscale : a.mscale;
    // a warp a token, a lane a pair: a pair's frequency stays in its lane
    for (int i = threadIdx.x & 31; i < half; i += 32) {
      const float f = ld_after(a.inv_freq + i);
#pragma unroll 1
      for (int k = threadIdx.x >> 5; k < tokens; k += kFastThreads / 32) {
        const int pos = ld_after(a.positions + t0 + k);
        const bool bad = pos < 0 || pos >= kMaxPosition;
        if (bad && a.status) {
          // of a row that is not written a position does not matter (asked only here: 65521 x 8
          // rows 57.9 us, 61.3 with every token's slot looked at)
          const int to = MODE != 0 && a.slots ? ld_after(a.slots + t0 + k) : 0;
          if (to >= 0 && (MODE == 0 || to < a.L)) atomicOr(a.status, HYTOPK_DEV_BAD_POSITION);
        }
        float c, s;
        rope_turn((float)pos, f, c, s);
        if (bad) c = s = __int_as_float(0x7fc00000);
        table[k * a.rot + i] = c * a.mscale;
        table[k * a.rot + half + i] = s * m_sin;
      }
    }
    __syncthreads();
  }
  [[maybe_unused]] const uint32_t group_mask =  // the lanes of this row
      GL == 32 ? 0xffffffffu : ((1u << (GL & 31)) - 1u) << ((threadIdx.x & 31) / GL * GL);
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const unsigned r = row0 + group + i * GROUPS;
    if (__all_sync(0xffffffffu, r >= rows)) break;
    float v[V][8];
#pragma unroll
    for (int u = 0; u < V; ++u) {
      unpack8<W>(raw[i][u], v[u]);
      if (!a.positions) continue;
      const int col = (j * V + u) * 8 - a.first;  // within the rotated part if 0 <= col < rot
      const bool turned = col >= 0 && col < a.rot;
      const float* tab = table + (ts[i] - t0) * a.rot;  // (rows past the end: the last token's)
      if (a.interleaved) {
        if (turned) {
          const float4 c = *reinterpret_cast<const float4*>(tab + col / 2);
          const float4 s = *reinterpret_cast<const float4*>(tab + half + col / 2);
          const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x1 = v[u][2 * e], x2 = v[u][2 * e + 1];
            v[u][2 * e] = x1 * cs[e] - x2 * sn[e];
            v[u][2 * e + 1] = x1 * sn[e] + x2 * cs[e];
          }
        }
      } else {
        // the other half of the pairs: the same vector of the lane half / (8 V) on or
        // back (V = 2: half is a multiple of 16)
        const bool upper = col >= half;
        const int peer = (threadIdx.x & 31) + (upper ? -half / (8 * V) : half / (8 * V));
        uint32_t other[W];
#pragma unroll
        for (int e = 0; e < W; ++e) other[e] = __shfl_sync(0xffffffffu, raw[i][u][e], peer & 31);
        if (turned) {
          float o[8];
          unpack8<W>(other, o);
          const int at = upper ? col - half : col;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const float4 c = *reinterpret_cast<const float4*>(tab + at + 4 * q);
            const float4 s = *reinterpret_cast<const float4*>(tab + half + at + 4 * q);
            const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float x = v[u][4 * q + e], y = o[4 * q + e];
              v[u][4 * q + e] = upper ? y * sn[e] + x * cs[e] : x * cs[e] - y * sn[e];
            }
          }
        }
      }
    }
    if constexpr (MODE == 0) {
      if (r < rows) {
        T* y = static_cast<T*>(a.out) + (size_t)ts[i] * a.out_row + (size_t)hs[i] * a.out_head;
#pragma unroll
        for (int u = 0; u < V; ++u) store8(y + (j * V + u) * 8, v[u]);
      }
    } else {
      const bool in = r < rows && slot[i] >= 0 && slot[i] < a.L;
      if (r < rows && !in && slot[i] != -1 && j == 0 && a.status)
        atomicOr(a.status, HYTOPK_DEV_BAD_INDEX);
      const uint64_t at_row = (uint64_t)(uint32_t)max(slot[i], 0) * (uint32_t)a.H + hs[i];
      const uint64_t at = at_row * D + j * (8 * V);
      if constexpr (MODE == 1) {
        if (in) {
#pragma unroll
          for (int u = 0; u < V; ++u)
            store8(static_cast<__nv_bfloat16*>(a.out) + at + 8 * u, v[u]);
        }
      } else {
        // The row's largest magnitude, two values an instruction; a NaN stays one, so
        // that its bits, like infinity's, lie above every finite value's.
        float most = 0.0f;
#pragma unroll
        for (int e = 0; e < 8 * V; e += 2)
          most = max3_nan(most, fabsf(v[e / 8][e % 8]), fabsf(v[e / 8][e % 8 + 1]));
#pragma unroll
        for (int o = GL / 2; o; o >>= 1)
          most = max3_nan(most, most, __shfl_xor_sync(0xffffffffu, most, o));
        const uint32_t top = __float_as_uint(most);
        float scale;
        uint32_t codes[2 * V];
        if (!in) {
          // (a row past the end or skipped holds anything: no work for it)
        } else if (top - kTinyRow < kHugeRow - kTinyRow) {
          // Divisions by the rounded reciprocal: one product, its exact remainder, one
          // correction give the correctly rounded quotient (Markstein, "Computation of
          // elementary functions on the IBM RISC System/6000", 1990) while nothing
          // underflows. With the reciprocal negated the quotient comes out negated, a
          // negative zero keeps its sign, and one XOR flips four codes.
          const float amax = __uint_as_float(top);
          scale = amax * (1.0f / 448.0f);
          scale = __fmaf_rn(__fmaf_rn(-scale, 448.0f, amax), 1.0f / 448.0f, scale);
          const float ninv = -__frcp_rn(scale);
#pragma unroll
          for (int w = 0; w < 2 * V; ++w) {
            float c[4];
#pragma unroll
            for (int e = 0; e < 4; e += 2)
              quotient2(v[w / 2][w % 2 * 4 + e], v[w / 2][w % 2 * 4 + e + 1], scale, ninv, c[e],
                        c[e + 1]);
            codes[w] = (e4m3x2(c[0], c[1]) | (e4m3x2(c[2], c[3]) << 16)) ^ 0x80808080u;
          }
        } else {
          // a row of zeros, of values whose remainders could underflow, or with a
          // value that is not finite
          constexpr float kMost = 3.402823466e38f;
          float amax = 0.0f;
#pragma unroll
          for (int e = 0; e < 8 * V; ++e) {
            const float m = fabsf(v[e / 8][e % 8]);
            amax = fmaxf(amax, m <= kMost ? m : 0.0f);
          }
#pragma unroll
          for (int o = GL / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(group_mask, amax, o));
          scale = amax > 0.0f ? fmaxf(__fdiv_rn(amax, 448.0f), 1.17549435e-38f) : 1.0f;
#pragma unroll
          for (int w = 0; w < 2 * V; ++w) {
            float c[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float y = v[w / 2][w % 2 * 4 + e];
              c[e] = fabsf(y) <= kMost ? __fdiv_rn(y, scale) : __int_as_float(0x7fc00000);
            }
            codes[w] = e4m3x2(c[0], c[1]) | (e4m3x2(c[2], c[3]) << 16);
          }
          if (top >= 0x7F800000u && a.status) atomicOr(a.status, HYTOPK_DEV_NONFINITE);
        }
        if (in) {
          uint8_t* y = static_cast<uint8_t*>(a.out) + at;
          if constexpr (V == 2)
            *reinterpret_cast<uint4*>(y) = make_uint4(codes[0], codes[1], codes[2], codes[3]);
          else
            *reinterpret_cast<uint2*>(y) = make_uint2(codes[0], codes[1]);
          if (j == 0) a.scale[at_row] = scale;
        }
      }
    }
  }
}

template <typename T, int D, int MODE, int V>
void launch_rows_of(const RowArgs& a, cudaStream_t st) {
  const int per = kFastThreads / (D / (8 * V)) * kIter;  // rows of a block
  // a block of `per` rows touches at most this many tokens (64 KB of angles at most, for rows
  // of one head: three blocks an SM)
  const int tokens = a.H >= per ? 2 : (per + a.H - 2) / a.H + 1;
  const size_t smem = a.positions ? (size_t)tokens * a.rot * sizeof(float) : 0;
  const unsigned grid = (unsigned)(((int64_t)a.n * a.H + per - 1) / per);
  if (smem > 48 * 1024)
    cudaFuncSetAttribute(k_rows<T, D, MODE, V>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                         (int)smem);
  launch_early(k_rows<T, D, MODE, V>, grid, kFastThreads, smem, st, 1, a);
}

template <typename T, int MODE>
bool launch_rows(const RowArgs& a, cudaStream_t st) {
  // two vectors a lane: when quantising bf16, and pairs lie whole lanes apart
  constexpr bool kTwo = MODE == 2 && sizeof(T) == 2;
  if constexpr (kTwo) {
    if (!a.positions || a.interleaved || a.rot % 32 == 0) {
      if (a.d == 64) launch_rows_of<T, 64, MODE, 2>(a, st);
      else if (a.d == 128) launch_rows_of<T, 128, MODE, 2>(a, st);
      else if (a.d == 256) launch_rows_of<T, 256, MODE, 2>(a, st);
      else return false;
      return true;
    }
  }
  if (a.d == 64) launch_rows_of<T, 64, MODE, 1>(a, st);
  else if (a.d == 128) launch_rows_of<T, 128, MODE, 1>(a, st);
  else if (a.d == 256) launch_rows_of<T, 256, MODE, 1>(a, st);
  else return false;
  return true;
}

struct ReadArgs {
  const void* cache;
  const float* scale;
  const int32_t* slots;
  void* out;
  int n, H, d, L;
  uint32_t* status;
};

// A thread converts 16-byte chunks of the cache (16 codes or 8 bf16 values),
// kIter of them kFastThreads apart, all loaded before the first is stored. Bound
// by memory: every row is read once and written once (262144 x 8 x 128 e4m3 rows as
// bf16: 130 us, 6.3 TB/s of 6.8).
template <bool E4M3, typename T>
__global__ void __launch_bounds__(kFastThreads) k_cache_read(const ReadArgs a) {
  allow_next();
  wait_for_earlier();
  constexpr int CE = E4M3 ? 16 : 8;  // elements of a chunk
  const unsigned per_row = a.d / CE;
  const int shift = (per_row & (per_row - 1)) ? -1 : 31 - __clz(per_row);
  const int64_t total = (int64_t)a.n * a.H * per_row;
  const int64_t f0 = (int64_t)blockIdx.x * (kFastThreads * kIter) + threadIdx.x;
  uint4 raw[kIter];
  float scale[kIter];
  bool in[kIter];
  int slot[kIter];
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const int64_t f = f0 + i * kFastThreads;
    slot[i] = -1;
    in[i] = false;
    raw[i] = make_uint4(0, 0, 0, 0);
    scale[i] = 1.0f;
    if (f < total) {
      // rows of a power of two of chunks by a shift (the others: a 64-bit division)
      const unsigned item = shift >= 0 ? (unsigned)(f >> shift) : (unsigned)(f / per_row);
      const unsigned c = (unsigned)(f - (int64_t)item * per_row);
      const unsigned t = item / a.H, h = item - t * a.H;
      slot[i] = a.slots ? ld_after(a.slots + t) : (int)t;
      in[i] = slot[i] >= 0 && slot[i] < a.L;
      if (in[i]) {
        const size_t row = (size_t)slot[i] * a.H + h;
        raw[i] = ld_after(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.cache) +
                                                         row * a.d * (E4M3 ? 1 : 2)) + c);
        if (E4M3) scale[i] = ld_after(a.scale + row);
      } else if (slot[i] != -1 && a.status) {
        atomicOr(a.status, HYTOPK_DEV_BAD_INDEX);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const int64_t f = f0 + i * kFastThreads;
    if (f >= total) break;
    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
    T* y = static_cast<T*>(a.out) + f * CE;
    const float none = slot[i] == -1 ? 0.0f : __int_as_float(0x7fc00000);
#pragma unroll
    for (int p = 0; p < CE / 8; ++p) {
      float v[8];
      if constexpr (E4M3) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint16_t two = (uint16_t)(w[2 * p + e / 2] >> (16 * (e % 2)));
          uint32_t h2;
          asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(two));
          const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h2));
          v[2 * e] = x.x * scale[i];
          v[2 * e + 1] = x.y * scale[i];
        }
      } else {
        unpack8<4>(w, v);
      }
      if (!in[i]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = none;
      }
      store8(y + 8 * p, v);
    }
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
int elem_bytes(hytopk_elem e) { return e == HYTOPK_ELEM_F32 ? 4 : (e == HYTOPK_ELEM_BF16 ? 2 : 1); }
bool stride_ok(int64_t s, hytopk_elem e) { return (s * elem_bytes(e)) % 16 == 0; }

// Shape, type and alignment checks that hytopk_rope and hytopk_cache_write share.
hytopk_status check_rows(const void* x, int64_t x_row, int64_t x_head, hytopk_elem type, int n,
                         int H, int d, const hytopk_rope_params* r) {
  if (n < 0 || H < 1) return HYTOPK_INVALID_ARG;
  if (type != HYTOPK_ELEM_BF16 && type != HYTOPK_ELEM_F32) return HYTOPK_INVALID_ARG;
  if (d < 8 || d > 1024 || d % 8) return HYTOPK_UNSUPPORTED;
  if (r) {
    if (r->rot < 2 || r->first < 0 || (int64_t)r->first + r->rot > d) return HYTOPK_INVALID_ARG;
    if (r->rot % 16 || r->first % 8) return HYTOPK_UNSUPPORTED;
  }
  if ((int64_t)n * H >= (int64_t)1 << 31) return HYTOPK_UNSUPPORTED;
  if (n == 0) return HYTOPK_OK;
  if (!x || (r && (!r->positions || !r->inv_freq))) return HYTOPK_INVALID_ARG;
  if (!aligned16(x) || !stride_ok(x_row, type) || !stride_ok(x_head, type))
    return HYTOPK_MISALIGNED;
  if (r && (!aligned4(r->positions) || !aligned4(r->inv_freq))) return HYTOPK_MISALIGNED;
  return HYTOPK_OK;
}

RowArgs row_args(const void* x, int64_t x_row, int64_t x_head, int n, int H, int d,
                 const hytopk_rope_params* r, uint32_t* status) {
  RowArgs a{};
  a.x = x;
  a.x_row = x_row;
  a.x_head = x_head;
  a.n = n;
  a.H = H;
  a.d = d;
  a.status = status;
  if (r) {
    a.positions = r->positions;
    a.inv_freq = r->inv_freq;
    a.rot = r->rot;
    a.first = r->first;
    a.interleaved = r->interleaved;
    a.inverse = r->inverse;
    a.mscale = r->mscale;
  }
  return a;
}

hytopk_status launched() {
  return cudaGetLastError() == cudaSuccess ? HYTOPK_OK : HYTOPK_CUDA_ERROR;
}

}  // namespace
}  // namespace hytopk

using namespace hytopk;

extern "C" hytopk_status hytopk_rope(const void* x, int64_t x_row, int64_t x_head,
                                     hytopk_elem type, int n, int H, int d,
                                     const hytopk_rope_params* rope, void* out, int64_t out_row,
                                     int64_t out_head, uint32_t* dev_status, cudaStream_t stream) {
  if (!rope) return HYTOPK_INVALID_ARG;
  hytopk_status s = check_rows(x, x_row, x_head, type, n, H, d, rope);
  if (s != HYTOPK_OK || n == 0) return s;
  if (!out) return HYTOPK_INVALID_ARG;
  if (!aligned16(out) || !stride_ok(out_row, type) || !stride_ok(out_head, type))
    return HYTOPK_MISALIGNED;
  if (out == x && (out_row != x_row || out_head != x_head)) return HYTOPK_INVALID_ARG;
  RowArgs a = row_args(x, x_row, x_head, n, H, d, rope, dev_status);
  a.out = out;
  a.out_row = out_row;
  a.out_head = out_head;
  const unsigned grid = (unsigned)(((int64_t)n * H + kWarps - 1) / kWarps);
  const size_t smem = sizeof(float) * kWarps * d;
  const bool f32 = type == HYTOPK_ELEM_F32;
  if (f32 ? launch_rows<float, 0>(a, stream) : launch_rows<__nv_bfloat16, 0>(a, stream))
    return launched();
  if (type == HYTOPK_ELEM_F32) launch_early(k_rope<float>, grid, 32 * kWarps, smem, stream, 1, a);
  else launch_early(k_rope<__nv_bfloat16>, grid, 32 * kWarps, smem, stream, 1, a);
  return launched();
}

extern "C" hytopk_status hytopk_cache_write(const void* x, int64_t x_row, int64_t x_head,
                                            hytopk_elem x_type, int n, int H, int d,
                                            const hytopk_rope_params* rope, const int32_t* slots,
                                            void* cache, hytopk_elem cache_type,
                                            float* cache_scale, int L, uint32_t* dev_status,
                                            cudaStream_t stream) {
  hytopk_status s = check_rows(x, x_row, x_head, x_type, n, H, d, rope);
  if (s != HYTOPK_OK) return s;
  const bool e4 = cache_type == HYTOPK_ELEM_E4M3;
  if (!e4 && cache_type != HYTOPK_ELEM_BF16) return HYTOPK_INVALID_ARG;
  if (L < 1 || (!slots && n > L)) return HYTOPK_INVALID_ARG;
  if (e4 && d % 16) return HYTOPK_UNSUPPORTED;
  if (n == 0) return HYTOPK_OK;
  if (!cache || e4 != (cache_scale != nullptr)) return HYTOPK_INVALID_ARG;
  if (!aligned16(cache) || !aligned4(cache_scale) || !aligned4(slots)) return HYTOPK_MISALIGNED;
  RowArgs a = row_args(x, x_row, x_head, n, H, d, rope, dev_status);
  a.out = cache;
  a.scale = cache_scale;
  a.slots = slots;
  a.L = L;
  const unsigned grid = (unsigned)(((int64_t)n * H + kWarps - 1) / kWarps);
  const size_t smem = sizeof(float) * kWarps * d;
  const bool f32 = x_type == HYTOPK_ELEM_F32;
  if (f32 ? (e4 ? launch_rows<float, 2>(a, stream) : launch_rows<float, 1>(a, stream))
          : (e4 ? launch_rows<__nv_bfloat16, 2>(a, stream) : launch_rows<__nv_bfloat16, 1>(a, stream)))
    return launched();
  if (x_type == HYTOPK_ELEM_F32) {
    if (e4) launch_early(k_cache_write<float, true>, grid, 32 * kWarps, smem, stream, 1, a);
    else launch_early(k_cache_write<float, false>, grid, 32 * kWarps, smem, stream, 1, a);
  } else {
    if (e4) launch_early(k_cache_write<__nv_bfloat16, true>, grid, 32 * kWarps, smem, stream, 1, a);
    else launch_early(k_cache_write<__nv_bfloat16, false>, grid, 32 * kWarps, smem, stream, 1, a);
  }
  return launched();
}

extern "C" hytopk_status hytopk_cache_read(const void* cache, hytopk_elem cache_type,
                                           const float* cache_scale, int L, const int32_t* slots,
                                           int n, int H, int d, void* out, hytopk_elem out_type,
                                           uint32_t* dev_status, cudaStream_t stream) {
  const bool e4 = cache_type == HYTOPK_ELEM_E4M3;
  if (n < 0 || H < 1 || L < 1 || (!slots && n > L)) return HYTOPK_INVALID_ARG;
  if (!e4 && cache_type != HYTOPK_ELEM_BF16) return HYTOPK_INVALID_ARG;
  if (out_type != HYTOPK_ELEM_BF16 && out_type != HYTOPK_ELEM_F32) return HYTOPK_INVALID_ARG;
  if (d < 8 || d > 1024 || d % (e4 ? 16 : 8)) return HYTOPK_UNSUPPORTED;
  if ((int64_t)n * H >= (int64_t)1 << 31) return HYTOPK_UNSUPPORTED;
  if (n == 0) return HYTOPK_OK;
  if (!cache || !out || e4 != (cache_scale != nullptr)) return HYTOPK_INVALID_ARG;
  if (!aligned16(cache) || !aligned16(out) || !aligned4(cache_scale) || !aligned4(slots))
    return HYTOPK_MISALIGNED;
  const ReadArgs a{cache, cache_scale, slots, out, n, H, d, L, dev_status};
  const int64_t per = kFastThreads * kIter;
  const int64_t blocks = ((int64_t)n * H * (d / (e4 ? 16 : 8)) + per - 1) / per;
  const unsigned grid = (unsigned)blocks;  // n H < 2^31 and at most 64 or 128 chunks a row: < 2^31
  if (out_type == HYTOPK_ELEM_F32) {
    if (e4) launch_early(k_cache_read<true, float>, grid, kFastThreads, 0, stream, 1, a);
    else launch_early(k_cache_read<false, float>, grid, kFastThreads, 0, stream, 1, a);
  } else {
    if (e4) launch_early(k_cache_read<true, __nv_bfloat16>, grid, kFastThreads, 0, stream, 1, a);
    else launch_early(k_cache_read<false, __nv_bfloat16>, grid, kFastThreads, 0, stream, 1, a);
  }
  return launched();
}
