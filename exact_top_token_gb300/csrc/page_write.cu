// page_write.cu -- rows, rotated, into the pages at the end of each context, as e4m3 codes with
// one scale per (page, head) (hytopk_page_write).
//
// A page's scale is the largest magnitude of all its new rows over 448, and of the earlier
// rows' scale; so a CTA takes a page and some of its heads: it finds the page, turns the
// rows' positions into cos and sin once (shared by the heads), and for each head loads the
// rows, rotates them, reduces their magnitudes over the block and writes codes. What it
// read stays in registers between the two. Where the scale of a page that holds earlier
// rows grows, their codes are rewritten: code * (old / new).
//
// What bounds it: instructions. 37000 rows of 8 heads of 128 bf16, all rotated, take 43 us, 17 of
// which the bytes need (114 MB): the angles are 10 of them, shared by eight heads (shared by
// four 56 us in all, by two 77); bf16 rows are held to 80 registers for three blocks an SM (two
// 45.6; up to 72 bytes spill). One row for each of 64 sequences, 8 heads, takes 6.9 us, a
// chain of sequence, page, rows and scale, magnitudes and earlier codes; 37 pieces of 500 fp32
// rows of 3 heads of 64 in pages of 16 rows 14.6, since a page is one CTA's, head after head.
#include "early.cuh"
#include "launch.h"
#include "pages.h"
#include "rope.cuh"
#include "rows.cuh"

namespace hytopk {
namespace pages {
namespace {

constexpr int kThreads = 256;
constexpr int kVec = 4;  // 8-column vectors of a head that a thread holds
constexpr float kMost = 3.402823466e38f;
constexpr uint32_t kInf = 0x7F800000u;

struct WriteArgs {
  const void* x;
  int64_t x_row, x_head;
  int n, H, heads;  // heads of a CTA
  const int32_t* positions;
  const float* inv_freq;  // NULL: no rotation
  int rot, first, interleaved, inverse;
  float mscale;
  uint8_t* pages;
  float* scale;
  hytopk_paged s;
  uint32_t* status;
};

__device__ __forceinline__ void flag(uint32_t* status, uint32_t bit) {
  if (status) atomicOr(status, bit);
}

// A page of a call: sequence's rows row0 .. of x go to rows lo .. hi - 1 of column `column` of
// sequence b's table row; `pos` is the first one's position.
struct Unit {
  int b, column, row0, lo, hi, pos;
};

// The unit-th page that the call's rows go to, in order; false past the last.
__device__ bool find_unit(const WriteArgs& a, int unit, Unit& u) {
  __shared__ int warps[kThreads / 32];
  __shared__ Unit found;
  const int P = a.s.P, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int base = 0;
  for (int b0 = 0; b0 < a.s.B; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    int pages = 0, start = 0;
    Seq q{};
    if (b < a.s.B) {
      q = seq_of(a.s, a.n, b);
      start = max(q.length - q.m, 0);
      if (q.m > 0 && q.length > start) pages = (q.length - 1) / P - start / P + 1;
      if (q.bad && blockIdx.x == 0) flag(a.status, HYTOPK_DEV_BAD_POSITION);
    }
    int sum = pages;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    if (lane == 31) warps[warp] = sum;
    __syncthreads();
    int before = base, total = base;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += warps[w];
      total += warps[w];
    }
    const int at = before + sum - pages;
    if (unit >= at && unit < at + pages) {
      const int column = start / P + (unit - at), first = max(start, column * P);
      found = Unit{b, column, q.row0 + q.m - (q.length - first), first - column * P,
                   min(q.length - column * P, P), first};
    }
    __syncthreads();
    if (unit < total) {
      u = found;
      // (all sequences are reported on, those of no unit here too)
      if (blockIdx.x == 0)
        for (int i = b0 + kThreads + threadIdx.x; i < a.s.B; i += kThreads)
          if (seq_of(a.s, a.n, i).bad) flag(a.status, HYTOPK_DEV_BAD_POSITION);
      return true;
    }
    base = total;
  }
  return false;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 3 : 2) k_page_write(const WriteArgs a) {
  allow_next();
  wait_for_earlier();
  constexpr int GL = D / 8, GROUPS = kThreads / GL, CHUNK = GROUPS * kVec, W = sizeof(T) * 2;
  extern __shared__ float4 table4[];
  float* table = reinterpret_cast<float*>(table4);  // [CHUNK rows][cos rot/2 | sin rot/2]
  __shared__ uint32_t tops[2][kThreads / 32];
  const int blocks = (a.H + a.heads - 1) / a.heads;
  Unit u;
  if (!find_unit(a, (int)(blockIdx.x / blocks), u)) return;
  const int h0 = (int)(blockIdx.x % blocks) * a.heads, h1 = min(h0 + a.heads, a.H);
  const int page = ld_after(a.s.table + (size_t)u.b * a.s.columns + u.column);
  if (page < 0 || page >= a.s.N) {
    if (page != -1 && threadIdx.x == 0) flag(a.status, HYTOPK_DEV_BAD_INDEX);
    return;
  }
  const int j = threadIdx.x % GL, group = threadIdx.x / GL, lane = threadIdx.x & 31;
  const int rows = u.hi - u.lo, half = a.rot / 2;
  const bool one = rows <= CHUNK;  // (uniform) the rows stay in registers
  const T* x0 = static_cast<const T*>(a.x) + (size_t)u.row0 * a.x_row + j * 8;
  const int64_t x_step = GROUPS * a.x_row, y_step = (int64_t)GROUPS * a.H * D;
  uint8_t* y0 = a.pages + ((size_t)page * a.s.P + u.lo) * a.H * D + j * 8;

  // cos and sin of the rows from r0 on
  auto angles = [&](int r0) {
    __syncthreads();
    const float m_sin = a.inverse ? -a.mscale : a.mscale;
    const int count = min(rows - r0, CHUNK);
    for (int i = lane; i < half; i += 32) {
      const float f = ld_after(a.inv_freq + i);
#pragma unroll 1
      for (int k = threadIdx.x >> 5; k < count; k += kThreads / 32) {
        const int pos = a.positions ? ld_after(a.positions + u.row0 + r0 + k) : u.pos + r0 + k;
        const bool bad = pos < 0 || pos >= kMaxPosition;
        if (bad) flag(a.status, HYTOPK_DEV_BAD_POSITION);
        float c, s;
        rope_turn((float)pos, f, c, s);
        if (bad) c = s = __int_as_float(0x7fc00000);
        table[k * a.rot + i] = c * a.mscale;
        table[k * a.rot + half + i] = s * m_sin;
      }
    }
    __syncthreads();
  };
  auto load = [&](int h, int r0, uint32_t (&raw)[kVec][W]) {
    const T* x = x0 + (int64_t)(r0 + group) * a.x_row + (int64_t)h * a.x_head;
    const int left = rows - r0 - group;
#pragma unroll
    for (int i = 0; i < kVec; ++i, x += x_step) {
#pragma unroll
      for (int e = 0; e < W; ++e) raw[i][e] = 0;
      if (i * GROUPS < left) load8(x, raw[i]);
    }
  };
  // vector i of a chunk as loaded, rotated (whole warps)
  auto rotated = [&](int i, int r0, const uint32_t (&raw)[W], float (&v)[8]) {
    unpack8<W>(raw, v);
    if (!a.inv_freq) return;
    const int col = j * 8 - a.first;
    const bool turned = col >= 0 && col < a.rot;
    const float* tab = table + min(group + i * GROUPS, rows - r0 - 1) * a.rot;
    if (a.interleaved) {
      if (!turned) return;
      const float4 c = *reinterpret_cast<const float4*>(tab + col / 2);
      const float4 s = *reinterpret_cast<const float4*>(tab + half + col / 2);
      const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x1 = v[2 * e], x2 = v[2 * e + 1];
        v[2 * e] = x1 * cs[e] - x2 * sn[e];
        v[2 * e + 1] = x1 * sn[e] + x2 * cs[e];
      }
      return;
    }
    // the other half of the pairs: the same vector, half / 8 lanes on or back
    const bool upper = col >= half;
    const int peer = (threadIdx.x & 31) + (upper ? -half / 8 : half / 8);
    uint32_t other[W];
#pragma unroll
    for (int e = 0; e < W; ++e) other[e] = __shfl_sync(0xffffffffu, raw[e], peer & 31);
    if (!turned) return;
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
        const float y = v[4 * q + e], z = o[4 * q + e];
        v[4 * q + e] = upper ? z * sn[e] + y * cs[e] : y * cs[e] - z * sn[e];
      }
    }
  };
  int turn = 0;  // reductions so far: two places in turn, so that one barrier does
  auto block_max = [&](uint32_t bits) {
    bits = __reduce_max_sync(0xffffffffu, bits);
    uint32_t* place = tops[turn & 1];
    ++turn;
    if (lane == 0) place[threadIdx.x >> 5] = bits;
    __syncthreads();
    uint32_t top = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) top = max(top, place[w]);
    return top;
  };
  // the largest magnitude's bits; with `finite`, of finite elements alone
  auto largest = [&](const float (&v)[8], bool finite) {
    float most = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      float p = fabsf(v[e]), q = fabsf(v[e + 1]);
      if (finite) {
        p = p <= kMost ? p : 0.0f;
        q = q <= kMost ? q : 0.0f;
      }
      most = max3_nan(most, p, q);
    }
    return __float_as_uint(most) & 0x7FFFFFFFu;
  };
  auto store = [&](uint8_t* y, const float (&v)[8], float scale, float ninv, bool fast) {
    uint32_t codes[2];
    if (fast) {
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        float c[4];
        quotient2(v[4 * w], v[4 * w + 1], scale, ninv, c[0], c[1]);
        quotient2(v[4 * w + 2], v[4 * w + 3], scale, ninv, c[2], c[3]);
        codes[w] = (e4m3x2(c[0], c[1]) | (e4m3x2(c[2], c[3]) << 16)) ^ 0x80808080u;
      }
    } else {
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        float c[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float y = v[4 * w + e];
          c[e] = fabsf(y) <= kMost ? __fdiv_rn(y, scale) : __int_as_float(0x7fc00000);
        }
        codes[w] = e4m3x2(c[0], c[1]) | (e4m3x2(c[2], c[3]) << 16);
      }
    }
    *reinterpret_cast<uint2*>(y) = make_uint2(codes[0], codes[1]);
  };

  if (one && a.inv_freq) angles(0);
  uint32_t raw[kVec][W];
  if (one) load(h0, 0, raw);
#pragma unroll 1
  for (int h = h0; h < h1; ++h) {
    float old = 0.0f;
    if (u.lo > 0) old = ld_after(a.scale + (size_t)page * a.H + h);
    float v[kVec][8];
    // this pass over the rows: f(vector, its row)
    auto each = [&](auto&& f) {
      if (one) {
        uint8_t* y = y0 + ((int64_t)group * a.H + h) * D;
        if (group < rows) f(v[0], y);
        if (rows > GROUPS) {
#pragma unroll
          for (int i = 1; i < kVec; ++i)
            if (i * GROUPS < rows - group) f(v[i], y + i * y_step);
        }
      } else {
#pragma unroll 1
        for (int r0 = 0; r0 < rows; r0 += CHUNK) {
          if (a.inv_freq) angles(r0);
          load(h, r0, raw);
#pragma unroll
          for (int i = 0; i < kVec; ++i) {
            rotated(i, r0, raw[i], v[i]);
            const int r = r0 + group + i * GROUPS;
            if (r < rows) f(v[i], y0 + ((int64_t)r * a.H + h) * D);
          }
        }
      }
    };
    if (one) {
      rotated(0, 0, raw[0], v[0]);
      if (rows > GROUPS) {  // (uniform)
#pragma unroll
        for (int i = 1; i < kVec; ++i) rotated(i, 0, raw[i], v[i]);
      }
      if (h + 1 < h1) load(h + 1, 0, raw);  // the next head's rows, under this one's work
    }
    uint32_t bits = 0;
    each([&](const float (&x)[8], uint8_t*) { bits = max(bits, largest(x, false)); });
    uint32_t top = block_max(bits);
    const bool odd = top >= kInf;
    if (odd) {
      bits = 0;
      each([&](const float (&x)[8], uint8_t*) { bits = max(bits, largest(x, true)); });
      top = block_max(bits);
      if (threadIdx.x == 0) flag(a.status, HYTOPK_DEV_NONFINITE);
    }
    const float amax = __uint_as_float(top);
    const float fresh = amax > 0.0f ? fmaxf(__fdiv_rn(amax, 448.0f), 1.17549435e-38f) : 0.0f;
    const bool lost = u.lo > 0 && !(old > 0.0f && old <= kMost);
    float scale = lost ? fresh : fmaxf(old, fresh);
    if (scale == 0.0f) scale = 1.0f;
    const bool fast = !odd && scale > 1e-18f && scale < 1e36f;
    const float ninv = -__frcp_rn(scale);
    each([&](const float (&x)[8], uint8_t* y) { store(y, x, scale, ninv, fast); });
    if (u.lo > 0 && (lost || scale > old)) {
      // earlier rows, under the new scale
      const float ratio = lost ? __int_as_float(0x7fc00000) : __fdiv_rn(old, scale);
      for (int f = threadIdx.x; f < u.lo * (D / 16); f += kThreads) {
        uint4* y = reinterpret_cast<uint4*>(
            a.pages + (((size_t)page * a.s.P + f / (D / 16)) * a.H + h) * D + f % (D / 16) * 16);
        const uint4 w4 = *y;
        uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float c[4];
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            uint32_t h2;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)(w[e] >> (16 * p))));
            const float2 two = __half22float2(*reinterpret_cast<const __half2*>(&h2));
            c[2 * p] = two.x * ratio;
            c[2 * p + 1] = two.y * ratio;
          }
          w[e] = e4m3x2(c[0], c[1]) | (e4m3x2(c[2], c[3]) << 16);
        }
        *y = make_uint4(w[0], w[1], w[2], w[3]);
      }
      if (lost && threadIdx.x == 0) flag(a.status, HYTOPK_DEV_BAD_SCALE);
    }
    if (threadIdx.x == 0 && (u.lo == 0 || lost || scale > old))
      a.scale[(size_t)page * a.H + h] = scale;
  }
}

template <typename T, int D>
cudaError_t launch(WriteArgs a, int sms, cudaStream_t st) {
  // pages that the rows can go to at most: each sequence's first and last are shared out
  const int64_t most = (int64_t)a.n / a.s.P + 2 * (int64_t)a.s.B;
  const int64_t units = most < a.n ? most : a.n;
  // Heads of a CTA share the angles; fewer heads where the pages alone do not fill the SMs.
  a.heads = a.H < 8 ? a.H : 8;
  while (a.heads > 1 && units * ((a.H + a.heads - 1) / a.heads) < 4 * (int64_t)sms)
    a.heads = (a.heads + 1) / 2;
  const int64_t grid = units * ((a.H + a.heads - 1) / a.heads);
  if (grid >= (int64_t)1 << 31) return cudaErrorInvalidConfiguration;
  constexpr int CHUNK = kThreads / (D / 8) * kVec;
  const int held = a.s.P < CHUNK ? a.s.P : CHUNK;
  const size_t smem = a.inv_freq ? (size_t)held * a.rot * sizeof(float) : 0;
  return launch_early(k_page_write<T, D>, (unsigned)grid, kThreads, smem, st, 1, a);
}

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace
}  // namespace pages
}  // namespace hytopk

using namespace hytopk;
using namespace hytopk::pages;

extern "C" hytopk_status hytopk_page_write(const void* x, int64_t x_row, int64_t x_head,
                                           hytopk_elem x_type, int n, int H, int d,
                                           const hytopk_rope_params* rope, void* pages,
                                           float* page_scale, const hytopk_paged* paged,
                                           uint32_t* dev_status, cudaStream_t stream) {
  const hytopk_status s = check_paged(paged, n);
  if (s != HYTOPK_OK) return s;
  if (H < 1 || (x_type != HYTOPK_ELEM_BF16 && x_type != HYTOPK_ELEM_F32)) return HYTOPK_INVALID_ARG;
  if (d != 64 && d != 128 && d != 256) return HYTOPK_UNSUPPORTED;
  if (rope) {
    if (rope->rot < 2 || rope->first < 0 || (int64_t)rope->first + rope->rot > d)
      return HYTOPK_INVALID_ARG;
    if (rope->rot % 16 || rope->first % 8) return HYTOPK_UNSUPPORTED;
  }
  if ((int64_t)n * H >= (int64_t)1 << 31) return HYTOPK_UNSUPPORTED;
  if (n == 0 || paged->B == 0) return HYTOPK_OK;
  if (!x || !pages || !page_scale || (rope && !rope->inv_freq)) return HYTOPK_INVALID_ARG;
  const int bytes = x_type == HYTOPK_ELEM_F32 ? 4 : 2;
  if (!aligned(x, 16) || x_row * bytes % 16 || x_head * bytes % 16 || !aligned(pages, 16) ||
      !aligned(page_scale, 4) ||
      (rope && (!aligned(rope->positions, 4) || !aligned(rope->inv_freq, 4))))
    return HYTOPK_MISALIGNED;
  WriteArgs a{};
  a.x = x;
  a.x_row = x_row;
  a.x_head = x_head;
  a.n = n;
  a.H = H;
  if (rope) {
    a.positions = rope->positions;
    a.inv_freq = rope->inv_freq;
    a.rot = rope->rot;
    a.first = rope->first;
    a.interleaved = rope->interleaved;
    a.inverse = rope->inverse;
    a.mscale = rope->mscale;
  }
  a.pages = static_cast<uint8_t*>(pages);
  a.scale = page_scale;
  a.s = *paged;
  a.status = dev_status;
  const int sms = num_sms();
  const bool f32 = x_type == HYTOPK_ELEM_F32;
  cudaError_t e;
  if (d == 64) e = f32 ? launch<float, 64>(a, sms, stream) : launch<__nv_bfloat16, 64>(a, sms, stream);
  else if (d == 128) e = f32 ? launch<float, 128>(a, sms, stream) : launch<__nv_bfloat16, 128>(a, sms, stream);
  else e = f32 ? launch<float, 256>(a, sms, stream) : launch<__nv_bfloat16, 256>(a, sms, stream);
  return e == cudaSuccess ? HYTOPK_OK : HYTOPK_CUDA_ERROR;
}
