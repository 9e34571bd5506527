// What the kernels of the tree attention share: their arguments, the axis of key
// tiles that is cut over the SMs, and small conversions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "cache.cuh"
#include "sm100.cuh"

namespace fp {
namespace tree {

// The reference of a row's exponents rises only when its maximum exceeds it by
// more than kSlack (log2 units): nearly every step of a short run would raise
// the exact maximum of one of the rows, and each rise rescales O. f16 weights
// (e4m3 caches) carry a factor 2^kShift: at most 2^15, and normal down to 2^-22
// below the reference.
constexpr float kSlack = 7.f, kShift = 8.f;

struct TreeArgs {
  CacheGeometry g;
  int Hq, G;
  uint32_t G_inv;         // ceil(2^32 / G)
  int max_tokens;
  int rows, rows_shift;   // rows per unit, a power of two
  int tile, tile_shift;   // keys per tile, a power of two
  int lead;               // places on the axis before a unit's tiles: what a segment costs beside them, in tiles
  int min_share;          // places of a CTA at least
  const uint32_t* mask;
  int mask_words;
  const __nv_bfloat16* q;
  long long q_stride;
  __nv_bfloat16* o;
  float* lse;
  float scale_log2;
  float* part_o;          // [2 * grid][rows][d]
  float* part_lse;        // [2 * grid][rows], base 2
  int grid;
};

// ---------------------------------------------------------------------------
// the axis of tiles
// ---------------------------------------------------------------------------
// Every unit takes `lead` places and then one per key tile. The CTAs' shares are
// equal runs of places, so that many short units are spread as evenly as the
// tiles of a few long ones (28 rows over five requests, one of 14 tokens: the
// CTA that got all heads of the short one took twice as long as the others).
// Where a request's rows and keys lie (n = 0: empty, or rejected).
struct Span {
  int off, n, kv;
};

__device__ __forceinline__ Span load_span(const TreeArgs& a, int r) {
  Span s;
  if (!cache_span<true>(a.g, r, s.off, s.n, s.kv)) {
    s.n = 0;
  } else if (s.n > a.max_tokens) {
    atomicOr(a.g.status, FP_DEV_BAD_SEQLENS);
    s.n = 0;
  }
  return s;
}

// Tiles of a request's keys, and units per KV head.
__device__ __forceinline__ int tiles_of(const TreeArgs& a, const Span& s) {
  return s.n == 0 ? 0 : (s.kv + a.tile - 1) >> a.tile_shift;
}
__device__ __forceinline__ int units_of(const TreeArgs& a, const Span& s) {
  return (s.n * a.G + a.rows - 1) >> a.rows_shift;
}

// Requests whose spans are kept in shared memory beside the prefix (16 bytes each; of more, 4 bytes each). Every
// role of every CTA asks for them at each segment: loads of the same few lines by all of the GPU's warps took
// 2700 clocks where shared memory takes 100.
constexpr int kSpanTable = 1024;
__host__ __device__ constexpr int axis_bytes(int R) { return (R + 1) * (R <= kSpanTable ? 16 : 4); }
constexpr int kAxisBytesMax = axis_bytes(kSpanTable) > axis_bytes(4096) ? axis_bytes(kSpanTable) : axis_bytes(4096);

// The requests along the axis: first place of each, and its span.
struct Axis {
  int* mem;  // axis_bytes(R) of shared memory, 16-byte aligned
  int R;
  bool spans;

  __device__ __forceinline__ Axis(void* m, int requests)
      : mem(static_cast<int*>(m)), R(requests), spans(requests <= kSpanTable) {}
  __device__ __forceinline__ int first(int r) const { return spans ? mem[4 * r] : mem[r]; }
  __device__ __forceinline__ int total() const { return first(R); }
  __device__ __forceinline__ Span span(const TreeArgs& a, int r) const {
    if (!spans) return load_span(a, r);
    const int4 v = reinterpret_cast<const int4*>(mem)[r];
    return {v.y, v.z, v.w};
  }
  __device__ __forceinline__ void put(int r, int at, const Span& s) {
    if (spans) reinterpret_cast<int4*>(mem)[r] = make_int4(at, s.off, s.n, s.kv);
    else mem[r] = at;
  }

  // All threads of the block; `warp_sum` has one int per warp. Ends with a block barrier. The host bounds the
  // total by INT_MAX.
  __device__ __forceinline__ void build(const TreeArgs& a, int* warp_sum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int carry = 0;
    const int threads = R <= 32 ? 32 : blockDim.x;  // few requests: one warp, without barriers
    if (threadIdx.x < threads) {
      for (int r0 = 0; r0 < R; r0 += threads) {
        const int r = r0 + threadIdx.x;
        Span s = {0, 0, 0};
        int mine = 0;
        if (r < R) {
          s = load_span(a, r);
          mine = s.n == 0 ? 0 : (a.lead + tiles_of(a, s)) * units_of(a, s) * a.g.Hkv;
        }
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        int before = carry;
        if (threads == 32) {
          carry += __shfl_sync(0xffffffffu, incl, 31);
        } else {
          if (lane == 31) warp_sum[warp] = incl;
          __syncthreads();
          for (int w = 0; w < warps; ++w) {
            if (w < warp) before += warp_sum[w];
            carry += warp_sum[w];
          }
          __syncthreads();
        }
        if (r < R) put(r, before + incl - mine, s);
      }
      if (threadIdx.x == 0) put(R, carry, {0, 0, 0});
    }
    __syncthreads();
  }

  // The request that place x belongs to (0 <= x < total).
  __device__ __forceinline__ int request_of(int x) const {
    int lo = 0, hi = R - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (first(mid + 1) > x) hi = mid;
      else lo = mid + 1;
    }
    return lo;
  }
};

// row / G, for rows below 2^16
__device__ __forceinline__ int group_of(const TreeArgs& a, int row) {
  return a.G == 1 ? row : (int)__umulhi((uint32_t)row, a.G_inv);
}
// x / y for 0 <= x, 0 < y: below 2^20 the float32 quotient (off by 2^-22 of it) is wrong by one at most.
__device__ __forceinline__ int quotient(int x, int y) {
  if (x < y) return 0;
  if (x >= 1 << 20) return x / y;
  int q = (int)__fdividef((float)x, (float)y);
  const int rest = x - q * y;
  return rest < 0 ? q - 1 : rest >= y ? q + 1 : q;
}

__device__ __forceinline__ int share_of(const TreeArgs& a, int total) {
  return max(quotient(total + a.grid - 1, a.grid), a.min_share);
}

// One run of tiles of one unit within a CTA's share.
struct Segment {
  int r, off, n, kv, base;
  int head, row0;    // KV head, first row of the M-tile
  int t0, t1, nt;    // tiles t0 .. t1 - 1 of nt
  __device__ __forceinline__ bool whole() const { return t1 - t0 == nt; }
};

// The segment that begins at place x of a share that ends at `end`; x goes on
// behind it. False if its places hold no tile.
__device__ __forceinline__ bool next_segment(const TreeArgs& a, const Axis& axis, int& x, int end, int& r, Segment& s) {
  while (axis.first(r + 1) <= x) ++r;
  const Span sp = axis.span(a, r);
  s.r = r;
  s.off = sp.off;
  s.n = sp.n;
  s.kv = sp.kv;
  s.nt = tiles_of(a, sp);
  s.base = s.kv - s.n;
  const int nm = units_of(a, sp), y = x - axis.first(r), len = a.lead + s.nt, unit = quotient(y, len);
  const int u0 = y - unit * len, u1 = min(len, u0 + (end - x));
  s.t0 = max(u0 - a.lead, 0);
  s.t1 = max(u1 - a.lead, 0);
  s.head = quotient(unit, nm);
  s.row0 = (unit - s.head * nm) * a.rows;
  x += u1 - u0;
  return s.t1 > s.t0;
}

// Which of the 32 positions from pos0 on a row of token `tok` sees, as bits (`in`: the row exists).
__device__ __forceinline__ uint32_t row_sees(const TreeArgs& a, const Segment& sg, bool in, int tok, int pos0) {
  const int there = sg.kv - pos0;  // positions behind the last token
  const uint32_t some = there >= 32 ? 0xffffffffu : there > 0 ? (1u << there) - 1u : 0u;
  const int j0 = pos0 - sg.base;   // the first position as a new token
  if (j0 <= -32) return some;
  const uint32_t cached = j0 < 0 ? (1u << -j0) - 1u : 0u;
  uint32_t bits = 0;
  if (in && a.mask) {
    const uint32_t* words = a.mask + (long long)(sg.off + tok) * a.mask_words;
    auto word = [&](int i) -> uint32_t { return i >= 0 && i * 32 < sg.n ? __ldg(words + i) : 0u; };
    const int i = j0 >> 5;  // (-1 for negative j0)
    bits = __funnelshift_r(word(i), word(i + 1), j0 & 31);
  } else if (in) {
    const int seen = tok + 1 - j0;  // (j0 + bit <= tok)
    bits = seen >= 32 ? 0xffffffffu : seen > 0 ? (1u << seen) - 1u : 0u;
  }
  return (bits | cached) & some;
}

// ---------------------------------------------------------------------------
// conversions and copies
// ---------------------------------------------------------------------------
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Token scales of V. A weight p = 2^(x - ref + kShift) times v_scale goes to f16 as
//   p (v_scale 2^-kScaleShift) 2^(ref - vref + kScaleShift) = 2^(x + log2 v_scale - vref + kShift)
// with vref, as ref, a row's maximum of x + log2 v_scale at its last rise: at most 2^15, whatever the scales of keys
// that the row does not see. The shift keeps both products within float32 for scales up to its largest value and
// rows whose scales are all tiny. Scales below 2^-100 count as 2^-100 here (their products just stay smaller).
constexpr float kScaleShift = 16.f, kScaleDown = 0x1p-16f;
__device__ __forceinline__ float scale_log2(float v) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(v));
  return fminf(fmaxf(y, -100.f), 128.f);  // (of NaN -100: what it enters becomes NaN by the scale itself)
}
__device__ __forceinline__ float products_factor(float ref, float vref) {
  return vref == -INFINITY ? 0.f : exp2_fast(ref - vref + kScaleShift);
}
// O relative to vref becomes O / sum, with sum relative to ref, by two multiplications with this factor (one with its square
// could leave float32's range). Zero where a row saw nothing.
__device__ __forceinline__ float products_back(float ref, float vref, float sum) {
  return sum == 0.f ? 0.f : exp2_fast(0.5f * (vref - ref)) * rsqrtf(sum);
}

// Two float32 -> two e4m3 codes (the first in the low byte), nearest even, NaN stays NaN.
__device__ __forceinline__ uint32_t pack_codes(float a, float b) {
  unsigned short h;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(b), "f"(a));
  return h;
}

// The low or high pair of four e4m3 codes -> two f16 (exact).
__device__ __forceinline__ uint32_t widen_lo(uint32_t x) {
  uint32_t u;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(u) : "r"(x));
  return u;
}
__device__ __forceinline__ uint32_t widen_hi(uint32_t x) {
  uint32_t u;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(u) : "r"(x));
  return u;
}

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t u;
  if constexpr (F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(u) : "f"(hi), "f"(lo));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u) : "f"(hi), "f"(lo));
  return u;
}

// What bf16 keeps of (lo, hi) after their bf16 pair `u`.
__device__ __forceinline__ uint32_t pack_rest(float lo, float hi, uint32_t u) {
  return pack2<false>(lo - __uint_as_float(u << 16), hi - __uint_as_float(u & 0xffff0000u));
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// The whole producer warp, before a tile's copies: zeros for the scales of a bad page (its codes are zeros; whatever
// scale another page has may be NaN). Returns the bytes that the scales' copies bring.
__device__ __forceinline__ uint32_t scales_of_tile(float* scales, bool bad, bool mine, int lane, int sub_rows) {
  if (__any_sync(0xffffffffu, bad)) {
    if (bad)
      for (int k = 0; k < sub_rows; ++k) scales[lane * sub_rows + k] = 0.f;
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // (later copies come to the same place)
    __syncwarp();
  }
  return (uint32_t)__popc(__ballot_sync(0xffffffffu, mine && !bad)) * (uint32_t)sub_rows * 4u;
}

// Infinities and NaN that new tokens of a segment (tiles t0 .., positions below
// `end`) hold in two columns of V reach the rows that see them: their sums for
// token t, else zeros (rare: they entered the products as zeros). By value, so
// that nothing of the callers' has to lie in memory.
template <bool E4M3, bool TOKEN, int D>
__device__ __noinline__ float2 odd_values(const TreeArgs& a, int r, int off, int head, int base, int t0, int end, int t,
                                          int d) {
  float2 acc = make_float2(0.f, 0.f);
  const CacheGeometry& g = a.g;
  const int32_t* row = g.table + (long long)r * g.max_pages;
  for (int pos = max(base, t0 << a.tile_shift); pos < end; ++pos) {
    const int j = pos - base;
    const bool see = a.mask ? (__ldg(a.mask + (long long)(off + t) * a.mask_words + (j >> 5)) >> (j & 31)) & 1u : j <= t;
    const int page = __ldg(row + (pos >> g.page_shift));
    if (!see || page < 0 || page >= g.num_pages) continue;
    const long long slot = ((long long)page << g.page_shift) + (pos & (g.page_size - 1));
    const long long at = (slot * g.Hkv + head) * D + d;
    float2 v;
    if constexpr (E4M3) {
      const uint32_t w = widen_lo(*reinterpret_cast<const uint16_t*>(g.v_pool + at));
      v = __half22float2(*reinterpret_cast<const __half2*>(&w));
      if (TOKEN) {
        const float sc = __ldg(g.v_scale + (((long long)page * g.Hkv + head) << g.page_shift) + (pos & (g.page_size - 1)));
        v.x *= sc;
        v.y *= sc;
      }
    } else {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(g.v_pool + at * 2);
      v = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    if (!isfinite(v.x)) acc.x += v.x;
    if (!isfinite(v.y)) acc.y += v.y;
  }
  return acc;
}

// bf16 weights enter the product with V as hi + lo, and infinity times a rest lo <= 0 is NaN. Where a row of finite weights
// got NaN in one of four columns of V: the sums of the infinities and NaN that the keys from .. end - 1 hold there as far as
// token t sees them (rare; a page's slots in turn, with eight loads in flight, until nothing can change any more).
template <int D>
__device__ __noinline__ float4 infinite_values(const TreeArgs& a, int r, int off, int head, int base, int from, int end,
                                               int t, int d) {
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  const CacheGeometry& g = a.g;
  const int32_t* row = g.table + (long long)r * g.max_pages;
  for (int p0 = from; p0 < end;) {
    const int p1 = min(end, (p0 | (g.page_size - 1)) + 1), page = __ldg(row + (p0 >> g.page_shift));
    if (page >= 0 && page < g.num_pages) {
      const uint8_t* v = g.v_pool + 2 * ((((long long)page << g.page_shift) * g.Hkv + head) * D + d);
#pragma unroll 8
      for (int pos = p0; pos < p1; ++pos) {
        const uint2 w = *reinterpret_cast<const uint2*>(v + (long long)(pos & (g.page_size - 1)) * g.Hkv * D * 2);
        const uint32_t m = 0x7f807f80u;
        if (((__vcmpeq2(w.x & m, m) | __vcmpeq2(w.y & m, m))) == 0) continue;
        const int j = pos - base;
        if (j >= 0 &&
            !(a.mask ? (__ldg(a.mask + (long long)(off + t) * a.mask_words + (j >> 5)) >> (j & 31)) & 1u : j <= t))
          continue;
        const float f[4] = {__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                            __uint_as_float(w.y & 0xffff0000u)};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!isfinite(f[e])) acc[e] += f[e];
      }
    }
    if (isnan(acc[0]) && isnan(acc[1]) && isnan(acc[2]) && isnan(acc[3])) break;
    p0 = p1;
  }
  return make_float4(acc[0], acc[1], acc[2], acc[3]);
}

// Lets a kernel take all the dynamic shared memory a CTA can have, and checks that it was built with the registers
// per thread that its setmaxnreg split counts on (a larger split would wait for registers for ever): once per kernel
// and device, as the runtime calls cost a fifth of a launch.
template <class K>
cudaError_t prepare(K kern, int launch_regs, std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  cudaFuncAttributes f;
  if ((e = cudaFuncGetAttributes(&f, kern)) != cudaSuccess) return e;
  if (f.numRegs < launch_regs) return cudaErrorInvalidConfiguration;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// The kernel for many rows (tree_wide.cu): a.rows is 128 or 256.
cudaError_t launch_wide(const TreeArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t s);

}  // namespace tree
}  // namespace fp
