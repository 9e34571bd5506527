// The paged cache's own kernels: tokens into it (quantised on the way), tokens
// out of it, and the accepted drafted tokens to their final slots.
//
// Write and read move every element once and compute little, so HBM bounds them:
// a cached row is hkv * d contiguous elements, so vectors of eight of them (16
// bytes of bf16, 8 of e4m3) along it coalesce whatever the head count, in the
// loads and in the stores, and each thread keeps several vectors of K and of V
// in flight. The chain cu_tokens -> kv_lens -> page table that leads to a row's
// slot is walked once per CTA (by one warp, for all of the CTA's tokens) while
// the first vectors are already on their way.
// Measured on the device, calls back to back: prompts of 4K-64K tokens, 8 heads,
// into an e4m3 cache 216 us (5.8 TB/s), out of one 198 us (6.4 TB/s), bf16 261 and
// 256 us (6.4 and 6.5 TB/s); a chunk of 32K tokens of 4 heads with token scales
// 24.4 us (4.2 TB/s); one token of eight requests 2.1 us. As calls between whose
// inputs the caches turn cold: 242, 201, 27 and 3.8 us (5.2, 6.3, 3.8 TB/s).
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "cache.cuh"
#include "packed.cuh"

namespace fp {

using namespace packed;

namespace {

constexpr int kMoveThreads = 256;
// CTAs per SM and vectors of K and of V in flight per thread: writing computes, and takes more warps (a chunk of
// whole prompts, e4m3: 220 us with 8 CTAs of one vector, 242 us with 5 of two); reading takes more loads each
// (213 us with 5 of four, 294 us with 8, whose registers spill).
constexpr int kWriteCtas = 8, kWriteVecs = 1, kReadCtas = 5, kReadVecs = 4;
constexpr int kMaxTokensPerCta = 64;
enum Format { kBf16 = 0, kHeadScale = 1, kTokenScale = 2 };

constexpr int kVec = 8;  // elements per thread and step

// The request that row t belongs to: the first r with cu[r + 1] > t (the last
// request if there is none; the caller checks the span). All lanes of the warp
// call it, each with its own t. Up to 32 requests cost one load per lane; more
// are first cut into 32 groups by the same shuffled search.
__device__ __forceinline__ int find_request(const int32_t* cu, int R, int t) {
  const int lane = threadIdx.x & 31;
  const int step = (R + 31) / 32;
  const int bound = __ldg(cu + min((lane + 1) * step, R));  // end of this lane's group
  int grp = 0;
#pragma unroll
  for (int b = 16; b > 0; b >>= 1) {
    const int probe = __shfl_sync(0xffffffffu, bound, grp + b - 1);
    if (probe <= t) grp += b;
  }
  int lo = min(grp * step, R - 1), hi = min(lo + step, R) - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(cu + mid + 1) > t) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

constexpr long long kSkip = -1;   // not a row of any request (or of a rejected one)
constexpr long long kZeros = -2;  // a row on a bad page

// Flat slot (page * page_size + offset) of packed row t, or kSkip / kZeros.
__device__ __forceinline__ long long row_slot(const CacheGeometry& g, const int32_t* starts, int t) {
  const int r = find_request(g.cu, g.R, t);
  int off, n, kv;
  if (!cache_span(g, r, off, n, kv) || t < off || t >= off + n) return kSkip;
  int first = kv - n;
  if (starts) {
    first = __ldg(starts + r);
    if (first < 0 || first > kv - n) {
      atomicOr(g.status, FP_DEV_BAD_SEQLENS);
      return kSkip;
    }
  }
  const int pos = first + (t - off);
  const int page = __ldg(g.table + (long long)r * g.max_pages + (pos >> g.page_shift));
  if (page < 0 || page >= g.num_pages) {
    atomicOr(g.status, FP_DEV_BAD_PAGE);
    return kZeros;
  }
  return ((long long)page << g.page_shift) + (pos & (g.page_size - 1));
}

// Slots of the CTA's tokens t0 .. t0 + nt - 1 into shared memory (warp 0);
// the second warp of CTA 0 checks every request's lengths meanwhile, so that a
// request none of whose rows is visited is reported too.
__device__ __forceinline__ void find_slots(const CacheGeometry& g, const int32_t* starts, int t0, int nt,
                                           long long* slot) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    for (int i = lane; i < (nt + 31) / 32 * 32; i += 32) {
      const long long s = row_slot(g, starts, t0 + min(i, nt - 1));
      if (i < nt) slot[i] = s;
    }
  } else if (warp == 1 && blockIdx.x == 0) {
    for (int r = lane; r < g.R; r += 32) {
      int off, n, kv;
      cache_span(g, r, off, n, kv);
    }
  }
  __syncthreads();
}

__device__ __forceinline__ uint4 load_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ void unpack_bf16(uint32_t u, float& a, float& b) {
  a = __uint_as_float(u << 16);
  b = __uint_as_float(u & 0xffff0000u);
}

// ... with their signs turned, in as many instructions (the low one's sign by the addition)
__device__ __forceinline__ void unpack_minus(uint32_t u, float& a, float& b) {
  uint32_t lo;
  asm("mad.lo.u32 %0, %1, 65536, 0x80000000;" : "=r"(lo) : "r"(u));
  a = __uint_as_float(lo);
  b = __uint_as_float((u & 0xffff0000u) ^ 0x80000000u);
}

// Two float32 -> two e4m3 codes (the first in the low byte), round to nearest
// even, saturating at +-448; NaN stays NaN.
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b) {
  unsigned short h;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(b), "f"(a));
  return h;
}

// What x is divided by, as quantise() takes it.
struct Divisor {
  float scale, inv;
  bool plain;  // neither the reciprocal nor a product of it leaves the normal range where it matters
};
__device__ __forceinline__ Divisor divisor(float scale) {
  const float s = scale == 0.f ? 1.f : scale;
  return {s, __frcp_rn(s), s >= 0x1p-80f && s <= 0x1p80f};
}

// Eight bf16 elements -> eight codes of x / scale, IEEE division. With y the
// correctly rounded reciprocal of s, q = x y and r = x - q s (exact in a fused
// multiply-add), q + r y is the correctly rounded quotient (P. Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor",
// 1990): three packed instructions for two elements. The general division took
// about twelve each and set the pace (4.2 of the 6.5 TB/s). Computed from -x as
// q = (-x)(-y), -r = q s + (-x), q + (-r)(-y): of x = -0 the other signs would
// make +0 (-r = +0 either way, and (+0)(-y) = -0 leaves q's sign).
// BOUNDED: no |x| exceeds 448 s.
template <bool BOUNDED>
__device__ __forceinline__ uint2 quantise(const uint4& in, const Divisor& d) {
  const uint32_t w[4] = {in.x, in.y, in.z, in.w};
  uint32_t code[4];
  const uint64_t ny = f2_pack(-d.inv, -d.inv), s = f2_pack(d.scale, d.scale);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;  // -x
    unpack_minus(w[i], a, b);
    float qa, qb;
    if (d.plain) {
      const uint64_t nx = f2_pack(a, b), q = f2_mul(nx, ny);
      float pa, pb;
      f2_unpack(q, pa, pb);
      f2_unpack(f2_fma(f2_fma(q, s, nx), ny, q), qa, qb);
      if constexpr (!BOUNDED) {  // far beyond the largest code the estimate does, and the correction may overflow
        qa = fabsf(pa) < 1024.f ? qa : pa;
        qb = fabsf(pb) < 1024.f ? qb : pb;
      }
    } else {
      qa = __fdiv_rn(a, -d.scale);
      qb = __fdiv_rn(b, -d.scale);
    }
    code[i] = pack_e4m3(qa, qb);
  }
  return make_uint2(code[0] | (code[1] << 16), code[2] | (code[3] << 16));
}

// m / 448, IEEE division, the same way (m >= 0; general division took a tenth of the whole chunk's time).
__device__ __forceinline__ float over_448(float m) {
  constexpr float inv = 1.f / 448.f;
  const float q = m * inv;
  return m >= 0x1p-90f && m < INFINITY ? fmaf(fmaf(-q, 448.f, m), inv, q) : __fdiv_rn(m, 448.f);
}

// max |x| of K's and of V's vector over the sixteen lanes that hold one head's 128 elements (NaN does not count). The
// bits of |x| order as integers, so two values are compared at a time, and K and V share the shuffles.
__device__ __forceinline__ float2 head_absmax(const uint4& k, const uint4& v) {
  auto top = [](const uint4& x) {
    const uint32_t m = 0x7fff7fffu;
    return __vmaxu2(__vmaxu2(x.x & m, x.y & m), __vmaxu2(x.z & m, x.w & m));
  };
  const uint32_t tk = top(k), tv = top(v);
  uint32_t both = __vmaxu2(__byte_perm(tk, tv, 0x5410), __byte_perm(tk, tv, 0x7632));  // low half K, high half V
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) both = __vmaxu2(both, __shfl_xor_sync(0xffffffffu, both, o, 16));
  float2 out = make_float2(__uint_as_float(both << 16), __uint_as_float(both & 0xffff0000u));
  // NaN bits are above infinity's: then the ordinary way
  if (__any_sync(0xffffffffu, (both & 0xffffu) > 0x7f80u || (both >> 16) > 0x7f80u)) {
    auto slow = [](const uint4& x) {
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
      float m = 0.f;
      for (int i = 0; i < 4; ++i) {
        float a, b;
        unpack_bf16(w[i], a, b);
        m = fmaxf(m, fmaxf(fabsf(a), fabsf(b)));
      }
      for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o, 16));
      return m;
    };
    out = make_float2(slow(k), slow(v));
  }
  return out;
}

struct MoveArgs {
  CacheGeometry g;
  const int32_t* starts;
  const uint8_t* k;  // packed rows (write: source, read: destination)
  const uint8_t* v;
  long long k_stride, v_stride;  // bytes between tokens
  int tokens;                    // per CTA
  int vecs;                      // vectors per cached row of K (and of V)
  uint32_t vecs_inv;             // ceil(2^32 / vecs): i / vecs = (i * vecs_inv) >> 32 below 2^32 / vecs
};

// Cached row -> (page, slot-in-page) parts of the token scale's address.
__device__ __forceinline__ long long scale_index(const CacheGeometry& g, long long slot, int head) {
  const long long page = slot >> g.page_shift;
  return ((page * g.Hkv + head) << g.page_shift) + (slot & (g.page_size - 1));
}

template <int FMT>
__global__ void __launch_bounds__(kMoveThreads, kWriteCtas) cache_write_kernel(const MoveArgs a) {
  constexpr int U = kWriteVecs;
  __shared__ long long slot[kMaxTokensPerCta];
  const CacheGeometry& g = a.g;
  const int t0 = blockIdx.x * a.tokens;
  const int nt = min(a.tokens, g.total_tokens - t0);
  const int items = nt * a.vecs;
  const int rounds = (items + U * kMoveThreads - 1) / (U * kMoveThreads);
  uint4 in[2][U];
  auto load = [&](int round, int u) {
    const int i = (round * U + u) * kMoveThreads + threadIdx.x;
    if (i < items) {
      const int t = __umulhi(i, a.vecs_inv), x = i - t * a.vecs;
      in[0][u] = load_stream(a.k + (t0 + t) * a.k_stride + x * 16);
      in[1][u] = load_stream(a.v + (t0 + t) * a.v_stride + x * 16);
    }
  };
#pragma unroll
  for (int u = 0; u < U; ++u) load(0, u);
  find_slots(g, a.starts, t0, nt, slot);
  for (int round = 0; round < rounds; ++round) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = (round * U + u) * kMoveThreads + threadIdx.x;
      // (whole warps go on: the absmax shuffles need their sixteen lanes)
      if (__all_sync(0xffffffffu, i >= items)) continue;
      const int j = min(i, items - 1), t = __umulhi(j, a.vecs_inv), x = j - t * a.vecs;
      const long long s = i < items ? slot[t] : kSkip;
      float2 top;
      if constexpr (FMT == kTokenScale) top = head_absmax(in[0][u], in[1][u]);
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        uint8_t* pool = which ? g.v_pool : g.k_pool;
        if constexpr (FMT == kBf16) {
          if (s >= 0) reinterpret_cast<uint4*>(pool)[s * a.vecs + x] = in[which][u];
        } else {
          float* scales = which ? g.v_scale : g.k_scale;
          const int head = x >> 4;
          float sc;
          if constexpr (FMT == kTokenScale) {
            sc = over_448(which ? top.y : top.x);
            if (s >= 0 && (x & 15) == 0) scales[scale_index(g, s, head)] = sc;
          } else {
            sc = __ldg(scales + head);
          }
          const uint2 codes = quantise<FMT == kTokenScale>(in[which][u], divisor(sc));
          if (s >= 0) reinterpret_cast<uint2*>(pool)[s * a.vecs + x] = codes;
        }
      }
      load(round + 1, u);  // on its way while the other vectors are worked on
    }
  }
}

__device__ __forceinline__ float2 e4m3_pair(uint32_t two_bytes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)two_bytes));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Four codes * scale -> four bf16 (float32 product, rounded to nearest even once)
__device__ __forceinline__ uint2 dequantise4(uint32_t codes, float scale) {
  const float2 a = e4m3_pair(codes & 0xffffu), b = e4m3_pair(codes >> 16);
  const __nv_bfloat162 lo = __floats2bfloat162_rn(a.x * scale, a.y * scale);
  const __nv_bfloat162 hi = __floats2bfloat162_rn(b.x * scale, b.y * scale);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

__device__ __forceinline__ uint2 load_stream8(const void* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

template <int FMT>
__global__ void __launch_bounds__(kMoveThreads, kReadCtas) cache_read_kernel(const MoveArgs a) {
  constexpr int U = kReadVecs;
  __shared__ long long slot[kMaxTokensPerCta];
  const CacheGeometry& g = a.g;
  const int t0 = blockIdx.x * a.tokens;
  const int nt = min(a.tokens, g.total_tokens - t0);
  const int items = nt * a.vecs;
  find_slots(g, a.starts, t0, nt, slot);
  using Vec = std::conditional_t<FMT == kBf16, uint4, uint2>;
  for (int i0 = threadIdx.x; i0 < items; i0 += U * kMoveThreads) {
    Vec in[2][U];
    float sc[2][U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kMoveThreads;
      if (i >= items) break;
      const int t = __umulhi(i, a.vecs_inv), x = i - t * a.vecs;
      const long long s = slot[t];
      const int head = x >> 4;
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        const uint8_t* pool = which ? g.v_pool : g.k_pool;
        const float* scales = which ? g.v_scale : g.k_scale;
        in[which][u] = Vec{};
        sc[which][u] = 0.f;
        if (s >= 0) {
          const Vec* p = reinterpret_cast<const Vec*>(pool) + s * a.vecs + x;
          if constexpr (FMT == kBf16) in[which][u] = load_stream(p);
          else in[which][u] = load_stream8(p);
          if constexpr (FMT == kHeadScale) sc[which][u] = __ldg(scales + head);
          if constexpr (FMT == kTokenScale) sc[which][u] = __ldg(scales + scale_index(g, s, head));
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kMoveThreads;
      if (i >= items) break;
      const int t = __umulhi(i, a.vecs_inv), x = i - t * a.vecs;
      if (slot[t] == kSkip) continue;
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        uint8_t* dst =
            const_cast<uint8_t*>(which ? a.v : a.k) + (t0 + t) * (which ? a.v_stride : a.k_stride) + x * 16;
        if constexpr (FMT == kBf16) {
          *reinterpret_cast<uint4*>(dst) = in[which][u];
        } else {
          const float f = sc[which][u];
          const uint2 lo = dequantise4(in[which][u].x, f), hi = dequantise4(in[which][u].y, f);
          *reinterpret_cast<uint4*>(dst) = make_uint4(lo.x, lo.y, hi.x, hi.y);
        }
      }
    }
  }
}

// One CTA per request; a thread owns 16-byte columns of the row (K's, then
// V's) and takes all accepted tokens through it in ascending order. Accepted
// indices are strictly ascending, so accept[i] >= i: a source row is never
// among the destinations written before it is read, and no column needs
// another's progress. Four rows are in flight per column.
template <bool TOKEN>
__global__ void __launch_bounds__(kMoveThreads)
    cache_commit_kernel(const CacheGeometry g, const int32_t* __restrict__ accept,
                        const int32_t* __restrict__ num_accept, int max_accept, int32_t* new_lens, int row_vecs) {
  extern __shared__ long long slots[];  // [2][max_accept]: source and destination of every accepted token
  const int r = blockIdx.x;
  int off, n, kv;
  const int num = __ldg(num_accept + r);
  const bool fits = cache_span(g, r, off, n, kv);
  const int base = kv - n;
  int bad = 0;
  if (num < 0 || num > max_accept) bad = FP_DEV_BAD_LIST;
  if (!fits) bad = FP_DEV_BAD_SEQLENS;
  if (!bad) {
    const int32_t* list = accept + (long long)r * max_accept;
    for (int i = threadIdx.x; i < num; i += kMoveThreads) {
      const int j = __ldg(list + i);
      // i <= j holds in an ascending list; it keeps `to` a cached position in any other
      if (j < 0 || j >= n || i > j || (i > 0 && __ldg(list + i - 1) >= j)) {
        bad |= FP_DEV_BAD_LIST;
        continue;
      }
      const int32_t* row = g.table + (long long)r * g.max_pages;
      const int from = base + j, to = base + i;
      const int p = __ldg(row + (from >> g.page_shift)), q = __ldg(row + (to >> g.page_shift));
      if (p < 0 || p >= g.num_pages || q < 0 || q >= g.num_pages) {
        bad |= FP_DEV_BAD_PAGE;
        continue;
      }
      slots[i] = ((long long)p << g.page_shift) + (from & (g.page_size - 1));
      slots[max_accept + i] = ((long long)q << g.page_shift) + (to & (g.page_size - 1));
    }
  }
  if (bad) atomicOr(g.status, (unsigned)bad);
  if (__syncthreads_or(bad)) {  // every thread has read kv_lens[r] before new_lens[r], perhaps the same word, changes
    if (threadIdx.x == 0) new_lens[r] = kv;
    return;
  }
  const long long* src = slots;
  const long long* dst = slots + max_accept;
  for (int x = threadIdx.x; x < 2 * row_vecs; x += kMoveThreads) {
    uint4* col = reinterpret_cast<uint4*>(x < row_vecs ? g.k_pool : g.v_pool) + (x < row_vecs ? x : x - row_vecs);
    for (int i = 0; i < num; i += 4) {
      uint4 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (i + u < num) v[u] = col[src[i + u] * row_vecs];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (i + u < num && src[i + u] != dst[i + u]) col[dst[i + u] * row_vecs] = v[u];
    }
  }
  if constexpr (TOKEN) {
    for (int x = threadIdx.x; x < 2 * g.Hkv; x += kMoveThreads) {
      float* sc = x < g.Hkv ? g.k_scale : g.v_scale;
      const int head = x < g.Hkv ? x : x - g.Hkv;
      for (int i = 0; i < num; i += 4) {
        float v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (i + u < num) v[u] = sc[scale_index(g, src[i + u], head)];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (i + u < num) sc[scale_index(g, dst[i + u], head)] = v[u];
      }
    }
  }
  if (threadIdx.x == 0) new_lens[r] = base + num;
}

// Tokens per CTA: as few as fill the SMs' CTAs at most once, and up to so many vectors of K that the chain of lookups is a
// small part of a CTA's life (one head of 128, token scales: 22.5 us for a write of 110K tokens, 24.6 us with 16 tokens per
// CTA). More than that leaves an uneven end: reads of whole prompts with 64 tokens of 8 heads took 213 us, not 197.
constexpr int kVectorsPerCta = 2048;

MoveArgs move_args(const CacheGeometry& g, const int32_t* starts, const void* k, long long k_stride, const void* v,
                   long long v_stride, int ctas_per_sm) {
  MoveArgs a;
  a.g = g;
  a.starts = starts;
  a.k = static_cast<const uint8_t*>(k);
  a.v = static_cast<const uint8_t*>(v);
  a.k_stride = k_stride * 2;
  a.v_stride = v_stride * 2;
  a.vecs = g.Hkv * g.d / kVec;
  a.vecs_inv = (uint32_t)(((1ull << 32) + a.vecs - 1) / a.vecs);
  const int ctas = sm_count() * ctas_per_sm, per = (int)(((long long)g.total_tokens + ctas - 1) / ctas);
  const int most = kVectorsPerCta / a.vecs < kMaxTokensPerCta ? kVectorsPerCta / a.vecs : kMaxTokensPerCta;
  a.tokens = per > most ? (most > 1 ? most : 1) : per;
  return a;
}

}  // namespace

cudaError_t launch_cache_write(const CacheGeometry& g, const void* k, long long k_stride, const void* v,
                               long long v_stride, cudaStream_t s) {
  const MoveArgs a = move_args(g, nullptr, k, k_stride, v, v_stride, kWriteCtas);
  const int grid = (g.total_tokens + a.tokens - 1) / a.tokens;
  if (!g.e4m3) cache_write_kernel<kBf16><<<grid, kMoveThreads, 0, s>>>(a);
  else if (g.token_scale) cache_write_kernel<kTokenScale><<<grid, kMoveThreads, 0, s>>>(a);
  else cache_write_kernel<kHeadScale><<<grid, kMoveThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_cache_read(const CacheGeometry& g, const int32_t* starts, void* k, long long k_stride, void* v,
                              long long v_stride, cudaStream_t s) {
  const MoveArgs a = move_args(g, starts, k, k_stride, v, v_stride, kReadCtas);
  const int grid = (g.total_tokens + a.tokens - 1) / a.tokens;
  if (!g.e4m3) cache_read_kernel<kBf16><<<grid, kMoveThreads, 0, s>>>(a);
  else if (g.token_scale) cache_read_kernel<kTokenScale><<<grid, kMoveThreads, 0, s>>>(a);
  else cache_read_kernel<kHeadScale><<<grid, kMoveThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_cache_commit(const CacheGeometry& g, const int32_t* accept, const int32_t* num_accept,
                                int max_accept, int32_t* new_lens, cudaStream_t s) {
  const int row_vecs = g.Hkv * g.d * (g.e4m3 ? 1 : 2) / 16;
  const size_t smem = (size_t)2 * max_accept * sizeof(long long);
  if (g.token_scale)
    cache_commit_kernel<true><<<g.R, kMoveThreads, smem, s>>>(g, accept, num_accept, max_accept, new_lens, row_vecs);
  else
    cache_commit_kernel<false><<<g.R, kMoveThreads, smem, s>>>(g, accept, num_accept, max_accept, new_lens, row_vecs);
  return cudaGetLastError();
}

}  // namespace fp
