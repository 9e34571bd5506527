// The paged cache's own kernels: tokens into it (quantised on the way), tokens
// out of it, and the accepted drafted tokens to their final slots.
//
// Write and read move every element once and compute next to nothing, so HBM
// bounds them: a cached row is hkv * d contiguous elements, so 16-byte vectors
// along it coalesce whatever the head count, and each thread keeps several
// vectors of K and of V in flight. The chain cu_tokens -> kv_lens -> page table
// that leads to a row's slot is walked once per CTA (by one warp, for all of the
// CTA's tokens) while the first vectors are already on their way.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "internal.cuh"

namespace fp {

namespace {

constexpr int kMoveThreads = 256;
constexpr int kMaxTokensPerCta = 64;
enum Format { kBf16 = 0, kHeadScale = 1, kTokenScale = 2 };

// Elements per thread and step: one 16-byte vector of the cached row.
template <int FMT>
constexpr int kVec = FMT == kBf16 ? 8 : 16;

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

// Two float32 -> two e4m3 codes (the first in the low byte), round to nearest
// even, saturating at +-448; NaN stays NaN.
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b) {
  unsigned short h;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(b), "f"(a));
  return h;
}

// 16 bf16 elements as loaded (two vectors) -> 16 codes of x / scale.
__device__ __forceinline__ uint4 quantise16(const uint4 (&in)[2], float scale) {
  const uint32_t w[8] = {in[0].x, in[0].y, in[0].z, in[0].w, in[1].x, in[1].y, in[1].z, in[1].w};
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b, c, d;
    unpack_bf16(w[2 * i], a, b);
    unpack_bf16(w[2 * i + 1], c, d);
    out[i] = pack_e4m3(__fdiv_rn(a, scale), __fdiv_rn(b, scale)) |
             (pack_e4m3(__fdiv_rn(c, scale), __fdiv_rn(d, scale)) << 16);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

// max |x| over the eight lanes that hold one head's 128 elements (NaN does not count)
__device__ __forceinline__ float head_absmax(const uint4 (&in)[2]) {
  const uint32_t w[8] = {in[0].x, in[0].y, in[0].z, in[0].w, in[1].x, in[1].y, in[1].z, in[1].w};
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float a, b;
    unpack_bf16(w[i], a, b);
    m = fmaxf(m, fmaxf(fabsf(a), fabsf(b)));
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o, 8));
  return m;
}

struct MoveArgs {
  CacheGeometry g;
  const int32_t* starts;
  const uint8_t* k;  // packed rows (write: source, read: destination)
  const uint8_t* v;
  long long k_stride, v_stride;  // bytes between tokens
  int tokens;                    // per CTA
  int vecs;                      // vectors per cached row of K (and of V)
};

// Cached row -> (page, slot-in-page) parts of the token scale's address.
__device__ __forceinline__ long long scale_index(const CacheGeometry& g, long long slot, int head) {
  const long long page = slot >> g.page_shift;
  return ((page * g.Hkv + head) << g.page_shift) + (slot & (g.page_size - 1));
}

template <int FMT>
__global__ void __launch_bounds__(kMoveThreads) cache_write_kernel(const MoveArgs a) {
  constexpr int V = kVec<FMT>, L = V / 8;  // elements, and 16-byte loads, per vector
  constexpr int U = 2;                     // vectors of K and of V in flight per thread
  __shared__ long long slot[kMaxTokensPerCta];
  const CacheGeometry& g = a.g;
  const int t0 = blockIdx.x * a.tokens;
  const int nt = min(a.tokens, g.total_tokens - t0);
  const int items = nt * a.vecs;
  // rounded up to whole warps: the absmax shuffles need their eight lanes
  const int rounds = (items + U * kMoveThreads - 1) / (U * kMoveThreads);
  uint4 in[2][U][L];
  auto load = [&](int round) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = (round * U + u) * kMoveThreads + threadIdx.x;
      if (i < items) {
        const int t = i / a.vecs, x = i - t * a.vecs;
        const uint8_t* kp = a.k + (t0 + t) * a.k_stride + (long long)x * (V * 2);
        const uint8_t* vp = a.v + (t0 + t) * a.v_stride + (long long)x * (V * 2);
#pragma unroll
        for (int l = 0; l < L; ++l) {
          in[0][u][l] = load_stream(kp + l * 16);
          in[1][u][l] = load_stream(vp + l * 16);
        }
      }
    }
  };
  load(0);
  find_slots(g, a.starts, t0, nt, slot);
  for (int round = 0; round < rounds; ++round) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = (round * U + u) * kMoveThreads + threadIdx.x;
      if (__all_sync(0xffffffffu, i >= items)) continue;
      const int t = min(i, items - 1) / a.vecs, x = min(i, items - 1) - t * a.vecs;
      const long long s = i < items ? slot[t] : kSkip;
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        uint8_t* pool = which ? g.v_pool : g.k_pool;
        float* scales = which ? g.v_scale : g.k_scale;
        uint4 out;
        if constexpr (FMT == kBf16) {
          out = in[which][u][0];
        } else {
          const int head = x / (128 / V);
          float sc;
          if constexpr (FMT == kTokenScale) {
            sc = __fdiv_rn(head_absmax(in[which][u]), 448.f);
            if (s >= 0 && x % (128 / V) == 0) scales[scale_index(g, s, head)] = sc;
          } else {
            sc = __ldg(scales + head);
          }
          out = quantise16(in[which][u], sc == 0.f ? 1.f : sc);
        }
        if (s >= 0) reinterpret_cast<uint4*>(pool)[s * a.vecs + x] = out;
      }
    }
    if (round + 1 < rounds) load(round + 1);
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

template <int FMT>
__global__ void __launch_bounds__(kMoveThreads) cache_read_kernel(const MoveArgs a) {
  constexpr int V = kVec<FMT>;
  constexpr int U = 2;
  __shared__ long long slot[kMaxTokensPerCta];
  const CacheGeometry& g = a.g;
  const int t0 = blockIdx.x * a.tokens;
  const int nt = min(a.tokens, g.total_tokens - t0);
  const int items = nt * a.vecs;
  find_slots(g, a.starts, t0, nt, slot);
  for (int i0 = threadIdx.x; i0 < items; i0 += U * kMoveThreads) {
    uint4 in[2][U];
    float sc[2][U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kMoveThreads;
      if (i >= items) break;
      const int t = i / a.vecs, x = i - t * a.vecs;
      const long long s = slot[t];
      const int head = x / (128 / V);
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        const uint8_t* pool = which ? g.v_pool : g.k_pool;
        const float* scales = which ? g.v_scale : g.k_scale;
        in[which][u] = make_uint4(0, 0, 0, 0);
        sc[which][u] = 0.f;
        if (s >= 0) {
          in[which][u] = load_stream(reinterpret_cast<const uint4*>(pool) + s * a.vecs + x);
          if constexpr (FMT == kHeadScale) sc[which][u] = __ldg(scales + head);
          if constexpr (FMT == kTokenScale) sc[which][u] = __ldg(scales + scale_index(g, s, head));
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kMoveThreads;
      if (i >= items) break;
      const int t = i / a.vecs, x = i - t * a.vecs;
      if (slot[t] == kSkip) continue;
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        uint8_t* dst = const_cast<uint8_t*>(which ? a.v : a.k) + (t0 + t) * (which ? a.v_stride : a.k_stride) +
                       (long long)x * (V * 2);
        const uint4 c = in[which][u];
        if constexpr (FMT == kBf16) {
          *reinterpret_cast<uint4*>(dst) = c;
        } else {
          const float f = sc[which][u];
          const uint2 p0 = dequantise4(c.x, f), p1 = dequantise4(c.y, f), p2 = dequantise4(c.z, f),
                      p3 = dequantise4(c.w, f);
          reinterpret_cast<uint4*>(dst)[0] = make_uint4(p0.x, p0.y, p1.x, p1.y);
          reinterpret_cast<uint4*>(dst)[1] = make_uint4(p2.x, p2.y, p3.x, p3.y);
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

// Tokens per CTA: as many as leave every SM eight CTAs (its 2048 threads), up
// to the slots' array, so that one token's chain of lookups serves many vectors.
MoveArgs move_args(const CacheGeometry& g, const int32_t* starts, const void* k, long long k_stride, const void* v,
                   long long v_stride) {
  MoveArgs a;
  a.g = g;
  a.starts = starts;
  a.k = static_cast<const uint8_t*>(k);
  a.v = static_cast<const uint8_t*>(v);
  a.k_stride = k_stride * 2;
  a.v_stride = v_stride * 2;
  a.vecs = g.Hkv * g.d / (g.e4m3 ? 16 : 8);
  const int per = g.total_tokens / (148 * 8);
  a.tokens = per < 1 ? 1 : (per > kMaxTokensPerCta ? kMaxTokensPerCta : per);
  return a;
}

}  // namespace

cudaError_t launch_cache_write(const CacheGeometry& g, const void* k, long long k_stride, const void* v,
                               long long v_stride, cudaStream_t s) {
  const MoveArgs a = move_args(g, nullptr, k, k_stride, v, v_stride);
  const int grid = (g.total_tokens + a.tokens - 1) / a.tokens;
  if (!g.e4m3) cache_write_kernel<kBf16><<<grid, kMoveThreads, 0, s>>>(a);
  else if (g.token_scale) cache_write_kernel<kTokenScale><<<grid, kMoveThreads, 0, s>>>(a);
  else cache_write_kernel<kHeadScale><<<grid, kMoveThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_cache_read(const CacheGeometry& g, const int32_t* starts, void* k, long long k_stride, void* v,
                              long long v_stride, cudaStream_t s) {
  const MoveArgs a = move_args(g, starts, k, k_stride, v, v_stride);
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
