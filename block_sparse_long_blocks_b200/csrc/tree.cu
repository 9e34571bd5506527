// Attention of a tree of drafted tokens (or of single tokens) over the paged cache.
//
// Row rho = t * G + h of a request and KV head is query head h of the group and
// new token t (PackGQA, as in the prefill). With base = kv_len - n:
//   x[rho, j] = scale * log2(e) * q[rho] . k[j]     (token-scale caches: * k_scale[j])
//   row rho sees j < base, and base + u iff bit u of its token's mask is set
//   m = max_j x, p = 2^(x - m), l = sum p, O = sum p v / l, lse = (m + log2 l) ln 2
// Online over the keys: when m grows, l and O are multiplied by 2^(m_old - m).
//
// What bounds it: every cached row is read once per M-tile of 16 or 32 rows,
// 4 * rows flops per element, so up to ~250 rows (bf16) HBM is the floor. The
// keys of ALL requests, KV heads and M-tiles form one axis of tiles (32 KB of K:
// 128 keys of 256 bytes, or 256 of 128), cut evenly over one persistent CTA per SM, however ragged the lengths. A unit
// (request, KV head, M-tile) that lies within one CTA's share is finished there;
// the others leave normalised partial rows (float32 O, base-2 lse) in the
// workspace, at most two per CTA, which a second kernel (a programmatic
// dependent launch) combines in a fixed order: O = sum_i 2^(lse_i - lse) O_i.
//
// A CTA: warp 8 issues TMA copies of K and V tiles (4-D boxes per page, 128-byte
// swizzle, and the tile's token scales) into a ring of five 32 KB slots; warps 0-7 hold the M-tiles' rows as mma.sync fragments (16 rows
// per warp) and split the tile's keys, so no warp waits for another until the
// unit's end, where the key groups' (m, l, O) meet in shared memory.
// mma.sync and not tcgen05 here: 8 or 16 useful rows would fill a sixteenth or
// an eighth of a 128-row tcgen05 tile, and the softmax would run in as many
// threads; at these row counts HBM is the limit and the legacy pipe is ~20 % busy.
//
// Operands: bf16 caches multiply bf16 q and k exactly, and p as bf16 hi + lo
// (two products: the weights keep 16 bits; the tensor pipe has room). e4m3 caches
// widen k and v exactly to f16; q goes to f16 as q * 2^e with e per row such that
// max |q| lies in [2^14, 2^15): exact for every element within 2^-29 of the
// largest. p carries a factor 2^14 (f16's normal range then reaches 2^-28 below
// the running maximum). Token scales of V multiply p, divided by a running power
// of two >= the largest v_scale so far, so p stays within f16.
// Every wait is bounded; after one ran out the consumers go on without waiting
// (their loops have fixed lengths, so they still meet at every barrier) and
// release no slot any more: its copy may be in flight. The producer stops and
// waits for its own copies. Outputs are invalid and FP_DEV_TIMEOUT is set.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <climits>
#include <cmath>
#include <type_traits>

#include "internal.cuh"
#include "sm100.cuh"

namespace fp {

namespace {

constexpr int kWarps = 8;                      // consumer warps
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kConsumers = kWarps * 32;
constexpr int kTileBytes = 32 * 1024;          // of K, and of V

struct TreeArgs {
  CacheGeometry g;
  int Hq, G;
  int max_tokens;
  int rows;               // rows per M-tile unit
  int tile;               // keys per tile
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
// Tiles of the keys of request r, and M-tile units per KV head (0 for a request
// that is empty, or rejected).
__device__ __forceinline__ void request_tiles(const TreeArgs& a, int r, int& off, int& n, int& kv, int& nt, int& nm) {
  nt = nm = 0;
  if (!cache_span(a.g, r, off, n, kv)) return;
  if (n > a.max_tokens) {
    atomicOr(a.g.status, FP_DEV_BAD_SEQLENS);
    n = 0;
  }
  if (n == 0) return;
  nt = (kv + a.tile - 1) / a.tile;
  nm = (n * a.G + a.rows - 1) / a.rows;
}

// Exclusive prefix of the requests' tile counts into pre[0 .. R] (all threads of
// the block; `warp_sum` has one int per warp). The host bounds the total by INT_MAX.
__device__ __forceinline__ void prefix_tiles(const TreeArgs& a, int* pre, int* warp_sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int carry = 0;
  for (int r0 = 0; r0 < a.g.R; r0 += blockDim.x) {
    const int r = r0 + threadIdx.x;
    int mine = 0;
    if (r < a.g.R) {
      int off, n, kv, nt, nm;
      request_tiles(a, r, off, n, kv, nt, nm);
      mine = nt * nm * a.g.Hkv;
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int before = carry, all = 0;
    for (int w = 0; w < warps; ++w) {
      if (w < warp) before += warp_sum[w];
      all += warp_sum[w];
    }
    if (r < a.g.R) pre[r] = before + incl - mine;
    carry += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) pre[a.g.R] = carry;
  __syncthreads();
}

// The request whose tiles hold tile x (0 <= x < pre[R]).
__device__ __forceinline__ int request_of(const int* pre, int R, int x) {
  int lo = 0, hi = R - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid + 1] > x) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

__device__ __forceinline__ int share_of(int total, int grid) { return (total + grid - 1) / grid; }

// One run of tiles of one unit within a CTA's share.
struct Segment {
  int r, off, n, kv, base;
  int head, row0;    // KV head, first row of the M-tile
  int t0, t1, nt;    // tiles t0 .. t1 - 1 of nt
  __device__ __forceinline__ bool whole() const { return t1 - t0 == nt; }
};

__device__ __forceinline__ Segment segment_at(const TreeArgs& a, const int* pre, int x, int end, int& r) {
  while (pre[r + 1] <= x) ++r;
  Segment s;
  int nm;
  s.r = r;
  request_tiles(a, r, s.off, s.n, s.kv, s.nt, nm);
  s.base = s.kv - s.n;
  const int y = x - pre[r];
  const int unit = y / s.nt;
  s.t0 = y - unit * s.nt;
  s.t1 = min(s.nt, s.t0 + (end - x));
  s.head = unit / nm;
  s.row0 = (unit - s.head * nm) * a.rows;
  return s;
}

// ---------------------------------------------------------------------------
// fragments
// ---------------------------------------------------------------------------
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int OFF>
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4 + %5];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr), "n"(OFF));
}
template <int OFF>
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4 + %5];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr), "n"(OFF));
}

// c += A (16 x 16, row) * B (16 x 8, col), float32 accumulators
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  } else {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
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

template <bool E4M3, int D>
struct Cfg {
  static constexpr int ES = E4M3 ? 1 : 2;
  static constexpr int TILE = kTileBytes / (D * ES);     // keys per tile: 128 or 256
  static constexpr int CHUNKS = D * ES / 128;            // 128-byte chunks of a row
  static constexpr int CH_ELEMS = 128 / ES;
  static constexpr int CHUNK = TILE * 128;               // bytes of a tile's chunk
  static constexpr int SLOT = kTileBytes + (E4M3 ? 1024 : 0);  // + the tile's token scales
  static constexpr int RED = 4 * 16 * D * 4;             // four key groups' O of 16 rows
  static constexpr int SLOTS = 5;
  static constexpr int SMEM_FIXED = 1024 + SLOTS * SLOT + RED + 2 * kWarps * 16 * 4 + 2 * SLOTS * 8 + 64;
  static_assert(D * ES % 128 == 0, "head dim 128, or 64 with bf16");
  static_assert(SMEM_FIXED + 4097 * 4 <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory"); }

// Infinities and NaN that new tokens of this segment hold in four columns of V
// reach the rows that see them (rare: they entered the products as zeros).
template <bool E4M3, bool TOKEN, int D>
__device__ __noinline__ void add_odd_values(const TreeArgs& a, const Segment& sg, int t, int d, int tile, float4& acc) {
  const CacheGeometry& g = a.g;
  const int32_t* row = g.table + (long long)sg.r * g.max_pages;
  for (int pos = max(sg.base, sg.t0 * tile); pos < min(sg.kv, sg.t1 * tile); ++pos) {
    const int j = pos - sg.base;
    const bool see = a.mask ? (__ldg(a.mask + (long long)(sg.off + t) * a.mask_words + (j >> 5)) >> (j & 31)) & 1u : j <= t;
    const int page = __ldg(row + (pos >> g.page_shift));
    if (!see || page < 0 || page >= g.num_pages) continue;
    const long long slot = ((long long)page << g.page_shift) + (pos & (g.page_size - 1));
    const long long at = (slot * g.Hkv + sg.head) * D + d;
    float v[4];
    if constexpr (E4M3) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(g.v_pool + at);
      float sc = 1.f;
      if (TOKEN) sc = __ldg(g.v_scale + (((long long)page * g.Hkv + sg.head) << g.page_shift) + (pos & (g.page_size - 1)));
      const __half2_raw lo = {(unsigned short)widen_lo(w), (unsigned short)(widen_lo(w) >> 16)};
      const __half2_raw hi = {(unsigned short)widen_hi(w), (unsigned short)(widen_hi(w) >> 16)};
      const float2 x = __half22float2(__half2(lo)), y = __half22float2(__half2(hi));
      v[0] = x.x * sc, v[1] = x.y * sc, v[2] = y.x * sc, v[3] = y.y * sc;
    } else {
      const uint2 w = *reinterpret_cast<const uint2*>(g.v_pool + at * 2);
      v[0] = __uint_as_float(w.x << 16), v[1] = __uint_as_float(w.x & 0xffff0000u);
      v[2] = __uint_as_float(w.y << 16), v[3] = __uint_as_float(w.y & 0xffff0000u);
    }
    if (!isfinite(v[0])) acc.x += v[0];
    if (!isfinite(v[1])) acc.y += v[1];
    if (!isfinite(v[2])) acc.z += v[2];
    if (!isfinite(v[3])) acc.w += v[3];
  }
}

// E4M3: cache type; TOKEN: token scales; WM: M-tiles of 16 rows held by the CTA
// (8 / WM warps split the keys of each).
template <bool E4M3, bool TOKEN, int D, int WM>
__global__ void __launch_bounds__(kThreads, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const TreeArgs a) {
  using C = Cfg<E4M3, D>;
  constexpr int KG = kWarps / WM;        // key groups
  constexpr int STEPS_ALL = C::TILE / KG / 16;         // 16-key steps per warp and tile,
  constexpr int STEPS = STEPS_ALL < 2 ? STEPS_ALL : 2;  // of which so many share a softmax update
  constexpr int NT = D / 8;              // 8-column tiles of O
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* red = reinterpret_cast<float*>(ring + C::SLOTS * C::SLOT);
  float* s_m = red + C::RED / 4;               // [warp][16]
  float* s_l = s_m + kWarps * 16;
  uint64_t* full = reinterpret_cast<uint64_t*>(s_l + kWarps * 16);
  uint64_t* empty = full + C::SLOTS;
  int* misc = reinterpret_cast<int*>(empty + C::SLOTS);
  volatile int* abort_flag = misc;
  int* warp_sum = misc + 1;                     // [9]
  volatile int* s_odd = misc + 10;              // [2], by segment parity: see below
  int* pre = misc + 16;                         // [R + 1]

  const CacheGeometry& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the combining kernel may be scheduled; it waits for this one's results
  asm volatile("griddepcontrol.launch_dependents;");
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::SLOTS; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, kWarps);
    }
    *abort_flag = 0;
    s_odd[0] = s_odd[1] = 0;
    fence_barrier_init();
  }
  prefix_tiles(a, pre, warp_sum);  // (its barriers publish the initialisation above)
  const int total = pre[g.R];
  const int share = share_of(total, a.grid);
  const long long x_first = (long long)blockIdx.x * share;
  if (x_first >= total) return;
  const int x_begin = (int)x_first, x_end = min(total, x_begin + share);

  if (warp == kWarps) {
    // ---------------------------------------------------------------- producer
    if (lane == 0) {
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
    const int sub_rows = min(g.page_size, C::TILE);
    const int sub_max = C::TILE / sub_rows;  // <= 16
    int slot = 0, issued = 0;
    uint32_t phase = 0;
    bool ok = true;
    int r = request_of(pre, g.R, x_begin);
    for (int x = x_begin; x < x_end && ok;) {
      const Segment sg = segment_at(a, pre, x, x_end, r);
      const int32_t* row = g.table + (long long)sg.r * g.max_pages;
      auto page_at = [&](int tile) {  // the page of this lane's part of a tile
        const int tok = tile * C::TILE + lane * sub_rows;
        return (lane < sub_max && tok < sg.kv) ? __ldg(row + (tok >> g.page_shift)) : -1;
      };
      int next_page = page_at(sg.t0);
      for (int t = sg.t0; t < sg.t1 && ok; ++t) {
        int page = next_page;
        if (t + 1 < sg.t1) next_page = page_at(t + 1);
        const int tok = t * C::TILE + lane * sub_rows;
        const bool mine = lane < sub_max && tok < sg.kv;
        const int subs = min(sub_max, (sg.kv - t * C::TILE + sub_rows - 1) / sub_rows);
        bool bad = mine && (page < 0 || page >= g.num_pages);
        if (bad) {
          atomicOr(g.status, FP_DEV_BAD_PAGE);
          page = g.num_pages;  // outside the pool: the copy fills zeros
        }
        const int at = tok & (g.page_size - 1);
#pragma unroll
        for (int which = 0; which < 2; ++which) {
          ok = mbar_wait<true>(empty + slot, phase ^ 1u, abort_flag, g.status, FP_DEV_TIMEOUT);
          if (!ok) break;
          uint8_t* dst = ring + slot * C::SLOT;
          const CUtensorMap* map = which ? &tmV : &tmK;
          if (lane == 0) {
            uint32_t bytes = (uint32_t)(subs * sub_rows) * (D * C::ES);
            if (TOKEN) bytes += (uint32_t)(subs * sub_rows) * 4u;
            mbar_arrive_expect_tx(full + slot, bytes);
          }
          __syncwarp();
          if (mine) {
#pragma unroll
            for (int ch = 0; ch < C::CHUNKS; ++ch)
              tma_load_4d(dst + ch * C::CHUNK + lane * sub_rows * 128, map, full + slot, ch * C::CH_ELEMS, sg.head, at,
                          page);
            if (TOKEN) {
              const float* sc = which ? g.v_scale : g.k_scale;
              const long long pg = bad ? 0 : page;  // (a bad page's codes are zeros: any scale does)
              bulk_load(dst + kTileBytes + lane * sub_rows * 4,
                        sc + ((pg * g.Hkv + sg.head) << g.page_shift) + at, (uint32_t)sub_rows * 4u, full + slot);
            }
          }
          ++issued;
          if (++slot == C::SLOTS) {
            slot = 0;
            phase ^= 1u;
          }
        }
      }
      x += sg.t1 - sg.t0;
    }
    // every copy lands before the CTA's shared memory is released
    if (lane == 0) {
      for (int k = 0; k < min(issued, C::SLOTS); ++k) {
        const int i = issued - 1 - k;
        mbar_drain(full + i % C::SLOTS, (uint32_t)((i / C::SLOTS) & 1), g.status, FP_DEV_TIMEOUT);
      }
    }
    return;
  }

  // ------------------------------------------------------------------ consumers
  const int mt = warp / KG, kg = warp % KG;
  const int gr = lane >> 2, c = lane & 3;  // fragment row and column group
  // ldmatrix addresses relative to a slot: slots are 1024-aligned, so the
  // 128-byte swizzle of granule 2 i + hi of row `key` is an exclusive or with i << 5
  uint32_t k_lane, v_lane;
  {
    const int kk = ((lane >> 4) << 3) + (lane & 7), khi = (lane >> 3) & 1;   // K: lanes 16-31 hold keys 8-15
    const int vk = (((lane >> 3) & 1) << 3) + (lane & 7), vhi = lane >> 4;  // V: lanes 8-15 and 24-31 do
    k_lane = smem_u32(ring) + (kg * STEPS_ALL * 16 + kk) * 128 + (((khi ^ kk) & 7) << 4);
    v_lane = smem_u32(ring) + (kg * STEPS_ALL * 16 + vk) * 128 + (((vhi ^ vk) & 7) << 4);
  }
  int slot = 0;
  uint32_t phase = 0;
  bool ok = true;
  int r = request_of(pre, g.R, x_begin);
  int segment = 0;
  for (int x = x_begin; x < x_end; ++segment) {
    const Segment sg = segment_at(a, pre, x, x_end, r);
    x += sg.t1 - sg.t0;
    const int nrows = sg.n * a.G;
    // ---- this thread's two rows of Q, as A fragments
    int rho[2], tok[2];
    bool in[2];
    uint32_t qf[D / 16][4];
    float sl2[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      rho[i] = sg.row0 + mt * 16 + gr + 8 * i;
      in[i] = rho[i] < nrows;
      const int t = in[i] ? rho[i] / a.G : 0;
      const int h = in[i] ? rho[i] - t * a.G : 0;
      tok[i] = t;
      const __nv_bfloat16* qp = a.q + (long long)(sg.off + t) * a.q_stride + (sg.head * a.G + h) * D;
      sl2[i] = a.scale_log2;
      if constexpr (!E4M3) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          qf[ks][i] = in[i] ? __ldg(reinterpret_cast<const uint32_t*>(qp + ks * 16 + 2 * c)) : 0u;
          qf[ks][2 + i] = in[i] ? __ldg(reinterpret_cast<const uint32_t*>(qp + ks * 16 + 8 + 2 * c)) : 0u;
        }
      } else {
        // four consecutive elements per 16: the order in which a thread finds K's bytes
        uint2 w[D / 16];
        float mx = 0.f;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          w[ks] = in[i] ? __ldg(reinterpret_cast<const uint2*>(qp + ks * 16 + 4 * c)) : make_uint2(0, 0);
          mx = fmaxf(mx, fmaxf(fmaxf(fabsf(__uint_as_float(w[ks].x << 16)), fabsf(__uint_as_float(w[ks].x & 0xffff0000u))),
                               fmaxf(fabsf(__uint_as_float(w[ks].y << 16)), fabsf(__uint_as_float(w[ks].y & 0xffff0000u)))));
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        // multiply by 2^(14 - floor(log2 max)); rows of zeros, infinities or below 2^-100 take the limits
        int e = (int)((__float_as_uint(mx) >> 23) & 255u) - 127;
        e = mx == 0.f || e > 127 ? 14 : max(e, -100);
        const float up = __uint_as_float((uint32_t)(14 - e + 127) << 23);
        sl2[i] *= __uint_as_float((uint32_t)(e - 14 + 127) << 23);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          qf[ks][i] = pack2<true>(__uint_as_float(w[ks].x << 16) * up, __uint_as_float(w[ks].x & 0xffff0000u) * up);
          qf[ks][2 + i] = pack2<true>(__uint_as_float(w[ks].y << 16) * up, __uint_as_float(w[ks].y & 0xffff0000u) * up);
        }
      }
    }
    float v_mul = 1.f;  // what O is multiplied by at the end
    if (E4M3 && !TOKEN) {
      const float ks = __ldg(g.k_scale + sg.head);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        sl2[i] *= ks;
        if (sl2[i] == 0.f) sl2[i] = 1.2e-38f;  // (0 * -inf of a masked key would be NaN)
      }
      v_mul = __ldg(g.v_scale + sg.head);
    }

    float o[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    // m: running maximum of the unscaled scores; ref = m * sl2 rounded, the exponents' reference
    float m[2] = {-INFINITY, -INFINITY}, ref[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    uint32_t v_exp = 0;  // token scales: exponent field of the power of two above the largest v_scale so far

    auto row_sees = [&](int i, int j) -> bool {  // row rho[i], new token j
      return a.mask ? (__ldg(a.mask + (long long)(sg.off + tok[i]) * a.mask_words + (j >> 5)) >> (j & 31)) & 1u
                    : j <= tok[i];
    };

    // STEPS steps of 16 keys of one tile: first position pos0, first key k0 of the
    // tile; SPECIAL: some are new tokens, or slots behind the last one.
    auto update = [&](auto special, int pos0, int k0, uint32_t ka, uint32_t va, const float* ksc, const float* vsc,
                      uint64_t* vfull, uint32_t vphase) {
      constexpr bool SPECIAL = decltype(special)::value;
      float s[STEPS][2][4];
#pragma unroll
      for (int st = 0; st < STEPS; ++st) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[st][0][e] = s[st][1][e] = 0.f;
        const uint32_t rowa = ka + st * (16 * 128);
        if constexpr (!E4M3) {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            uint32_t b[4];
            if (ks < 4) ldsm4<0>(b, rowa ^ ((ks & 3) << 5));
            else ldsm4<C::CHUNK>(b, rowa ^ ((ks & 3) << 5));
            mma16816<false>(s[st][0], qf[ks], b[0], b[1]);
            mma16816<false>(s[st][1], qf[ks], b[2], b[3]);
          }
        } else {
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk) {
            uint32_t b[4];  // (keys 0-7, granules 2kk and 2kk + 1), (keys 8-15, the same)
            ldsm4<0>(b, rowa ^ (kk << 5));
            mma16816<true>(s[st][0], qf[2 * kk], widen_lo(b[0]), widen_hi(b[0]));
            mma16816<true>(s[st][1], qf[2 * kk], widen_lo(b[2]), widen_hi(b[2]));
            mma16816<true>(s[st][0], qf[2 * kk + 1], widen_lo(b[1]), widen_hi(b[1]));
            mma16816<true>(s[st][1], qf[2 * kk + 1], widen_lo(b[3]), widen_hi(b[3]));
          }
        }
      }
      // this thread's keys are 16 st + 8 nt + 2c + {0, 1} (elements 0, 1: row gr; 2, 3: row gr + 8)
      uint32_t vm[STEPS][2];  // V rows that enter the product, as masks of key pairs
      float mx[2] = {m[0], m[1]};
#pragma unroll
      for (int st = 0; st < STEPS; ++st)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          if constexpr (TOKEN) {
            const float2 kf = *reinterpret_cast<const float2*>(ksc + k0 + st * 16 + nt * 8 + 2 * c);
#pragma unroll
            for (int e = 0; e < 4; ++e) s[st][nt][e] *= (e & 1) ? kf.y : kf.x;
          }
          if constexpr (SPECIAL) {
            vm[st][nt] = 0xffffffffu;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int pos = pos0 + st * 16 + nt * 8 + 2 * c + e;
              const int j = pos - sg.base;
              if (pos >= sg.kv) vm[st][nt] &= e ? 0x0000ffffu : 0xffff0000u;
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                bool see = j < 0;
                if (j >= 0 && j < sg.n && in[i]) see = row_sees(i, j);
                if (!see) s[st][nt][2 * i + e] = -INFINITY;
              }
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e >> 1] = fmaxf(mx[e >> 1], s[st][nt][e]);
        }

      // ---- softmax
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
      }
      if (__any_sync(0xffffffffu, mx[0] > m[0] || mx[1] > m[1])) {
        float f[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float nref = mx[i] * sl2[i];
          f[i] = mx[i] > m[i] ? exp2_fast(ref[i] - nref) : 1.f;
          if (mx[i] > m[i]) {
            m[i] = mx[i];
            ref[i] = nref;
          }
          l[i] *= f[i];
        }
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][e] *= f[e >> 1];
      }
      // weights relative to the running maximum; f16 ones to 2^14 above it
      float neg[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) neg[i] = ref[i] == -INFINITY ? 0.f : (E4M3 ? 14.f - ref[i] : -ref[i]);

      if (ok) ok = mbar_wait<true>(vfull, vphase, abort_flag, g.status, FP_DEV_TIMEOUT);
      float inv_ref = 1.f;
      if constexpr (TOKEN) {
        // the largest v_scale of these keys (scales are not negative: they compare as integers)
        uint32_t top = 0;
        if (STEPS == 2 || lane < 16) top = __float_as_uint(vsc[k0 + lane]);
        if constexpr (SPECIAL) {  // not those of slots behind the last token, or of new tokens without a finite one
          const int pos = pos0 + lane;
          if (pos >= sg.kv || (pos >= sg.base && top >= 0x7f800000u)) top = 0;
        }
        top = __reduce_max_sync(0xffffffffu, top);
        // the next power of two above it, within 2^-100 .. 2^127
        const uint32_t need = top == 0 ? 0 : min(max((top >> 23) + 1u, 27u), 254u);
        if (need > v_exp) {  // (the whole warp agrees)
          if (v_exp != 0) {
            const float k = exp2_fast((float)((int)v_exp - (int)need));
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[i][e] *= k;
          }
          v_exp = need;
        }
        // 2^-(v_exp - 127); where every scale so far was zero it does not matter
        inv_ref = __uint_as_float((v_exp == 254u ? 1u : 254u - max(v_exp, 27u)) << 23);
        if (v_exp == 254u) inv_ref *= 0.5f;
      }
      uint32_t pf[STEPS][4], pl[STEPS][4];
      bool odd = false;  // a new token's V or scale is an infinity or NaN
#pragma unroll
      for (int st = 0; st < STEPS; ++st)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          float2 vf = make_float2(1.f, 1.f);
          if constexpr (TOKEN) {
            vf = *reinterpret_cast<const float2*>(vsc + k0 + st * 16 + nt * 8 + 2 * c);
            if constexpr (SPECIAL) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float& y = e ? vf.y : vf.x;
                const int pos = pos0 + st * 16 + nt * 8 + 2 * c + e;
                if (pos >= sg.base && !(y < INFINITY)) {
                  odd |= pos < sg.kv;
                  y = 0.f;
                }
              }
            }
            vf.x *= inv_ref;
            vf.y *= inv_ref;
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float p0 = exp2_fast(fmaf(s[st][nt][2 * i], sl2[i], neg[i]));
            float p1 = exp2_fast(fmaf(s[st][nt][2 * i + 1], sl2[i], neg[i]));
            l[i] += p0 + p1;
            if constexpr (TOKEN) {
              p0 *= vf.x;
              p1 *= vf.y;
            }
            const uint32_t u = pack2<E4M3>(p0, p1);
            pf[st][2 * nt + i] = u;
            if (!E4M3) pl[st][2 * nt + i] = pack_rest(p0, p1, u);
          }
        }
      // ---- O += P V
#pragma unroll
      for (int st = 0; st < STEPS; ++st) {
        const uint32_t rowa = va + st * (16 * 128);
#pragma unroll
        for (int dt = 0; dt < D / 16; dt += E4M3 ? 2 : 1) {  // (two granules per load)
          uint32_t b[4];
          if constexpr (E4M3) ldsm4_t<0>(b, rowa ^ (dt << 4));
          else if (dt < 4) ldsm4_t<0>(b, rowa ^ ((dt & 3) << 5));
          else ldsm4_t<C::CHUNK>(b, rowa ^ ((dt & 3) << 5));
          if constexpr (SPECIAL) {
            // slots behind the last token hold anything: they enter as zeros; so do the
            // infinities and NaN of new tokens, which only some rows see (added at the end)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              b[e] &= vm[st][e & 1];
              const int j = pos0 + st * 16 + (e & 1) * 8 + 2 * c - sg.base;  // of the pair's first key
              uint32_t keep = 0xffffffffu;
              if constexpr (!E4M3) {
                if (j >= 0 && (b[e] & 0x00007f80u) == 0x00007f80u) keep &= 0xffff0000u;
                if (j + 1 >= 0 && (b[e] & 0x7f800000u) == 0x7f800000u) keep &= 0x0000ffffu;
              } else {
                if (j >= 0 && (b[e] & 0x0000007fu) == 0x0000007fu) keep &= 0xffffff00u;
                if (j >= 0 && (b[e] & 0x00007f00u) == 0x00007f00u) keep &= 0xffff00ffu;
                if (j + 1 >= 0 && (b[e] & 0x007f0000u) == 0x007f0000u) keep &= 0xff00ffffu;
                if (j + 1 >= 0 && (b[e] & 0x7f000000u) == 0x7f000000u) keep &= 0x00ffffffu;
              }
              odd |= keep != 0xffffffffu;
              b[e] &= keep;
            }
          }
          if constexpr (!E4M3) {
            mma16816<false>(o[2 * dt], pf[st], b[0], b[1]);
            mma16816<false>(o[2 * dt + 1], pf[st], b[2], b[3]);
            mma16816<false>(o[2 * dt], pl[st], b[0], b[1]);
            mma16816<false>(o[2 * dt + 1], pl[st], b[2], b[3]);
          } else {
            // bytes (key 2c: d, d + 1), (key 2c + 1: d, d + 1) -> the even d's pair, the odd d's pair
            const uint32_t e0 = __byte_perm(b[0], 0, 0x3120), e1 = __byte_perm(b[1], 0, 0x3120);
            const uint32_t e2 = __byte_perm(b[2], 0, 0x3120), e3 = __byte_perm(b[3], 0, 0x3120);
            mma16816<true>(o[2 * dt], pf[st], widen_lo(e0), widen_lo(e1));
            mma16816<true>(o[2 * dt + 1], pf[st], widen_hi(e0), widen_hi(e1));
            mma16816<true>(o[2 * dt + 2], pf[st], widen_lo(e2), widen_lo(e3));
            mma16816<true>(o[2 * dt + 3], pf[st], widen_hi(e2), widen_hi(e3));
          }
        }
      }
      if constexpr (SPECIAL) {
        if (odd) s_odd[segment & 1] = 1;
      }
    };

    for (int t = sg.t0; t < sg.t1; ++t) {
      const int kslot = slot, vslot = slot + 1 == C::SLOTS ? 0 : slot + 1;
      const uint32_t kphase = phase, vphase = vslot == 0 ? phase ^ 1u : phase;
      slot = vslot + 1 == C::SLOTS ? 0 : vslot + 1;
      phase = slot == 0 ? vphase ^ 1u : vphase;
      if (ok) ok = mbar_wait<true>(full + kslot, kphase, abort_flag, g.status, FP_DEV_TIMEOUT);
      const float* ksc = reinterpret_cast<const float*>(ring + kslot * C::SLOT + kTileBytes);
      const float* vsc = reinterpret_cast<const float*>(ring + vslot * C::SLOT + kTileBytes);
#pragma unroll 1
      for (int st = 0; st < STEPS_ALL; st += STEPS) {
        const int k0 = (kg * STEPS_ALL + st) * 16;
        const uint32_t ka = k_lane + kslot * C::SLOT + st * (16 * 128), va = v_lane + vslot * C::SLOT + st * (16 * 128);
        if (t * C::TILE + k0 + STEPS * 16 > sg.base)
          update(std::true_type(), t * C::TILE + k0, k0, ka, va, ksc, vsc, full + vslot, vphase);
        else
          update(std::false_type(), t * C::TILE + k0, k0, ka, va, ksc, vsc, full + vslot, vphase);
      }
      __syncwarp();
      if (ok && lane == 0) {
        mbar_arrive(empty + kslot);
        mbar_arrive(empty + vslot);
      }
    }

    // ---- the key groups' results meet
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      if (c == 0) {
        s_m[warp * 16 + gr + 8 * i] = ref[i];
        s_l[warp * 16 + gr + 8 * i] = l[i];
      }
    }
    if (TOKEN) v_mul = v_exp == 0 ? 0.f : __uint_as_float(v_exp << 23);
    consumers_sync();
    if (threadIdx.x == 0) s_odd[(segment + 1) & 1] = 0;  // (its readers have passed the barrier above)
    float big[2], sum[2], w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float* pm = s_m + mt * KG * 16 + gr + 8 * i;
      const float* pl2 = s_l + mt * KG * 16 + gr + 8 * i;
      big[i] = -INFINITY;
      for (int k = 0; k < KG; ++k) big[i] = fmaxf(big[i], pm[k * 16]);
      sum[i] = 0.f;
      // (a group that saw nothing has m = -inf and l = 0; l may be NaN without a maximum)
      for (int k = 0; k < KG; ++k) sum[i] += pl2[k * 16] * (big[i] == -INFINITY ? 1.f : exp2_fast(pm[k * 16] - big[i]));
      w[i] = big[i] == -INFINITY ? 1.f : exp2_fast(ref[i] - big[i]);
      w[i] = sum[i] == 0.f ? 0.f : w[i] * v_mul / sum[i];
    }
#pragma unroll
    for (int q = 0; q < NT; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[q][e] = w[e >> 1] == 0.f ? 0.f : o[q][e] * w[e >> 1];
    // sum over the key groups: the upper half adds to the lower through `red`, then all threads add what is left
    constexpr int HALF = kWarps / 2;
    auto red_at = [&](int buf, int q, int i, int e) -> float* {
      const int d = E4M3 ? (q >> 1) * 16 + 4 * c + 2 * e + (q & 1) : q * 8 + 2 * c + e;
      return red + (buf * 16 + gr + 8 * i) * D + d;
    };
    // pairs (mt, kg) and (mt, kg + KG / 2) share a buffer
    const bool upper = kg >= KG / 2;
    const int buf = mt * (KG / 2) + (upper ? kg - KG / 2 : kg);
    static_assert(WM * (KG / 2) == HALF, "four buffers");
    if (upper) {
#pragma unroll
      for (int q = 0; q < NT; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) *red_at(buf, q, e >> 1, e & 1) = o[q][e];
    }
    consumers_sync();
    if (!upper) {
#pragma unroll
      for (int q = 0; q < NT; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float* p = red_at(buf, q, e >> 1, e & 1);
          *p += o[q][e];
        }
    }
    consumers_sync();
    const bool whole = sg.whole();
    const int part = 2 * blockIdx.x + (segment == 0 ? 0 : 1);
    const bool odd = s_odd[segment & 1] != 0;
    for (int i = threadIdx.x; i < WM * 16 * (D / 4); i += kConsumers) {
      const int lr = i / (D / 4), d4 = i % (D / 4);  // row of the M-tiles, four columns
      const int row = sg.row0 + lr;
      if (row >= nrows) continue;
      const float* src = red + (((lr >> 4) * (KG / 2)) * 16 + (lr & 15)) * D + d4 * 4;
      float4 acc = *reinterpret_cast<const float4*>(src);
#pragma unroll
      for (int k = 1; k < KG / 2; ++k) {
        const float4 y = *reinterpret_cast<const float4*>(src + k * 16 * D);
        acc.x += y.x;
        acc.y += y.y;
        acc.z += y.z;
        acc.w += y.w;
      }
      if (odd) add_odd_values<E4M3, TOKEN, D>(a, sg, row / a.G, d4 * 4, C::TILE, acc);
      if (whole) {
        const int t = row / a.G, h = row - t * a.G;
        uint2 pk = make_uint2(pack2<false>(acc.x, acc.y), pack2<false>(acc.z, acc.w));
        *reinterpret_cast<uint2*>(a.o + ((long long)(sg.off + t) * a.Hq + sg.head * a.G + h) * D + d4 * 4) = pk;
      } else {
        *reinterpret_cast<float4*>(a.part_o + ((long long)part * a.rows + lr) * D + d4 * 4) = acc;
      }
    }
    if (kg == 0 && c == 0) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (!in[i]) continue;
        // the weights' 2^14 (e4m3) comes off the logarithm
        const float lse2 = sum[i] == 0.f ? -INFINITY
                                         : (big[i] == -INFINITY ? 0.f : big[i]) + log2f(sum[i]) - (E4M3 ? 14.f : 0.f);
        if (!whole) {
          a.part_lse[(long long)part * a.rows + mt * 16 + gr + 8 * i] = lse2;
        } else if (a.lse) {
          const int h = rho[i] - tok[i] * a.G;
          a.lse[(long long)(sg.head * a.G + h) * g.total_tokens + sg.off + tok[i]] = lse2 * 0.69314718055994531f;
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// combining partial rows
// ---------------------------------------------------------------------------
constexpr int kMergeThreads = 128;

// One CTA per (token, query head) row: the partial rows its unit left in the
// workspace, in CTA order; its four warps take every fourth one.
template <int D>
__global__ void __launch_bounds__(kMergeThreads) tree_merge_kernel(const TreeArgs a) {
  extern __shared__ int pre[];  // [R + 1]
  __shared__ int warp_sum[kMergeThreads / 32];
  __shared__ float acc[kMergeThreads / 32][D];
  constexpr int PER = D / 32;   // columns per lane
  const CacheGeometry& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int token = blockIdx.x / a.Hq, hq = blockIdx.x % a.Hq;
  prefix_tiles(a, pre, warp_sum);
  const int total = pre[g.R];
  // the request of this token
  int lo = 0, hi = g.R - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(g.cu + mid + 1) > token) hi = mid;
    else lo = mid + 1;
  }
  int off, n, kv, nt, nm;
  request_tiles(a, lo, off, n, kv, nt, nm);
  // every thread waits, also those with nothing to do: this grid is not to end
  // before the one that it depends on
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (nt == 0 || token < off || token >= off + n) return;
  const int row = (token - off) * a.G + hq % a.G, head = hq / a.G;
  const int x0 = pre[lo] + (head * nm + row / a.rows) * nt, x1 = x0 + nt;
  const int share = share_of(total, a.grid);
  const int c0 = x0 / share, c1 = (x1 - 1) / share;
  if (c0 == c1) return;  // one CTA had the whole unit and finished it
  const int lr = row % a.rows;
  // its partial in CTA c: the CTA's first segment, unless the unit begins inside the CTA's share
  auto part = [&](int c) { return (long long)(2 * c + ((long long)c * share < x0 ? 1 : 0)) * a.rows + lr; };
  float big = -INFINITY;
  for (int c = c0 + lane; c <= c1; c += 32) big = fmaxf(big, __ldcg(a.part_lse + part(c)));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
  const float ref = big == -INFINITY ? 0.f : big;
  float sum = 0.f, v[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) v[e] = 0.f;
  for (int c = c0 + warp; c <= c1; c += kMergeThreads / 32) {
    const long long p = part(c);
    const float w = exp2_fast(__ldcg(a.part_lse + p) - ref);
    const float* src = a.part_o + p * D + lane * PER;
    float y[PER];
    if constexpr (PER == 4) {
      const float4 f = __ldcg(reinterpret_cast<const float4*>(src));
      y[0] = f.x, y[1] = f.y, y[2] = f.z, y[3] = f.w;
    } else {
      const float2 f = __ldcg(reinterpret_cast<const float2*>(src));
      y[0] = f.x, y[1] = f.y;
    }
    sum += w;
#pragma unroll
    for (int e = 0; e < PER; ++e) v[e] += w == 0.f ? 0.f : w * y[e];
  }
  __shared__ float sums[kMergeThreads / 32];
#pragma unroll
  for (int e = 0; e < PER; ++e) acc[warp][lane * PER + e] = v[e];
  if (lane == 0) sums[warp] = sum;
  __syncthreads();
  sum = (sums[0] + sums[1]) + (sums[2] + sums[3]);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  for (int d = threadIdx.x; d < D; d += kMergeThreads)
    a.o[((long long)token * a.Hq + hq) * D + d] =
        __float2bfloat16_rn(((acc[0][d] + acc[1][d]) + (acc[2][d] + acc[3][d])) * inv);
  if (a.lse && threadIdx.x == 0)
    a.lse[(long long)hq * g.total_tokens + token] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.69314718055994531f;
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 148;
  return n;
}

int unit_rows(int max_rows) { return max_rows <= 16 ? 16 : 32; }

template <bool E4M3, bool TOKEN, int D, int WM>
cudaError_t run(const TreeArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t s) {
  using C = Cfg<E4M3, D>;
  auto kern = tree_kernel<E4M3, TOKEN, D, WM>;
  const int smem = C::SMEM_FIXED + (a.g.R + 1) * 4;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<a.grid, kThreads, smem, s>>>(mk, mv, a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)a.g.total_tokens * a.Hq));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.dynamicSmemBytes = (size_t)(a.g.R + 1) * 4;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_merge_kernel<D>, a);
}

template <bool E4M3, bool TOKEN, int D>
cudaError_t run_rows(const TreeArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t s) {
  return a.rows == 16 ? run<E4M3, TOKEN, D, 1>(a, mk, mv, s) : run<E4M3, TOKEN, D, 2>(a, mk, mv, s);
}

size_t pad256(size_t bytes) { return (bytes + 255) / 256 * 256; }

}  // namespace

// Two partial units per CTA: float32 O rows, then their logarithms.
size_t tree_workspace(const CacheGeometry& g, int hq, int max_tokens) {
  const size_t rows = (size_t)2 * sm_count() * unit_rows(max_tokens * (hq / g.Hkv));
  return pad256(rows * g.d * sizeof(float)) + pad256(rows * sizeof(float));
}

fp_status_t launch_tree(const CacheGeometry& g, const fp_tree_t& t, const void* q, void* o, float* lse, void* ws,
                        cudaStream_t s) {
  TreeArgs a;
  a.g = g;
  a.Hq = t.hq;
  a.G = t.hq / g.Hkv;
  a.max_tokens = t.max_tokens;
  a.rows = unit_rows(t.max_tokens * a.G);
  a.mask = t.mask;
  a.mask_words = t.mask_words;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.q_stride = t.q_stride ? t.q_stride : (long long)t.hq * g.d;
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  const double scale = t.softmax_scale > 0.f ? (double)t.softmax_scale : 1.0 / std::sqrt((double)g.d);
  a.scale_log2 = (float)(scale * 1.4426950408889634);
  a.grid = sm_count();
  a.tile = kTileBytes / (g.d * (g.e4m3 ? 1 : 2));
  const size_t rows = (size_t)2 * a.grid * a.rows;
  a.part_o = static_cast<float*>(ws);
  a.part_lse = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + pad256(rows * g.d * sizeof(float)));

  CUtensorMap mk, mv;
  const cuuint64_t es = g.e4m3 ? 1 : 2, P = (cuuint64_t)g.page_size;
  const cuuint64_t dims[4] = {(cuuint64_t)g.d, (cuuint64_t)g.Hkv, P, (cuuint64_t)g.num_pages};
  const cuuint64_t strides[3] = {g.d * es, (cuuint64_t)g.Hkv * g.d * es, P * g.Hkv * g.d * es};
  const cuuint32_t box[4] = {(cuuint32_t)(128 / es), 1, (cuuint32_t)(g.page_size < a.tile ? g.page_size : a.tile), 1};
  const CUtensorMapDataType type = g.e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  if (!encode_tiled(&mk, type, 4, g.k_pool, dims, strides, box) ||
      !encode_tiled(&mv, type, 4, g.v_pool, dims, strides, box))
    return FP_ERR_CUDA;
  cudaError_t e;
  if (g.e4m3) e = g.token_scale ? run_rows<true, true, 128>(a, mk, mv, s) : run_rows<true, false, 128>(a, mk, mv, s);
  else e = g.d == 128 ? run_rows<false, false, 128>(a, mk, mv, s) : run_rows<false, false, 64>(a, mk, mv, s);
  if (e != cudaSuccess) {
    set_last_error("tree attention launch", (int)e, cudaGetErrorString(e));
    return FP_ERR_CUDA;
  }
  return FP_OK;
}

}  // namespace fp
