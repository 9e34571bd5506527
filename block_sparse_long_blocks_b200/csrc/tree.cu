// Attention of a tree of drafted tokens (or of single tokens) over the paged cache.
//
// Row rho = t * G + h of a request and KV head is query head h of the group and
// new token t (PackGQA, as in the prefill). With base = kv_len - n:
//   x[rho, j] = scale * log2(e) * q[rho] . k[j]     (token-scale caches: * k_scale[j])
//   row rho sees j < base, and base + u iff bit u of its token's mask is set
//   m = max_j x, p = 2^(x - m), l = sum p, O = sum p v / l, lse = (m + log2 l) ln 2
// Online over the keys: when m grows, l and O are multiplied by 2^(m_old - m).
//
// What bounds it: every cached row is read once per unit, 4 * rows flops per
// element, so up to ~250 rows (bf16) HBM is the floor. The keys of ALL requests,
// KV heads and units form one axis of tiles (32 KB of K: 128 keys of 256 bytes,
// or 256 of 128), cut evenly over one persistent CTA per SM, however ragged the
// lengths. A unit (request, KV head, rows) that lies within one CTA's share is
// finished there; the others leave normalised partial rows (float32 O, base-2
// lse) in the workspace, at most two per CTA, which a second kernel (a
// programmatic dependent launch) combines in a fixed order:
// O = sum_i 2^(lse_i - lse) O_i.
// This file: units of 8 or 16 rows, single tokens and small trees. More rows go
// to tree_wide.cu, where tcgen05 multiplies M-tiles of 128.
// Measured, calls whose inputs change: one token each of eight requests of 4K-64K
// (bf16, 8 KV heads of 4 query heads) 177 to 183 us, 6.5 to 6.7 TB/s with everything;
// one token of 128K (e4m3 with token scales, 4 KV heads of 8) 36 us, of which 20 us
// stream at 6.8 TB/s; one token of 2K 10 us, two launches (8.8 us on the device).
//
// A CTA: warp 8 issues TMA copies of K and V tiles (4-D boxes per page, 128-byte
// swizzle, and the tile's token scales) into a ring of five 32 KB slots; warps
// 0-7 all hold the unit's rows and split the tile's keys, so no warp waits for
// another until the unit's end, where their (m, l, O) meet in shared memory.
// mma.sync and not tcgen05 here: 8 or 16 useful rows would fill a sixteenth or
// an eighth of a 128-row tcgen05 tile. S = Q K^T has the rows as M (16); the
// second product is transposed, O^T = V^T P^T, so that 8 rows are its whole N
// and the weights go from accumulators to operands within their thread.
//
// Operands: bf16 caches multiply bf16 q and k exactly, and p as bf16 hi + lo
// (two products: the weights keep 16 bits; the tensor pipe has room). e4m3
// caches: S on the e4m3 path (mma.m16n8k32 runs at 4.4 clocks a warp, half the
// f16 instruction's for twice the keys, and needs no widening; its sums were
// measured exact to 2^-22 of sum |q k|), with q * 2^e (e per row such that max |q|
// lies in [2^7, 2^8)) as hi + 2^-5 lo, two e4m3 values whose sum is q exactly for
// every element within 2^-14 of the largest, and to 2^-22 of it for others; up to
// 8 rows both fill one M tile.
// V is widened exactly to f16; p carries a factor 2^kShift into f16's normal
// range. Token scales of V multiply p, and f16 holds the product p v_scale
// relative to the row's own largest one so far (its logarithm's reference is kept
// beside the softmax's): a reference shared by the rows would let the scale of a
// key that a row does not see, or hardly weighs, push that row's weights below
// f16. It costs a multiply-add and a maximum per score.
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

#include "tree.cuh"

namespace fp {

using namespace tree;

namespace {

constexpr int kWarps = 8;                      // consumer warps
constexpr int kThreads = (kWarps + 4) * 32;    // + the producer, alone in a third warpgroup
// Registers: launched with 168 a thread (three warps per SM sub-partition); the consumers then
// take 208 and the producer's warpgroup 88: 2 x 128 x 208 + 128 x 88 = 384 x 168.
constexpr uint32_t kLaunchRegs = 168, kConsumerRegs = 208, kProducerRegs = 88;
static_assert(2 * 128 * kConsumerRegs + 128 * kProducerRegs <= kThreads * kLaunchRegs, "register split");
constexpr int kConsumers = kWarps * 32;
constexpr int kTileBytes = 32 * 1024;          // of K, and of V

// ---------------------------------------------------------------------------
// fragments
// ---------------------------------------------------------------------------
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

// 16 x 16 bytes per half-warp's addresses, transposed: r[0], r[1] hold (source rows 4c .. 4c + 3) of columns
// gr and gr + 8 of the first 16 rows, r[2], r[3] those of the second 16
__device__ __forceinline__ void ldsm2_t8(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
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
// c += A (16 x 32, row) * B (32 x 8, col), e4m3
__device__ __forceinline__ void mma16832(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <bool E4M3, int D, int NB>
struct Cfg {
  static constexpr int ES = E4M3 ? 1 : 2;
  static constexpr int TILE = kTileBytes / (D * ES);     // keys per tile: 128 or 256
  static constexpr int CHUNKS = D * ES / 128;            // 128-byte chunks of a row
  static constexpr int CH_ELEMS = 128 / ES;
  static constexpr int CHUNK = TILE * 128;               // bytes of a tile's chunk
  static constexpr int SLOT = kTileBytes + (E4M3 ? 1024 : 0);  // + the tile's token scales
  static constexpr int SLOTS = 5;
  static constexpr int ROWS = 8 * NB;
  static_assert(NB <= 2, "an A tile has 16 rows");
  static constexpr int QT = E4M3 ? NB : 1;               // 16-row A tiles of Q (e4m3: high, then low parts)
  // the warps' O meet in NB rounds of D / NB columns; rows are padded so that the fragments' stores hit 32 banks
  static constexpr int RED_COLS = D / NB, RED_ROW = RED_COLS + 4;
  static constexpr int RED = kWarps * ROWS * RED_ROW * 4;
  static_assert(QT * 16 * D * ES <= RED, "Q lies in the same place while the keys are read");
  static constexpr int SMEM_FIXED = 1024 + SLOTS * SLOT + RED + (2 * kWarps + 1) * ROWS * 4 + 2 * SLOTS * 8 + 64;
  static_assert(D * ES % 128 == 0, "head dim 128, or 64 with bf16");
  static_assert(SMEM_FIXED + kAxisBytesMax <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory"); }

// E4M3: cache type; TOKEN: token scales; NB: blocks of 8 rows held by every warp.
template <bool E4M3, bool TOKEN, int D, int NB>
__global__ void __launch_bounds__(kThreads, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                const __grid_constant__ TreeArgs a) {
  using C = Cfg<E4M3, D, NB>;
  constexpr int STEPS = C::TILE / kWarps / 16;          // 16-key blocks per warp and tile: one softmax update
  static_assert(STEPS <= 2 && (!E4M3 || STEPS == 2), "blocks of a warp");
  constexpr int KS = D * C::ES / 32;                    // 32-byte steps of a row
  constexpr int MT = D / 16;                            // 16-column tiles of O
  constexpr int QT = C::QT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* red = reinterpret_cast<float*>(ring + C::SLOTS * C::SLOT);
  uint8_t* q_smem = reinterpret_cast<uint8_t*>(red);
  float* s_m = red + C::RED / 4;               // [warp][row]
  float* s_l = s_m + kWarps * C::ROWS;
  float* s_scale = s_l + kWarps * C::ROWS;     // [row]: what a raw score is multiplied by
  uint64_t* full = reinterpret_cast<uint64_t*>(s_scale + C::ROWS);
  uint64_t* empty = full + C::SLOTS;
  int* misc = reinterpret_cast<int*>(empty + C::SLOTS);
  volatile int* abort_flag = misc;
  int* warp_sum = misc + 1;                     // [12]
  volatile int* s_odd = misc + 13;              // [2], by segment parity: see below
  Axis axis(misc + 16, a.g.R);

  const CacheGeometry& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the combining kernel may be scheduled; it waits for this one's results
  asm volatile("griddepcontrol.launch_dependents;");
  if (threadIdx.x == kWarps * 32) {  // (warp 0 has the axis to build)
    for (int s = 0; s < C::SLOTS; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, kWarps);
    }
    *abort_flag = 0;
    s_odd[0] = s_odd[1] = 0;
    fence_barrier_init();
  }
  axis.build(a, warp_sum);  // (its barrier publishes the initialisation above)
  const int total = axis.total();
  const int share = share_of(a, total);
  const long long x_first = (long long)blockIdx.x * share;
  if (x_first >= total) return;
  const int x_begin = (int)x_first, x_end = min(total, x_begin + share);

  if (warp >= kWarps) {
    reg_dealloc<kProducerRegs>();
    if (warp > kWarps) return;
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
    int r = axis.request_of(x_begin);
    for (int x = x_begin; x < x_end && ok;) {
      Segment sg;
      if (!next_segment(a, axis, x, x_end, r, sg)) continue;
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
          uint32_t bytes = (uint32_t)(subs * sub_rows) * (D * C::ES);
          if (TOKEN) bytes += scales_of_tile(reinterpret_cast<float*>(dst + kTileBytes), bad, mine, lane, sub_rows);
          if (lane == 0) mbar_arrive_expect_tx(full + slot, bytes);
          __syncwarp();
          if (mine) {
#pragma unroll
            for (int ch = 0; ch < C::CHUNKS; ++ch)
              tma_load_4d(dst + ch * C::CHUNK + lane * sub_rows * 128, map, full + slot, ch * C::CH_ELEMS, sg.head, at,
                          page);
            if (TOKEN && !bad)
              bulk_load(dst + kTileBytes + lane * sub_rows * 4,
                        (which ? g.v_scale : g.k_scale) + (((long long)page * g.Hkv + sg.head) << g.page_shift) + at,
                        (uint32_t)sub_rows * 4u, full + slot);
          }
          ++issued;
          if (++slot == C::SLOTS) {
            slot = 0;
            phase ^= 1u;
          }
        }
      }
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
  reg_alloc<kConsumerRegs>();
  const int gr = lane >> 2, c = lane & 3;  // fragment row (or column) and column group
  // Keys of a 16-key block that this thread's scores belong to: fragment column 2c + e of tile 0 and of tile 1.
  // e4m3: V's transposed load gives a thread four consecutive source rows, two of either tile; tile 1 takes key
  // 8 + (n ^ 4) as its column n so that eight rows of one load never share a bank, in K or in V.
  const int key0 = 2 * c, key1 = E4M3 ? 8 + ((2 * c) ^ 4) : 8 + 2 * c;
  // ldmatrix addresses relative to a slot: slots are 1024-aligned, so the
  // 128-byte swizzle of granule 2 i + hi of row `key` is an exclusive or with i << 5
  uint32_t k_lane, v_lane, q_lane;
  {
    const int n = lane & 7, hi = (lane >> 3) & 1;
    const int kk = lane < 16 ? n : 8 + (E4M3 ? n ^ 4 : n);  // K: lanes 16-31 hold tile 1
    k_lane = smem_u32(ring) + (warp * STEPS * 16 + kk) * 128 + (((hi ^ kk) & 7) << 4);
    int vk, vg;                                             // V: key, and granule (16 bytes) within a d tile's
    if (E4M3) {
      const int i = lane & 15, pair = 2 * (i >> 2) + (i & 1);
      vk = (i & 2) ? 8 + (pair ^ 4) : pair;
      vg = 0;
      vk += lane & 16;                                      // lanes 16-31: the next block's keys
    } else {
      vk = ((lane >> 4) << 3) + n;
      vg = hi;
    }
    v_lane = smem_u32(ring) + (warp * STEPS * 16 + vk) * 128 + (((vg ^ vk) & 7) << 4);
    const int qr = lane & 15, qh = lane >> 4;
    q_lane = smem_u32(q_smem) + qr * 128 + (((qh ^ qr) & 7) << 4);
  }
  // fragment `ks` of A tile `qt` of Q
  auto load_q = [&](uint32_t(&f)[4], int qt, int ks) {
    ldsm4<0>(f, (q_lane ^ ((ks & 3) << 5)) + (ks >> 2) * (QT * 16 * 128) + qt * (16 * 128));
  };
  int slot = 0;
  uint32_t phase = 0;
  bool ok = true;
  int r = axis.request_of(x_begin);
  int segment = 0;
  for (int x = x_begin; x < x_end;) {
    Segment sg;
    if (!next_segment(a, axis, x, x_end, r, sg)) continue;
    const int nrows = sg.n * a.G;
    // ---- Q to shared memory, as the rows of A tiles
    if constexpr (!E4M3) {
      for (int i = threadIdx.x; i < QT * 16 * (D / 8); i += kConsumers) {
        const int row = i / (D / 8), gran = i % (D / 8), rho = sg.row0 + row;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (row < C::ROWS && rho < nrows) {
          const int t = group_of(a, rho), h = rho - t * a.G;
          w = __ldg(reinterpret_cast<const uint4*>(a.q + (long long)(sg.off + t) * a.q_stride +
                                                   (sg.head * a.G + h) * D) + gran);
        }
        *reinterpret_cast<uint4*>(q_smem + (gran >> 3) * (QT * 16 * 128) + row * 128 + (((gran ^ row) & 7) << 4)) = w;
      }
      if (threadIdx.x < C::ROWS) s_scale[threadIdx.x] = a.scale_log2;
    } else {
      constexpr int TPR = 32 / NB, EL = 4 * NB;  // threads per row, elements per thread
      const int row = threadIdx.x / TPR, part = threadIdx.x % TPR, rho = sg.row0 + row;
      uint32_t w[EL / 2];
#pragma unroll
      for (int i = 0; i < EL / 2; ++i) w[i] = 0;
      if (rho < nrows) {
        const int t = group_of(a, rho), h = rho - t * a.G;
        const __nv_bfloat16* qp = a.q + (long long)(sg.off + t) * a.q_stride + (sg.head * a.G + h) * D + part * EL;
#pragma unroll
        for (int i = 0; i < EL / 4; ++i) {
          const uint2 u = __ldg(reinterpret_cast<const uint2*>(qp) + i);
          w[2 * i] = u.x;
          w[2 * i + 1] = u.y;
        }
      }
      float mx = 0.f;
#pragma unroll
      for (int i = 0; i < EL / 2; ++i)
        mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xffff0000u))));
#pragma unroll
      for (int o = TPR / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      // times 2^(7 - floor(log2 max)): the largest lies in [2^7, 2^8); rows of zeros or below 2^-100 take the limits
      const int e = mx == 0.f ? 7 : max((int)((__float_as_uint(mx) >> 23) & 255u) - 127, -100);
      const float up = mx < INFINITY ? __uint_as_float((uint32_t)(7 - e + 127) << 23) : __uint_as_float(0x7fc00000u);
      const int hi_row = row, lo_row = row + C::ROWS;
#pragma unroll
      for (int i = 0; i < EL / 4; ++i) {
        float v[4] = {__uint_as_float(w[2 * i] << 16) * up, __uint_as_float(w[2 * i] & 0xffff0000u) * up,
                      __uint_as_float(w[2 * i + 1] << 16) * up, __uint_as_float(w[2 * i + 1] & 0xffff0000u) * up};
        const uint32_t hi = pack_codes(v[0], v[1]) | (pack_codes(v[2], v[3]) << 16);
        const uint32_t h01 = widen_lo(hi), h23 = widen_hi(hi);
        const float2 f01 = __half22float2(*reinterpret_cast<const __half2*>(&h01));
        const float2 f23 = __half22float2(*reinterpret_cast<const __half2*>(&h23));
        const uint32_t lo = pack_codes((v[0] - f01.x) * 32.f, (v[1] - f01.y) * 32.f) |
                            (pack_codes((v[2] - f23.x) * 32.f, (v[3] - f23.y) * 32.f) << 16);
        const int at = part * EL + 4 * i, gran = at >> 4;
        *reinterpret_cast<uint32_t*>(q_smem + hi_row * 128 + (((gran ^ hi_row) & 7) << 4) + (at & 15)) = hi;
        *reinterpret_cast<uint32_t*>(q_smem + lo_row * 128 + (((gran ^ lo_row) & 7) << 4) + (at & 15)) = lo;
      }
      if (part == 0) {
        float f = a.scale_log2 * __uint_as_float((uint32_t)(e - 7 + 127) << 23);
        if (!TOKEN) f *= __ldg(g.k_scale + sg.head);
        if (f == 0.f) f = 1.2e-38f;  // (0 * -inf of a masked key would be NaN)
        s_scale[row] = f;
      }
    }
    consumers_sync();
    uint32_t qf[QT][KS][4];
#pragma unroll
    for (int qt = 0; qt < QT; ++qt)
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) load_q(qf[qt][ks], qt, ks);
    // this thread's rows of S: gr + 8 b
    float sl2[NB];
    int tok[NB];
    bool in[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int rho = sg.row0 + gr + 8 * b;
      in[b] = rho < nrows;
      tok[b] = in[b] ? group_of(a, rho) : 0;
      sl2[b] = s_scale[gr + 8 * b];
    }
    float v_mul = 1.f;  // what O is multiplied by at the end
    if (E4M3 && !TOKEN) v_mul = __ldg(g.v_scale + sg.head);
    // what O is relative to where that is not ref (TOKEN): a maximum of x + log2(v_scale)
    [[maybe_unused]] float vref[NB];

    float o[MT][NB][4];  // columns 16 mt + gr (elements 0, 1) and + 8 (2, 3) of rows 8 b + 2c + {0, 1}
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][b][e] = 0.f;
    // ref: the exponents' reference, the scaled maximum at its last rise
    float ref[NB], l[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      ref[b] = vref[b] = -INFINITY;
      l[b] = 0.f;
    }

    // STEPS blocks of 16 keys of one tile: first position pos0, first key k0 of the
    // tile; SPECIAL: some are new tokens, or slots behind the last one.
    auto update = [&](auto special, int pos0, int k0, uint32_t ka, uint32_t va, const float* ksc, const float* vsc,
                      uint64_t* vfull, uint32_t vphase) {
      constexpr bool SPECIAL = decltype(special)::value;
      float s[STEPS][NB][2][2];
      {
        float acc[STEPS][2][QT][4];
#pragma unroll
        for (int st = 0; st < STEPS; ++st)
#pragma unroll
          for (int qt = 0; qt < QT; ++qt)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[st][0][qt][e] = acc[st][1][qt][e] = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          uint32_t kb[STEPS][4];  // (tile 0, first and second 16 bytes), (tile 1, the same)
#pragma unroll
          for (int st = 0; st < STEPS; ++st) {
            const uint32_t rowa = (ka + st * (16 * 128)) ^ ((ks & 3) << 5);
            if (ks < 4) ldsm4<0>(kb[st], rowa);
            else ldsm4<C::CHUNK>(kb[st], rowa);
          }
#pragma unroll
          for (int qt = 0; qt < QT; ++qt) {
#pragma unroll
            for (int st = 0; st < STEPS; ++st)
#pragma unroll
              for (int nt = 0; nt < 2; ++nt) {
                if constexpr (E4M3) mma16832(acc[st][nt][qt], qf[qt][ks], kb[st][2 * nt], kb[st][2 * nt + 1]);
                else mma16816<false>(acc[st][nt][qt], qf[qt][ks], kb[st][2 * nt], kb[st][2 * nt + 1]);
              }
          }
        }
#pragma unroll
        for (int st = 0; st < STEPS; ++st)
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                if constexpr (!E4M3) s[st][b][nt][e] = acc[st][nt][0][b * 2 + e];
                else if constexpr (NB == 1) s[st][b][nt][e] = fmaf(acc[st][nt][0][2 + e], 0x1p-5f, acc[st][nt][0][e]);
                else s[st][b][nt][e] = fmaf(acc[st][nt][QT - 1][b * 2 + e], 0x1p-5f, acc[st][nt][0][b * 2 + e]);
              }
      }
      // V rows that enter the product: masks of this thread's keys (e4m3: four bytes; bf16: two halves of two words),
      // and which of them are new tokens
      uint32_t vkeep[STEPS][E4M3 ? 1 : 2], vnew[STEPS][E4M3 ? 1 : 2];
      float mx[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) mx[b] = -INFINITY;
      uint32_t see[SPECIAL ? NB : 1];
      if constexpr (SPECIAL) {
#pragma unroll
        for (int b = 0; b < NB; ++b) see[b] = row_sees(a, sg, in[b], tok[b], pos0);
      }
#pragma unroll
      for (int st = 0; st < STEPS; ++st) {
        if constexpr (SPECIAL) vkeep[st][0] = vnew[st][0] = vkeep[st][E4M3 ? 0 : 1] = vnew[st][E4M3 ? 0 : 1] = 0u;
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const int key = st * 16 + (nt ? key1 : key0);
          if constexpr (TOKEN) {
            const float2 kf = *reinterpret_cast<const float2*>(ksc + k0 + key);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              s[st][b][nt][0] *= kf.x;
              s[st][b][nt][1] *= kf.y;
            }
          }
          if constexpr (SPECIAL) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int pos = pos0 + key + e;
              const uint32_t bits = E4M3 ? 0xffu << (16 * nt + 8 * e) : 0xffffu << (16 * e);
              if (pos < sg.kv) vkeep[st][E4M3 ? 0 : nt] |= bits;
              if (pos >= sg.base) vnew[st][E4M3 ? 0 : nt] |= bits;
#pragma unroll
              for (int b = 0; b < NB; ++b)
                if (!(see[b] >> (key + e) & 1u)) s[st][b][nt][e] = -INFINITY;
            }
          }
#pragma unroll
          for (int b = 0; b < NB; ++b) mx[b] = fmaxf(mx[b], fmaxf(s[st][b][nt][0], s[st][b][nt][1]));
        }
      }

      if (TOKEN && ok) ok = mbar_wait<true>(vfull, vphase, abort_flag, g.status, FP_DEV_TIMEOUT);
      bool odd = false;  // a new token's V or scale is an infinity or NaN
      [[maybe_unused]] float2 vf[STEPS][2];   // token scales of V, times 2^-kScaleShift
      [[maybe_unused]] float vmx[NB];         // maximum of x + log2(v_scale)
      if constexpr (TOKEN) {
#pragma unroll
        for (int b = 0; b < NB; ++b) vmx[b] = -INFINITY;
#pragma unroll
        for (int st = 0; st < STEPS; ++st)
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            const int key = st * 16 + (nt ? key1 : key0);
            float2 y = *reinterpret_cast<const float2*>(vsc + k0 + key);
            if constexpr (SPECIAL) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float& f = e ? y.y : y.x;
                const int pos = pos0 + key + e;
                if (pos >= sg.kv) {
                  f = 0.f;  // (whatever the slot held before: times a weight of zero it may be NaN)
                } else if (pos >= sg.base && !(f < INFINITY)) {
                  odd = true;
                  f = 0.f;
                }
              }
            }
            const float lx = scale_log2(y.x), ly = scale_log2(y.y);
#pragma unroll
            for (int b = 0; b < NB; ++b)
              vmx[b] = fmaxf(vmx[b], fmaxf(fmaf(s[st][b][nt][0], sl2[b], lx), fmaf(s[st][b][nt][1], sl2[b], ly)));
            vf[st][nt] = make_float2(y.x * kScaleDown, y.y * kScaleDown);
          }
      }

      // ---- softmax
      bool grew = false;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        mx[b] = fmaxf(mx[b], __shfl_xor_sync(0xffffffffu, mx[b], 1));
        mx[b] = fmaxf(mx[b], __shfl_xor_sync(0xffffffffu, mx[b], 2)) * sl2[b];
        grew |= mx[b] > ref[b] + kSlack;
        if constexpr (TOKEN) {
          vmx[b] = fmaxf(vmx[b], __shfl_xor_sync(0xffffffffu, vmx[b], 1));
          vmx[b] = fmaxf(vmx[b], __shfl_xor_sync(0xffffffffu, vmx[b], 2));
          grew |= vmx[b] > vref[b] + kSlack;
        }
      }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          float f = 1.f;
          if (mx[b] > ref[b] + kSlack) {
            f = exp2_fast(ref[b] - mx[b]);
            ref[b] = mx[b];
          }
          l[b] *= f;
          if constexpr (TOKEN) {
            f = 1.f;
            if (vmx[b] > vref[b] + kSlack) {
              f = exp2_fast(vref[b] - vmx[b]);
              vref[b] = vmx[b];
            }
          }
          // O's columns are rows 2c and 2c + 1 of the block
          const float f0 = __shfl_sync(0xffffffffu, f, 8 * c), f1 = __shfl_sync(0xffffffffu, f, 8 * c + 4);
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][b][e] *= (e & 1) ? f1 : f0;
        }
      }
      // weights relative to the reference; f16 ones times 2^kShift
      float neg[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) neg[b] = ref[b] == -INFINITY ? 0.f : (E4M3 ? kShift - ref[b] : -ref[b]);

      if (!TOKEN && ok) ok = mbar_wait<true>(vfull, vphase, abort_flag, g.status, FP_DEV_TIMEOUT);
      [[maybe_unused]] float to_v[NB];  // from weights relative to ref to products relative to vref
      if constexpr (TOKEN) {
#pragma unroll
        for (int b = 0; b < NB; ++b) to_v[b] = products_factor(ref[b], vref[b]);
      }
      uint32_t pf[STEPS][NB][2], pl[STEPS][NB][2];
#pragma unroll
      for (int st = 0; st < STEPS; ++st)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            float p0 = exp2_fast(fmaf(s[st][b][nt][0], sl2[b], neg[b]));
            float p1 = exp2_fast(fmaf(s[st][b][nt][1], sl2[b], neg[b]));
            l[b] += p0 + p1;
            if constexpr (TOKEN) {
              p0 = p0 * vf[st][nt].x * to_v[b];
              p1 = p1 * vf[st][nt].y * to_v[b];
            }
            const uint32_t u = pack2<E4M3>(p0, p1);
            pf[st][b][nt] = u;
            if (!E4M3) pl[st][b][nt] = pack_rest(p0, p1, u);
          }
        }
      // ---- O^T += V^T P^T
      // slots behind the last token hold anything: they enter as zeros; so do the
      // infinities and NaN of new tokens, which only some rows see (added at the end)
      auto clean = [&](uint32_t& w, int st, int half) {
        if constexpr (SPECIAL) {
          const uint32_t magic = E4M3 ? 0x7f7f7f7fu : 0x7f807f80u;
          w &= vkeep[st][half];
          const uint32_t bad = (E4M3 ? __vcmpeq4(w & magic, magic) : __vcmpeq2(w & magic, magic)) & vnew[st][half];
          odd |= bad != 0;
          w &= ~bad;
        }
      };
      if constexpr (!E4M3) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int st = 0; st < STEPS; ++st) {
            uint32_t w[4];
            const uint32_t rowa = (va + st * (16 * 128)) ^ ((mt & 3) << 5);
            if (mt < 4) ldsm4_t<0>(w, rowa);
            else ldsm4_t<C::CHUNK>(w, rowa);
#pragma unroll
            for (int e = 0; e < 4; ++e) clean(w[e], st, e >> 1);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              mma16816<false>(o[mt][b], w, pf[st][b][0], pf[st][b][1]);
              mma16816<false>(o[mt][b], w, pl[st][b][0], pl[st][b][1]);
            }
          }
      } else {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          uint32_t w[4];
          ldsm2_t8(w, va ^ (mt << 4));
#pragma unroll
          for (int st = 0; st < 2; ++st) {  // the load's halves: a block of keys each
            clean(w[2 * st], st, 0);
            clean(w[2 * st + 1], st, 0);
            const uint32_t f[4] = {widen_lo(w[2 * st]), widen_lo(w[2 * st + 1]), widen_hi(w[2 * st]),
                                   widen_hi(w[2 * st + 1])};
#pragma unroll
            for (int b = 0; b < NB; ++b) mma16816<true>(o[mt][b], f, pf[st][b][0], pf[st][b][1]);
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
      const int k0 = warp * STEPS * 16;
      const uint32_t ka = k_lane + kslot * C::SLOT, va = v_lane + vslot * C::SLOT;
      if (t * C::TILE + k0 + STEPS * 16 > sg.base)
        update(std::true_type(), t * C::TILE + k0, k0, ka, va, ksc, vsc, full + vslot, vphase);
      else
        update(std::false_type(), t * C::TILE + k0, k0, ka, va, ksc, vsc, full + vslot, vphase);
      __syncwarp();
      if (ok && lane == 0) {
        mbar_arrive(empty + kslot);
        mbar_arrive(empty + vslot);
      }
    }

    // ---- the warps' results meet
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      l[b] += __shfl_xor_sync(0xffffffffu, l[b], 1);
      l[b] += __shfl_xor_sync(0xffffffffu, l[b], 2);
      if (c == 0) {
        s_m[warp * C::ROWS + gr + 8 * b] = ref[b];
        s_l[warp * C::ROWS + gr + 8 * b] = l[b];
      }
    }
    consumers_sync();
    if (threadIdx.x == 0) s_odd[(segment + 1) & 1] = 0;  // (its readers have passed the barrier above)
    const bool whole = sg.whole();
    const int part = 2 * blockIdx.x + (segment == 0 ? 0 : 1);
    float top[NB], all[NB];  // reference and sum of the rows over the warps
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const float* pm = s_m + gr + 8 * b;
      const float* pl2 = s_l + gr + 8 * b;
      float big = -INFINITY, sum = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) big = fmaxf(big, pm[k * C::ROWS]);
      // (a warp that saw nothing has ref = -inf and l = 0; l may be NaN without a maximum)
#pragma unroll
      for (int k = 0; k < kWarps; ++k)
        sum += pl2[k * C::ROWS] * (big == -INFINITY ? 1.f : exp2_fast(pm[k * C::ROWS] - big));
      float w = big == -INFINITY ? 1.f : exp2_fast(ref[b] - big);
      w = sum == 0.f ? 0.f : __fdividef(w * v_mul, sum);
      if constexpr (TOKEN) w = products_back(big, vref[b], sum);  // (NaN without a maximum: then so is the sum)
      top[b] = big;
      all[b] = sum;
      const float w0 = __shfl_sync(0xffffffffu, w, 8 * c), w1 = __shfl_sync(0xffffffffu, w, 8 * c + 4);
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float we = (e & 1) ? w1 : w0;
          o[i][b][e] = TOKEN ? o[i][b][e] * we * we : o[i][b][e] * we;  // (by zero too: NaN of V stays)
        }
    }
    const bool odd = s_odd[segment & 1] != 0;
#pragma unroll
    for (int round = 0; round < NB; ++round) {
#pragma unroll
      for (int i = 0; i < MT / NB; ++i)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            red[(warp * C::ROWS + 8 * b + 2 * c + (e & 1)) * C::RED_ROW + i * 16 + gr + (e >> 1) * 8] =
                o[round * (MT / NB) + i][b][e];
      consumers_sync();
      constexpr int VECS = C::RED_COLS / 4;
      const int lr = threadIdx.x / VECS, col = threadIdx.x % VECS * 4;
      const int row = sg.row0 + lr;
      if (lr < C::ROWS && row < nrows) {
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
          const float4 y = *reinterpret_cast<const float4*>(red + (k * C::ROWS + lr) * C::RED_ROW + col);
          acc.x += y.x;
          acc.y += y.y;
          acc.z += y.z;
          acc.w += y.w;
        }
        const int d = round * C::RED_COLS + col;
        const int t = group_of(a, row), h = row - t * a.G;
        if (odd) {
          const int end = min(sg.kv, sg.t1 << a.tile_shift);
          const float2 lo = odd_values<E4M3, TOKEN, D>(a, sg.r, sg.off, sg.head, sg.base, sg.t0, end, t, d);
          const float2 hi = odd_values<E4M3, TOKEN, D>(a, sg.r, sg.off, sg.head, sg.base, sg.t0, end, t, d + 2);
          acc = make_float4(acc.x + lo.x, acc.y + lo.y, acc.z + hi.x, acc.w + hi.y);
        }
        if (!E4M3 && isnan((acc.x + acc.y) + (acc.z + acc.w))) {
          float sum = 0.f;
          for (int k = 0; k < kWarps; ++k) sum += s_l[k * C::ROWS + lr];
          if (sum == sum) {
            const float4 f = infinite_values<D>(a, sg.r, sg.off, sg.head, sg.base, sg.t0 << a.tile_shift,
                                                min(sg.kv, sg.t1 << a.tile_shift), t, d);
            acc = make_float4(f.x != 0.f ? f.x : acc.x, f.y != 0.f ? f.y : acc.y, f.z != 0.f ? f.z : acc.z,
                              f.w != 0.f ? f.w : acc.w);
          }
        }
        if (whole) {
          *reinterpret_cast<uint2*>(a.o + ((long long)(sg.off + t) * a.Hq + sg.head * a.G + h) * D + d) =
              make_uint2(pack2<false>(acc.x, acc.y), pack2<false>(acc.z, acc.w));
        } else {
          *reinterpret_cast<float4*>(a.part_o + ((long long)part * a.rows + lr) * D + d) = acc;
        }
      }
      consumers_sync();  // the next round, or the next segment's Q, may be written
    }
    if (warp == kWarps - 1 && c == 0) {  // (behind the barriers: the others are off to the next segment)
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        if (!in[b]) continue;
        // the weights' factor (e4m3) comes off the logarithm
        const float lse2 =
            all[b] == 0.f ? -INFINITY : (top[b] == -INFINITY ? 0.f : top[b]) + log2f(all[b]) - (E4M3 ? kShift : 0.f);
        if (!whole) {
          a.part_lse[(long long)part * a.rows + gr + 8 * b] = lse2;
        } else if (a.lse) {
          const int h = sg.row0 + gr + 8 * b - tok[b] * a.G;
          a.lse[(long long)(sg.head * a.G + h) * g.total_tokens + sg.off + tok[b]] = lse2 * 0.69314718055994531f;
        }
      }
    }
    ++segment;
  }
}

// ---------------------------------------------------------------------------
// combining partial rows
// ---------------------------------------------------------------------------
constexpr int kMergeThreads = 256, kMergeWarps = kMergeThreads / 32;

// The partial rows that a (token, query head) row's unit left in the workspace,
// in CTA order. WIDE: a row per CTA, whose warps sum every eighth partial row
// each; otherwise a row per warp. Which: a CTA has a prologue of a microsecond,
// so many rows go to as many CTAs as run at once, warp by warp (64512 rows, most
// of them finished before: 207 us with a CTA each, 56 us so), and few rows get
// the latency of a CTA. Loads of four rows are in flight, the first ones beside
// the rows' logarithms; a loop of dependent loads took 8-16 us.
template <int D, bool WIDE>
__global__ void __launch_bounds__(kMergeThreads) tree_merge_kernel(const __grid_constant__ TreeArgs a) {
  constexpr int SPLIT = WIDE ? kMergeWarps : 1;  // warps of a row
  constexpr int MOST = 8;       // logarithms per lane: up to 256 SMs
  constexpr int PER = D / 32;   // columns per lane
  constexpr int BATCH = 4;
  extern __shared__ int4 axis_mem[];
  __shared__ int warp_sum[kMergeWarps];
  __shared__ float acc[WIDE ? kMergeWarps : 1][D];
  const CacheGeometry& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, first = WIDE ? warp : 0;
  Axis axis(axis_mem, g.R);
  axis.build(a, warp_sum);
  const int share = share_of(a, axis.total()), rows = g.total_tokens * a.Hq;
  // every thread waits, also those with nothing to do: this grid is not to end
  // before the one that it depends on
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int step = gridDim.x * (WIDE ? 1 : kMergeWarps);
  for (long long at = WIDE ? blockIdx.x : blockIdx.x * kMergeWarps + warp; at < rows; at += step) {
    const int i = (int)at, token = quotient(i, a.Hq), hq = i - token * a.Hq;
    // the request of this token
    int r = 0;
    for (int hi = g.R - 1; r < hi;) {
      const int mid = (r + hi) >> 1;
      if (__ldg(g.cu + mid + 1) > token) hi = mid;
      else r = mid + 1;
    }
    const Span sp = axis.span(a, r);
    if (sp.n == 0 || token < sp.off || token >= sp.off + sp.n) continue;
    const int head = group_of(a, hq), row = (token - sp.off) * a.G + hq - head * a.G, nt = tiles_of(a, sp);
    const int x0 = axis.first(r) + (head * units_of(a, sp) + (row >> a.rows_shift)) * (a.lead + nt), x1 = x0 + a.lead + nt;
    const int c0 = quotient(x0 + a.lead, share), c1 = quotient(x1 - 1, share);
    if (c0 == c1) continue;  // one CTA had the whole unit and finished it
    const int lr = row & (a.rows - 1);
    // its partial in CTA c: the CTA's first segment, unless the unit begins inside the CTA's share
    auto part = [&](int c) { return (long long)(2 * c + ((long long)c * share < x0 ? 1 : 0)) * a.rows + lr; };
    auto load_row = [&](int c, float* y) {
      const float* src = a.part_o + part(c) * D + lane * PER;
      if constexpr (PER == 4) {
        const float4 x = __ldcg(reinterpret_cast<const float4*>(src));
        y[0] = x.x, y[1] = x.y, y[2] = x.z, y[3] = x.w;
      } else {
        const float2 x = __ldcg(reinterpret_cast<const float2*>(src));
        y[0] = x.x, y[1] = x.y;
      }
    };
    float y[BATCH][PER], w[MOST], big = -INFINITY;
#pragma unroll
    for (int j = 0; j < BATCH; ++j) load_row(min(c0 + first + j * SPLIT, c1), y[j]);
#pragma unroll
    for (int k = 0; k < MOST; ++k) {
      const int c = c0 + lane + 32 * k;
      w[k] = c <= c1 ? __ldcg(a.part_lse + part(c)) : -INFINITY;
      big = fmaxf(big, w[k]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
    const float ref = big == -INFINITY ? 0.f : big;
    float sum = 0.f, v[PER];
#pragma unroll
    for (int k = 0; k < MOST; ++k) sum += exp2_fast(w[k] - ref);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
#pragma unroll
    for (int e = 0; e < PER; ++e) v[e] = 0.f;
    for (int c = c0 + first; c <= c1; c += BATCH * SPLIT) {
      if (c != c0 + first) {
#pragma unroll
        for (int j = 0; j < BATCH; ++j) load_row(min(c + j * SPLIT, c1), y[j]);
      }
#pragma unroll
      for (int j = 0; j < BATCH; ++j) {
        const int cj = c + j * SPLIT;
        const float f = cj <= c1 ? exp2_fast(__ldcg(a.part_lse + part(cj)) - ref) : 0.f;
        if (cj > c1) break;  // (the rows behind c1 repeat it)
#pragma unroll
        for (int e = 0; e < PER; ++e) v[e] += f * y[j][e];
      }
    }
    // A weight of zero has made NaN of an infinity, or there is NaN: infinities and NaN of V stay what they are, however
    // small the weight. (Checked for every row above, it took 0.7 to 2 us of a call.)
    float nan = 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) nan += v[e];
    if (isnan(nan) && !isnan(sum)) {
#pragma unroll
      for (int e = 0; e < PER; ++e) v[e] = 0.f;
#pragma unroll 1
      for (int c = c0 + first; c <= c1; c += SPLIT) {
        load_row(c, y[0]);
        const float f = exp2_fast(__ldcg(a.part_lse + part(c)) - ref);
#pragma unroll
        for (int e = 0; e < PER; ++e) v[e] += isfinite(y[0][e]) ? f * y[0][e] : y[0][e];
      }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    __nv_bfloat16* out = a.o + ((long long)token * a.Hq + hq) * D;
    if constexpr (WIDE) {
#pragma unroll
      for (int e = 0; e < PER; ++e) acc[warp][lane * PER + e] = v[e];
      __syncthreads();
      if (threadIdx.x < D) {
        float o = 0.f;
#pragma unroll
        for (int k = 0; k < kMergeWarps; ++k) o += acc[k][threadIdx.x];
        out[threadIdx.x] = __float2bfloat16_rn(o * inv);
      }
      __syncthreads();
    } else {
      uint32_t p[PER / 2];
#pragma unroll
      for (int e = 0; e < PER / 2; ++e) p[e] = pack2<false>(v[2 * e] * inv, v[2 * e + 1] * inv);
      if constexpr (PER == 4) *reinterpret_cast<uint2*>(out + lane * 4) = make_uint2(p[0], p[1]);
      else *reinterpret_cast<uint32_t*>(out + lane * 2) = p[0];
    }
    if (a.lse && lane == 0 && (!WIDE || warp == 0))
      a.lse[(long long)hq * g.total_tokens + token] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.69314718055994531f;
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// Rows per unit: the kernel here holds 8 or 16, the one for many rows (tree_wide.cu) one or two M-tiles of 128. 17 to
// 32 rows are two units here where the page table has room for 1 MB of K and V per KV head at most: a segment of many
// rows takes 25000 clocks beside its tiles, here 4500 (16 requests, 4 KV heads, 32 rows: 256 keys 15.1 -> 11.2 us,
// 1024 keys 25.2 -> 21.9 us bf16 and 27.1 -> 15.4 us e4m3; 4096 keys 38.5 -> 43.8 us bf16, 40.9 -> 38.0 us e4m3).
int unit_rows(const CacheGeometry& g, int max_rows) {
  if (max_rows <= 8) return 8;
  const long long bytes = (long long)g.max_pages * g.page_size * g.d * (g.e4m3 ? 2 : 4);
  if (max_rows <= 16 || (max_rows <= 32 && bytes <= 1 << 20)) return 16;
  return max_rows <= 128 ? 128 : 256;
}

// What a segment takes beside its tiles, in tiles.
constexpr int kNarrowLead = 2, kWideLead = 6;

int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

template <bool E4M3, bool TOKEN, int D, int NB>
cudaError_t run(const TreeArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t s) {
  using C = Cfg<E4M3, D, NB>;
  auto kern = tree_kernel<E4M3, TOKEN, D, NB>;
  const int smem = C::SMEM_FIXED + axis_bytes(a.g.R);
  static std::atomic<unsigned long long> prepared{0};
  const cudaError_t e = prepare(kern, kLaunchRegs, prepared);
  if (e != cudaSuccess) return e;
  kern<<<a.grid, kThreads, smem, s>>>(mk, mv, a);
  return cudaGetLastError();
}

template <int D>
cudaError_t run_merge(const TreeArgs& a, cudaStream_t s) {
  const long long rows = (long long)a.g.total_tokens * a.Hq, resident = (long long)a.grid * 8;
  // Rounds of CTAs, times a prologue and the loads of the partial rows that a row may have (four in flight per warp):
  // about 1.5 us and 0.2 us a partial row of a warp. 512 rows of 37 parts: 60 us with a CTA each, 73 us with a warp;
  // 2048 rows of 2 or 3: 32 us and 26 us.
  const long long units = (long long)a.g.R * a.g.Hkv * ((a.max_tokens * a.G + a.rows - 1) / a.rows);
  const double parts = units < a.grid ? (double)a.grid / units + 1 : 2;
  const double by_cta = (double)((rows + resident - 1) / resident) * (1.5 + 0.2 * parts / kMergeWarps);
  const double by_warp = (double)((rows + resident * kMergeWarps - 1) / (resident * kMergeWarps)) * (1.5 + 0.2 * parts);
  const bool wide = by_cta <= by_warp;
  const long long ctas = wide ? rows : (rows + kMergeWarps - 1) / kMergeWarps;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(ctas < resident || wide ? ctas : resident));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.dynamicSmemBytes = (size_t)axis_bytes(a.g.R);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return wide ? cudaLaunchKernelEx(&cfg, tree_merge_kernel<D, true>, a)
              : cudaLaunchKernelEx(&cfg, tree_merge_kernel<D, false>, a);
}

template <bool E4M3, bool TOKEN, int D>
cudaError_t run_rows(const TreeArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t s) {
  return a.rows == 8 ? run<E4M3, TOKEN, D, 1>(a, mk, mv, s) : run<E4M3, TOKEN, D, 2>(a, mk, mv, s);
}

size_t pad256(size_t bytes) { return (bytes + 255) / 256 * 256; }

}  // namespace

// Two partial units per CTA: float32 O rows, then their logarithms.
size_t tree_workspace(const CacheGeometry& g, int hq, int max_tokens) {
  const size_t rows = (size_t)2 * sm_count() * unit_rows(g, max_tokens * (hq / g.Hkv));
  return pad256(rows * g.d * sizeof(float)) + pad256(rows * sizeof(float));
}

fp_status_t launch_tree(const CacheGeometry& g, const fp_tree_t& t, const void* q, void* o, float* lse, void* ws,
                        cudaStream_t s) {
  TreeArgs a;
  a.g = g;
  a.Hq = t.hq;
  a.G = t.hq / g.Hkv;
  a.max_tokens = t.max_tokens;
  a.rows = unit_rows(g, t.max_tokens * a.G);
  a.mask = t.mask;
  a.mask_words = t.mask_words;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.G_inv = (uint32_t)(((1ull << 32) + a.G - 1) / a.G);
  a.q_stride = t.q_stride ? t.q_stride : (long long)t.hq * g.d;
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  const double scale = t.softmax_scale > 0.f ? (double)t.softmax_scale : 1.0 / std::sqrt((double)g.d);
  a.scale_log2 = (float)(scale * 1.4426950408889634);
  a.grid = sm_count();
  a.tile = a.rows <= 16 ? kTileBytes / (g.d * (g.e4m3 ? 1 : 2)) : 128;
  a.lead = a.rows <= 16 ? kNarrowLead : kWideLead;
  a.min_share = a.rows <= 16 ? 1 : 2;
  a.rows_shift = log2_of(a.rows);
  a.tile_shift = log2_of(a.tile);
  const size_t rows = (size_t)2 * a.grid * a.rows;
  a.part_o = static_cast<float*>(ws);
  a.part_lse = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + pad256(rows * g.d * sizeof(float)));

  CUtensorMap mk, mv;
  const cuuint64_t es = g.e4m3 ? 1 : 2, P = (cuuint64_t)g.page_size;
  const cuuint64_t dims[4] = {(cuuint64_t)g.d, (cuuint64_t)g.Hkv, P, (cuuint64_t)g.num_pages};
  const cuuint64_t strides[3] = {g.d * es, (cuuint64_t)g.Hkv * g.d * es, P * g.Hkv * g.d * es};
  const cuuint32_t box[4] = {(cuuint32_t)(128 / es), 1, (cuuint32_t)(g.page_size < a.tile ? g.page_size : a.tile), 1};
  const CUtensorMapDataType type = g.e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const auto promotion = g.d * es == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
  if (!encode_tiled(&mk, type, 4, g.k_pool, dims, strides, box, promotion) ||
      !encode_tiled(&mv, type, 4, g.v_pool, dims, strides, box, promotion))
    return FP_ERR_CUDA;
  cudaError_t e;
  if (a.rows > 16) e = launch_wide(a, mk, mv, s);
  else if (g.e4m3) e = g.token_scale ? run_rows<true, true, 128>(a, mk, mv, s) : run_rows<true, false, 128>(a, mk, mv, s);
  else e = g.d == 128 ? run_rows<false, false, 128>(a, mk, mv, s) : run_rows<false, false, 64>(a, mk, mv, s);
  if (e == cudaSuccess) e = g.d == 128 ? run_merge<128>(a, s) : run_merge<64>(a, s);
  if (e != cudaSuccess) {
    set_last_error("tree attention launch", (int)e, cudaGetErrorString(e));
    return FP_ERR_CUDA;
  }
  return FP_OK;
}

}  // namespace fp
