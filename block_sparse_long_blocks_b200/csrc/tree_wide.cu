// Attention over the paged cache for many rows: more than 16 (token, head) rows
// per request and KV head, as larger trees and chunks of a prompt bring.
//
// The mathematics, the axis of key tiles, the shares, partial rows and their
// combination are those of tree.cu. Here an M-tile has 128 rows, one per thread
// of a softmax warpgroup, and both products run on tcgen05:
//   S = Q K^T (tensor memory), P = 2^(x - ref) written over S, O += P V.
// PAIR (more than 128 rows): a unit has two M-tiles; every K and V tile serves
// both, and one's softmax overlaps the other's products. Otherwise the unit has
// one M-tile, and the two warpgroups take its key tiles in turn, each with its
// own O, which meet at the segment's end: HBM, not the softmax of one
// warpgroup, then bounds it.
// Measured on the device, whole calls (both launches) back to back: 64 tokens of 8
// query heads over 128K keys (4 KV heads) 144 to 156 us in bf16, 880 to 950 TFLOP/s,
// the tensor pipe busy 48 % of the time (174 to 184 us where inputs change from
// call to call), 147 us in e4m3 with head scales, 222 with token scales; 16 tokens
// (128 rows) 58 us in bf16 (4.6 TB/s) and e4m3, 76 with token scales.
//
// Roles (one CTA per SM): warps 0-3 and 4-7 softmax, warp 8 TMA producer, warps
// 9 and 10 MMA issuers, one per softmax warpgroup, the last warps converters.
// PAIR: the issuers take turns, which keeps one M-tile's products under the
// other's softmax; untied, both warpgroups fell into step, softmax and products
// one after the other (64-token tree over 128K keys: 234 us untied, 206 us with
// one issuer that waits for either warpgroup in turn, 191 us with turns).
// Operands: bf16 caches multiply bf16, with P rounded to bf16 (as hi + lo, 191
// us, otherwise 165). e4m3 caches: S on the e4m3 path with q * 2^e (e per row
// such that max |q| lies in [2^7, 2^8)) as the sum hi + lo of two e4m3 values,
// exact for elements within 2^-9 of the row's largest, others to 2^-17 of it (both
// products go to the same accumulators, which leaves no factor for lo); they take
// the time of one on 16-bit operands, and K is multiplied as it was loaded. V is widened exactly to f16 by the converters, P goes to f16.
// The converters also pass the V tiles on in order, and make those that hold new
// tokens or end behind the last one safe to multiply: rows behind the last token
// become zeros, and so do infinities and NaN of new tokens, which only some rows
// see (those are added to the rows that see them at the end).
// An issuer may watch the phase of a slot only if all earlier ones of that slot
// are over: key tiles alternate between the warpgroups over all segments, and
// the K ring has an even number of slots, so a slot is always of one issuer;
// V tiles come from the converters, in order where three slots are shared.
// Every wait is bounded; after one ran out every role leaves its loop, the MMA
// issuers and the producer wait for what they have in flight, outputs are
// invalid and FP_DEV_TIMEOUT is set.
#include <cuda.h>

#include <climits>

#include "packed.cuh"
#include "tree.cuh"

namespace fp {
namespace tree {

using namespace packed;

namespace {

constexpr int kProducerWarp = 8, kMmaWarp = 9;  // MMA issuers: kMmaWarp + softmax warpgroup
template <bool E4M3>
struct Roles {
  static constexpr int THREADS = E4M3 ? 512 : 384;
  static constexpr int CONVERT_WARP = E4M3 ? 12 : 11;
  static constexpr int GROUPS = E4M3 ? 2 : 1;         // of converters, which take the V tiles in turn
  static constexpr int CONVERTERS = E4M3 ? 64 : 32;   // threads of a group
  // launched with 128 or 168 registers a thread: 2 x 128 x 176 + 256 x 80 = 512 x 128,
  // 2 x 128 x 200 + 128 x 104 = 384 x 168
  static constexpr uint32_t LAUNCH_REGS = E4M3 ? 128 : 168;
  static constexpr uint32_t SOFTMAX_REGS = E4M3 ? 176 : 200, CONTROL_REGS = E4M3 ? 80 : 104;
  static_assert(256 * SOFTMAX_REGS + (THREADS - 256) * CONTROL_REGS <= THREADS * LAUNCH_REGS, "register split");
};
constexpr int kKeys = 128;           // per tile
constexpr int kChunk = kKeys * 128;  // bytes of a tile's 128-byte-wide chunk
constexpr int kFlags = 8;            // > segments that the ring can reach into
constexpr int kScales = 8;           // tiles whose token scales are kept (see the producer),
constexpr int kLogs = 4;             // and the logarithms of V's (see the converters)

template <bool E4M3, int D, bool PAIR>
struct Cfg {
  static constexpr int ES = E4M3 ? 1 : 2;
  static constexpr int CH = D / 64;                     // chunks of a 16-bit tile
  static constexpr int TILE = CH * kChunk;              // bytes of a 16-bit tile
  static constexpr int LOAD_CH = D * ES / 128;          // chunks of a loaded tile
  static constexpr int LOAD = LOAD_CH * kChunk;         // bytes of a loaded tile
  static constexpr int CH_ELEMS = 128 / ES;
  static constexpr int Q1 = E4M3 ? 2 * kChunk : TILE;   // one M-tile's Q (e4m3: hi, then lo)
  static constexpr int Q = (PAIR ? 2 : 1) * Q1;
  // slots: K and V tiles as loaded, and (e4m3) V tiles as f16
  static constexpr int K_SLOTS = D == 64 ? 4 : E4M3 && !PAIR ? 4 : 2;
  static constexpr int V_SLOTS = D == 64 ? 4 : !E4M3 && !PAIR ? 3 : 2;
  static constexpr int W_SLOTS = E4M3 ? 2 : 0;
  static constexpr int M_SLOTS = E4M3 ? W_SLOTS : V_SLOTS;  // V tiles as multiplied
  static constexpr int AHEAD = PAIR ? 1 : 2;            // K tiles loaded before the first V tile; tiles from one
                                                        // of a warpgroup to its next
  static constexpr int NUM_BARS = 2 * K_SLOTS + 2 * V_SLOTS + 2 * M_SLOTS + 2 + 2 + 4 + 2 + 6 + kLogs;
  static constexpr int SMEM_FIXED = 1024 + Q + (K_SLOTS + V_SLOTS) * LOAD + W_SLOTS * TILE +
                                    (E4M3 ? (kScales * 2 + kLogs + 1) * kKeys * 4 : 0) + 256 * 16 + 1024 + NUM_BARS * 8 +
                                    336;
  // columns of O that either of two warpgroups hands the other through Q's place at a time
  static constexpr int COLS = Q1 / 1024;
  static_assert(SMEM_FIXED + kAxisBytesMax <= 227 * 1024, "shared memory");
  static_assert(K_SLOTS % 2 == 0, "a slot is of one issuer");
  static_assert(PAIR || (COLS % 16 == 0 && D / 2 % COLS == 0), "rounds of whole TMEM loads");
};

__device__ __forceinline__ void copy_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// Columns c .. c + 15 of TMEM lanes l .. l + 15 (taddr) as matrix fragments: element 4 j + e of a lane is row
// lane / 4 + 8 (e / 2), column 8 j + 2 (lane % 4) + e % 2.
__device__ __forceinline__ void tmem_ld_frag16(uint32_t taddr, float* f) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7])
               : "r"(taddr));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

template <bool E4M3, bool TOKEN, int D, bool PAIR>
__global__ void __launch_bounds__(Roles<E4M3>::THREADS, 1)
    wide_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                const __grid_constant__ TreeArgs a) {
  using C = Cfg<E4M3, D, PAIR>;
  using L = Roles<E4M3>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + C::Q;
  uint8_t* sV = sK + C::K_SLOTS * C::LOAD;
  uint8_t* sW = sV + C::V_SLOTS * C::LOAD;       // f16 V tiles (e4m3)
  uint8_t* sM = E4M3 ? sW : sV;                  // V tiles as multiplied
  float* s_ksc = reinterpret_cast<float*>(sW + C::W_SLOTS * C::TILE);  // [kScales][kKeys]
  float* s_vsc = s_ksc + (E4M3 ? kScales * kKeys : 0);
  float* s_vlog = s_vsc + (E4M3 ? kScales * kKeys : 0);                // [kLogs][kKeys]: log2 of V's scales (TOKEN)
  float* s_ones = s_vlog + (E4M3 ? kLogs * kKeys : 0);                 // [kKeys] (TOKEN)
  float4* s_half = reinterpret_cast<float4*>(s_ones + (E4M3 ? kKeys : 0));  // [2][128] the warpgroups' sums
  float* s_back = reinterpret_cast<float*>(s_half + 256);                   // [2][128] factors of Q's rows (e4m3)
  uint64_t* k_full = reinterpret_cast<uint64_t*>(s_back + 256);
  uint64_t* k_empty = k_full + C::K_SLOTS;
  uint64_t* v_full = k_empty + C::K_SLOTS;        // loaded
  uint64_t* v_empty = v_full + C::V_SLOTS;
  uint64_t* m_full = v_empty + C::V_SLOTS;        // ready to be multiplied
  uint64_t* m_empty = m_full + C::M_SLOTS;        // (bf16: the loaded tiles themselves, v_empty)
  uint64_t* q_full = m_empty + C::M_SLOTS;        // [2]
  uint64_t* s_full = q_full + 2;                  // [2]
  uint64_t* p_full = s_full + 2;                  // [warpgroup][half of the keys]
  uint64_t* o_full = p_full + 4;                  // [2]
  uint64_t* half_full = o_full + 2;
  uint64_t* half_empty = half_full + 1;
  uint64_t* drain = half_empty + 1;               // [2]
  uint64_t* turn = drain + 2;                     // [2] (PAIR)
  uint64_t* log_full = turn + 2;                  // [kLogs] V's scales are clean, with their logarithms (TOKEN)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(log_full + kLogs);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* warp_sum = reinterpret_cast<int*>(tmem_slot + 2);             // [16]
  volatile uint32_t* s_vmax = tmem_slot + 18;                        // [kLogs][2]: V's largest scales, as bits (TOKEN)
  volatile int* s_odd = reinterpret_cast<volatile int*>(tmem_slot + 50);  // [kFlags][4]
  Axis axis(tmem_slot + 84, a.g.R);

  const CacheGeometry& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;");
  if (threadIdx.x < kFlags * 4) s_odd[threadIdx.x] = 0;
  if (TOKEN && threadIdx.x < kKeys) s_ones[threadIdx.x] = 1.f;
  if (threadIdx.x == (kMmaWarp + 1) * 32) {  // (warp 0 has the axis to build)
    constexpr uint32_t issuers = PAIR ? 2 : 1;  // that multiply with a tile
    for (int s = 0; s < C::K_SLOTS; ++s) {
      mbar_init(k_full + s, 1);
      mbar_init(k_empty + s, issuers);
    }
    for (int s = 0; s < C::V_SLOTS; ++s) {
      mbar_init(v_full + s, 1);
      mbar_init(v_empty + s, E4M3 ? L::CONVERTERS : issuers);
    }
    for (int s = 0; s < C::M_SLOTS; ++s) {
      mbar_init(m_full + s, L::CONVERTERS);
      mbar_init(m_empty + s, issuers);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(q_full + w, PAIR ? 128 : 256);
      mbar_init(s_full + w, 1);
      mbar_init(p_full + 2 * w, 128);
      mbar_init(p_full + 2 * w + 1, 128);
      mbar_init(o_full + w, PAIR ? 1 : 2);
      mbar_init(drain + w, 1);
      mbar_init(turn + w, 1);
    }
    for (int s = 0; s < kLogs; ++s) mbar_init(log_full + s, L::CONVERTERS);
    mbar_init(half_full, 256);
    mbar_init(half_empty, 256);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  axis.build(a, warp_sum);  // (its barrier publishes the initialisation above)
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int total = axis.total();
  const int share = share_of(a, total);
  const long long x_first = (long long)blockIdx.x * share;
  if (x_first >= total) {
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
    return;
  }
  const int x_begin = (int)x_first, x_end = min(total, x_begin + share);
  if (warp >= 8) reg_dealloc<L::CONTROL_REGS>();

  bool ok = true;
  int r = axis.request_of(x_begin);
  if (warp == kProducerWarp) {
    // ------------------------------------------------------------------ producer
    if (lane == 0) {
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
    const int sub_rows = min(g.page_size, kKeys), sub_max = kKeys / sub_rows;  // sub_max <= 8
    int kn = 0, vn = 0;  // K and V tiles issued
    for (int x = x_begin; x < x_end && ok;) {
      Segment sg;
      if (!next_segment(a, axis, x, x_end, r, sg)) continue;
      const int nt = sg.t1 - sg.t0;
      const int32_t* row = g.table + (long long)sg.r * g.max_pages;
      auto page_at = [&](int i) {  // the page of this lane's part of tile i of the segment
        const int tok = (sg.t0 + i) * kKeys + lane * sub_rows;
        return (i < nt && lane < sub_max && tok < sg.kv) ? __ldg(row + (tok >> g.page_shift)) : -1;
      };
      // Token scales go to rings of kScales tiles. Tile n's replace those of n - 8, whose softmax is over: K n waits
      // for the product with K n - 2 or n - 4 and so for the softmax of n - 3 or n - 6 (of its warpgroup), V n for
      // the conversion of V n - 2 and so for the product with V n - 4.
      auto load = [&](bool v, int i, int page) {
        const int tok = (sg.t0 + i) * kKeys + lane * sub_rows;
        const bool mine = lane < sub_max && tok < sg.kv;
        const int subs = min(sub_max, (sg.kv - (sg.t0 + i) * kKeys + sub_rows - 1) / sub_rows);
        const bool bad = mine && (page < 0 || page >= g.num_pages);
        if (bad) {
          atomicOr(g.status, FP_DEV_BAD_PAGE);
          page = g.num_pages;  // outside the pool: the copy fills zeros
        }
        const int n = v ? vn : kn, slots = v ? C::V_SLOTS : C::K_SLOTS, slot = n % slots;
        uint64_t* bar = (v ? v_full : k_full) + slot;
        ok = mbar_wait<true>((v ? v_empty : k_empty) + slot, ((uint32_t)(n / slots) & 1u) ^ 1u, abort_flag, g.status,
                             FP_DEV_TIMEOUT);
        if (!ok) return;
        uint8_t* dst = (v ? sV : sK) + slot * C::LOAD;
        float* scales = (v ? s_vsc : s_ksc) + n % kScales * kKeys;
        uint32_t bytes = (uint32_t)(subs * sub_rows) * (D * C::ES);
        if (TOKEN) bytes += scales_of_tile(scales, bad, mine, lane, sub_rows);
        if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
        __syncwarp();
        if (mine) {
          const int at = tok & (g.page_size - 1);
#pragma unroll
          for (int ch = 0; ch < C::LOAD_CH; ++ch)
            tma_load_4d(dst + ch * kChunk + lane * sub_rows * 128, v ? &tmV : &tmK, bar, ch * C::CH_ELEMS, sg.head, at,
                        page);
          if (TOKEN && !bad)
            bulk_load(scales + lane * sub_rows,
                      (v ? g.v_scale : g.k_scale) + (((long long)page * g.Hkv + sg.head) << g.page_shift) + at,
                      (uint32_t)sub_rows * 4u, bar);
        }
        if (v) ++vn;
        else ++kn;
      };
      int p0 = page_at(0), p1 = page_at(1), p2 = page_at(2);
      load(false, 0, p0);
      if (!PAIR && ok && nt > 1) load(false, 1, p1);
      for (int i = 0; i < nt && ok; ++i) {
        const int p3 = page_at(i + 3);
        load(true, i, p0);
        if (ok && i + C::AHEAD < nt) load(false, i + C::AHEAD, PAIR ? p1 : p2);
        p0 = p1;
        p1 = p2;
        p2 = p3;
      }
    }
    // every copy lands before the CTA's shared memory is released
    if (lane == 0) {
      for (int k = max(0, kn - C::K_SLOTS); k < kn; ++k)
        mbar_drain(k_full + k % C::K_SLOTS, (uint32_t)(k / C::K_SLOTS) & 1u, g.status, FP_DEV_TIMEOUT);
      for (int k = max(0, vn - C::V_SLOTS); k < vn; ++k)
        mbar_drain(v_full + k % C::V_SLOTS, (uint32_t)(k / C::V_SLOTS) & 1u, g.status, FP_DEV_TIMEOUT);
    }
  } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
    // ------------------------------------------------------------------ MMA issuer of softmax warpgroup w
    const int w = warp - kMmaWarp;
    if (lane == 0) {
      // S: e4m3 or bf16; O += P V: f16 or bf16
      constexpr uint32_t idesc_qk = instr_desc(E4M3 ? 0u : 1u, 128, kKeys, 0, 0);
      constexpr uint32_t idesc_pv = instr_desc(E4M3 ? 0u : 1u, 128, D, 0, 1);
      const uint64_t dQ = smem_desc_sw128(smem_u32(sQ) + (PAIR ? w : 0) * C::Q1, 16, 1024);
      const uint64_t dK = smem_desc_sw128(smem_u32(sK), 16, 1024);
      const uint64_t dV = smem_desc_sw128(smem_u32(sM), kChunk, 1024);
      const uint32_t tS = tmem + w * 128, tO = tmem + 256 + w * 128;
      auto issue_qk = [&](int slot) {
        const uint64_t b0 = dK + (uint64_t)((slot * C::LOAD) >> 4);
        if constexpr (E4M3) {
#pragma unroll
          for (int ks = 0; ks < 2 * D / 32; ++ks)  // hi, then lo
            umma_f8_ss(tS, dQ + (uint32_t)(((ks >> 2) * kChunk + (ks & 3) * 32) >> 4), b0 + (uint32_t)(((ks & 3) * 32) >> 4),
                       idesc_qk, ks > 0);
        } else {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t off = (uint32_t)((ks >> 2) * kChunk + (ks & 3) * 32) >> 4;
            umma_f16_ss(tS, dQ + off, b0 + off, idesc_qk, ks > 0);
          }
        }
      };
      // P of a half of the keys: 32 columns
      auto issue_pv = [&](int slot, bool acc, int hf) {
        const uint64_t b0 = dV + (uint64_t)((slot * C::TILE) >> 4);
#pragma unroll
        for (int ks = 0; ks < kKeys / 32; ++ks) {
          const uint64_t bd = b0 + ((uint32_t)((hf * (kKeys / 32) + ks) * 16 * 128) >> 4);
          umma_f16_ts(tO, tS + hf * 32 + ks * 8, bd, idesc_pv, (acc || ks > 0) ? 1u : 0u);
        }
      };
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        ok = mbar_wait(bar, parity, abort_flag, g.status, FP_DEV_TIMEOUT);
        return ok;
      };
      auto wait_k = [&](int n) { return wait(k_full + n % C::K_SLOTS, (uint32_t)(n / C::K_SLOTS) & 1u); };
      auto wait_v = [&](int n) { return wait(m_full + n % C::M_SLOTS, (uint32_t)(n / C::M_SLOTS) & 1u); };
      uint64_t* v_done = E4M3 ? m_empty : v_empty;
      int tn = 0, qn = 0, pn = 0, turns = 0;
      if (PAIR && w == 1) mbar_arrive(turn);  // the first turn is issuer 0's
      for (int x = x_begin; x < x_end && ok;) {
        Segment sg;
        if (!next_segment(a, axis, x, x_end, r, sg)) continue;
        const int nt = sg.t1 - sg.t0;
        const int first = PAIR ? 0 : (w - tn) & 1;  // tiles first, first + AHEAD, ...
        if (!wait(q_full + (PAIR ? w : 0), (uint32_t)qn & 1u)) break;
        ++qn;
        if (first < nt) {
          const int n = tn + first;
          if (!wait_k(n)) break;
          tc_fence_after();
          issue_qk(n % C::K_SLOTS);
          umma_commit(s_full + w);
          umma_commit(k_empty + n % C::K_SLOTS);
        }
        for (int i = first; i < nt; i += C::AHEAD) {
          const bool more = i + C::AHEAD < nt;
          const int v = tn + i, vslot = v % C::M_SLOTS, k = v + C::AHEAD, kslot = k % C::K_SLOTS;
          if (!wait_v(v)) break;
          if (PAIR && more && !wait_k(k)) break;
          if (!wait(p_full + 2 * w, (uint32_t)pn & 1u)) break;
          if (PAIR && !wait(turn + w, (uint32_t)turns & 1u)) break;
          ++turns;
          tc_fence_after();
          issue_pv(vslot, i > first, 0);
          if (!PAIR && more && !wait_k(k)) break;
          if (!wait(p_full + 2 * w + 1, (uint32_t)pn & 1u)) break;
          ++pn;
          tc_fence_after();
          issue_pv(vslot, true, 1);
          if (more) {
            issue_qk(kslot);
            umma_commit(s_full + w);
          }
          if (PAIR) mbar_arrive(turn + (w ^ 1));
          umma_commit(v_done + vslot);
          if (more) umma_commit(k_empty + kslot);
        }
        if (!ok) break;
        umma_commit(o_full + w);
        if (!PAIR) umma_commit(o_full + 1 - w);  // (a shared Q tile is free when both have done)
        tn += nt;
      }
      // every MMA this thread issued has completed once `drain` flips
      umma_commit(drain + w);
      mbar_drain(drain + w, 0u, g.status, FP_DEV_TIMEOUT);
    }
  } else if (warp >= L::CONVERT_WARP) {
    // ------------------------------------------------------------------ converters
    const int cw = warp - L::CONVERT_WARP, team = L::GROUPS == 1 ? 0 : cw >> 1;
    const int ct = threadIdx.x - (L::CONVERT_WARP * 32 + team * L::CONVERTERS);
    int tn = 0, segment = 0;
    for (int x = x_begin; x < x_end && ok;) {
      Segment sg;
      if (!next_segment(a, axis, x, x_end, r, sg)) continue;
      const int nt = sg.t1 - sg.t0;
      for (int i = 0; i < nt; ++i, ++tn) {
        if (L::GROUPS == 2 && (tn & 1) != team) continue;
        const int vs = tn % C::V_SLOTS, ms = tn % C::M_SLOTS;
        ok = mbar_wait<true>(v_full + vs, (uint32_t)(tn / C::V_SLOTS) & 1u, abort_flag, g.status, FP_DEV_TIMEOUT);
        if (!ok) break;
        const int pos0 = (sg.t0 + i) * kKeys;
        const bool special = pos0 + kKeys > sg.base;
        uint8_t* dst = sM + ms * C::TILE;
        bool odd = false;
        if constexpr (!E4M3) {
          if (special) {
            for (int q = ct; q < C::CH * kKeys * 8; q += L::CONVERTERS) {  // (where a granule lies in its row does not matter)
              const int pos = pos0 + ((q >> 3) & (kKeys - 1));
              if (pos < sg.base) continue;
              uint4* p = reinterpret_cast<uint4*>(dst) + q;
              if (pos >= sg.kv) {
                *p = make_uint4(0, 0, 0, 0);
                continue;
              }
              const uint4 w = *p;
              const uint32_t m = 0x7f807f80u;
              const uint32_t b0 = __vcmpeq2(w.x & m, m), b1 = __vcmpeq2(w.y & m, m), b2 = __vcmpeq2(w.z & m, m),
                             b3 = __vcmpeq2(w.w & m, m);
              if (b0 | b1 | b2 | b3) {
                odd = true;
                *p = make_uint4(w.x & ~b0, w.y & ~b1, w.z & ~b2, w.w & ~b3);
              }
            }
          }
        } else {
          if constexpr (TOKEN) {
            // The softmax needs the scales before the products with V need the tile, so they are out before the wait for
            // its place. Tile n's logarithms replace those of n - 4, whose softmax is over: V n is here, so V n - 2 and
            // V n - 3 are converted, which followed the products with V n - 4 and V n - 5. Whoever waits for tile n of
            // log_full has its scores, which follow the products with V n - 4, and n + 4 comes after those with V n.
            float2& at = reinterpret_cast<float2*>(s_vsc + tn % kScales * kKeys)[ct];  // (two keys per converter)
            float2 sc = at;
            if (special) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float& y = e ? sc.y : sc.x;
                const int pos = pos0 + 2 * ct + e;
                if (pos >= sg.kv) {
                  y = 0.f;
                } else if (pos >= sg.base && !(y < INFINITY)) {
                  y = 0.f;
                  odd = true;
                }
              }
            }
            at = make_float2(sc.x * kScaleDown, sc.y * kScaleDown);
            reinterpret_cast<float2*>(s_vlog + tn % kLogs * kKeys)[ct] = make_float2(scale_log2(sc.x), scale_log2(sc.y));
            // (scales are not negative: without the sign of a -0 they compare as integers)
            const uint32_t top =
                __reduce_max_sync(0xffffffffu, max(__float_as_uint(fabsf(sc.x)), __float_as_uint(fabsf(sc.y))));
            if (lane == 0) s_vmax[tn % kLogs * 2 + (cw & 1)] = top;
            mbar_arrive(log_full + tn % kLogs);
          }
          ok = mbar_wait<true>(m_empty + ms, ((uint32_t)(tn / C::M_SLOTS) & 1u) ^ 1u, abort_flag, g.status,
                               FP_DEV_TIMEOUT);
          if (!ok) break;
          const uint8_t* src = sV + vs * C::LOAD;
          constexpr int U = TOKEN ? 2 : 4;  // (more would spill: 235 us, not 223, 64 tokens over 128K keys)
#pragma unroll U
          for (int q = ct; q < kKeys * 8; q += L::CONVERTERS) {
            // eight threads take four granules each of keys k and k ^ 5: their 16-byte places differ in the swizzled
            // row that is read and in the two that are written
            const int key = ((q >> 6) << 3) | (((q >> 4) & 3) ^ ((q & 4) ? 5 : 0));
            const int g8 = (q & 3) | ((q >> 1) & 4), sw = key & 7;
            uint4 w = *reinterpret_cast<const uint4*>(src + key * 128 + ((g8 ^ sw) << 4));
            if (special && pos0 + key >= sg.base) {
              const uint32_t m = 0x7f7f7f7fu;
              if (pos0 + key >= sg.kv) w = make_uint4(0, 0, 0, 0);
              const uint32_t b0 = __vcmpeq4(w.x & m, m), b1 = __vcmpeq4(w.y & m, m), b2 = __vcmpeq4(w.z & m, m),
                             b3 = __vcmpeq4(w.w & m, m);
              odd |= (b0 | b1 | b2 | b3) != 0;
              w = make_uint4(w.x & ~b0, w.y & ~b1, w.z & ~b2, w.w & ~b3);
            }
            uint8_t* row = dst + (g8 >> 2) * kChunk + key * 128;
            const int p = 2 * (g8 & 3);
            *reinterpret_cast<uint4*>(row + ((p ^ sw) << 4)) =
                make_uint4(widen_lo(w.x), widen_hi(w.x), widen_lo(w.y), widen_hi(w.y));
            *reinterpret_cast<uint4*>(row + (((p + 1) ^ sw) << 4)) =
                make_uint4(widen_lo(w.z), widen_hi(w.z), widen_lo(w.w), widen_hi(w.w));
          }
        }
        if (odd) s_odd[segment % kFlags * 4 + cw] = segment + 1;
        // the tensor cores read the tile through the async proxy
        if (E4M3 || special) fence_async();
        mbar_arrive(m_full + ms);
        if (E4M3) mbar_arrive(v_empty + vs);
      }
      ++segment;
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------------ softmax warpgroups
    reg_alloc<L::SOFTMAX_REGS>();
    const int w = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lane_base = (uint32_t)(row & ~31) << 16;
    const uint32_t tS = tmem + lane_base + w * 128;
    const uint32_t tO = tmem + lane_base + 256 + w * 128;
    int tn = 0, sn = 0, on = 0, hn = 0, segment = 0;
    for (int x = x_begin; x < x_end;) {
      Segment sg;
      if (!next_segment(a, axis, x, x_end, r, sg)) continue;
      const int nt = sg.t1 - sg.t0;
      // The unit's rows go round the warps, 4 i + warp in lane i: the start and the end of a segment, which take a warp
      // as long as it has rows, are shared evenly by the four of a warpgroup also where rows are few.
      const int lr = (PAIR ? w * 128 : 0) + 4 * lane + (warp & 3), rho = sg.row0 + lr;
      const bool in = rho < sg.n * a.G;
      const int tok = in ? group_of(a, rho) : 0, h = in ? rho - tok * a.G : 0;
      const int rows_in = __popc(__ballot_sync(0xffffffffu, in));  // (the warp's first ones)
      // ---- Q: the rows that exist, with consecutive lanes on a row. (What stays in the others' place makes scores
      // of rows that nobody stores.) Of a shared tile either warpgroup takes half of every row, or every other pair.
      float sl2 = a.scale_log2;
      {
        const long long mine = in ? (long long)(sg.off + tok) * a.q_stride + (sg.head * a.G + h) * D : 0;
        uint8_t* dst = sQ + (PAIR ? w * C::Q1 : 0);
        if constexpr (!E4M3) {
          constexpr int PER = PAIR ? D / 8 : 8;  // granules of a row that this warpgroup copies
          const int ch0 = PAIR ? 0 : w, gran = lane % PER;
          if (ch0 < C::CH) {
#pragma unroll 2
            for (int rr = lane / PER; rr < 32; rr += 32 / PER) {
              const long long q = __shfl_sync(0xffffffffu, mine, rr);
              const int at = (warp & 3) * 32 + rr;
              if (rr < rows_in)
                copy_async16(dst + (ch0 + (gran >> 3)) * kChunk + at * 128 + (((gran ^ at) & 7) << 4),
                             a.q + q + ch0 * 64 + gran * 8);
            }
          }
          copies_wait();
        } else {
          const int gran = lane & 15, step = PAIR ? 2 : 4, rr0 = (PAIR ? 0 : 2 * w) + (lane >> 4);
          auto fetch = [&](int rr) {
            const long long q = __shfl_sync(0xffffffffu, mine, rr & 31);
            return rr < rows_in ? __ldg(reinterpret_cast<const uint4*>(a.q + q) + gran) : make_uint4(0, 0, 0, 0);
          };
          uint4 next[2] = {fetch(rr0), fetch(rr0 + step)};
#pragma unroll 1
          for (int rr = rr0; rr - (lane >> 4) < rows_in; rr += 2 * step) {
            const uint4 v[2] = {next[0], next[1]};
            next[0] = fetch(rr + 2 * step);
            next[1] = fetch(rr + 3 * step);
            float mx[2] = {0.f, 0.f};
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t u[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
              for (int e = 0; e < 4; ++e)
                mx[k] = max3(mx[k], fabsf(__uint_as_float(u[e] << 16)), fabsf(__uint_as_float(u[e] & 0xffff0000u)));
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1)
#pragma unroll
              for (int k = 0; k < 2; ++k) mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], o));
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t u[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
              // times 2^(7 - floor(log2 max)): the largest lies in [2^7, 2^8); rows of zeros or below 2^-100 take the
              // limits
              const int e2 = mx[k] == 0.f ? 7 : max((int)((__float_as_uint(mx[k]) >> 23) & 255u) - 127, -100);
              const float up =
                  mx[k] < INFINITY ? __uint_as_float((uint32_t)(7 - e2 + 127) << 23) : __uint_as_float(0x7fc00000u);
              uint32_t hi[2], lo[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float x0 = __uint_as_float(u[2 * e] << 16) * up, x1 = __uint_as_float(u[2 * e] & 0xffff0000u) * up;
                const float x2 = __uint_as_float(u[2 * e + 1] << 16) * up;
                const float x3 = __uint_as_float(u[2 * e + 1] & 0xffff0000u) * up;
                hi[e] = pack_codes(x0, x1) | (pack_codes(x2, x3) << 16);
                const uint32_t h01 = widen_lo(hi[e]), h23 = widen_hi(hi[e]);
                const float2 f01 = __half22float2(*reinterpret_cast<const __half2*>(&h01));
                const float2 f23 = __half22float2(*reinterpret_cast<const __half2*>(&h23));
                lo[e] = pack_codes(x0 - f01.x, x1 - f01.y) | (pack_codes(x2 - f23.x, x3 - f23.y) << 16);
              }
              const int r1 = rr + k * step, at = (warp & 3) * 32 + r1;
              if (r1 < rows_in) {
                uint8_t* put = dst + at * 128 + ((((gran >> 1) ^ at) & 7) << 4) + (gran & 1) * 8;
                *reinterpret_cast<uint2*>(put) = make_uint2(hi[0], hi[1]);
                *reinterpret_cast<uint2*>(put + kChunk) = make_uint2(lo[0], lo[1]);
                if (gran == 0) s_back[(PAIR ? w * 128 : 0) + at] = __uint_as_float((uint32_t)(e2 - 7 + 127) << 23);
              }
            }
          }
        }
        fence_async();
        mbar_arrive(q_full + (PAIR ? w : 0));
      }
      float v_mul = 1.f;  // what O is multiplied by at the end
      if (E4M3 && !TOKEN) v_mul = __ldg(g.v_scale + sg.head);
      // what O is relative to where that is not ref (TOKEN, see products_factor): a maximum of x + log2(v_scale)
      [[maybe_unused]] float vref = -INFINITY;

      // l: the sum of the weights; lu: of the weights as they are multiplied with V (bf16), by which O is
      // divided, so that O stays an average of V rows whatever the rounding
      float ref = -INFINITY, l = 0.f, lu = 0.f;
      const bool any_rows = __any_sync(0xffffffffu, in);
      const int first = PAIR ? 0 : (w - tn) & 1;
      for (int i = first; i < nt; i += C::AHEAD) {
        ok = mbar_wait<true>(s_full + w, (uint32_t)sn & 1u, abort_flag, g.status, FP_DEV_TIMEOUT);
        if (!ok) break;
        ++sn;
        tc_fence_after();
        if (E4M3 && i == first) {  // (the tile's rows are there: the product was made of them)
          sl2 *= in ? s_back[(PAIR ? w * 128 : 0) + row] : 1.f;
          if (!TOKEN) sl2 *= __ldg(g.k_scale + sg.head);
          if (sl2 == 0.f) sl2 = 1.2e-38f;  // (0 * -inf of a masked key would be NaN)
        }
        if (!any_rows) {  // (what P holds for them goes to rows that nobody stores)
          tc_fence_before();
          mbar_arrive(p_full + 2 * w);
          mbar_arrive(p_full + 2 * w + 1);
          continue;
        }
        const int pos0 = (sg.t0 + i) * kKeys;
        const float* ksc = s_ksc + (tn + i) % kScales * kKeys;
        if (pos0 + kKeys > sg.base) {
          // New tokens, or slots behind the last one: the scores are scaled and masked where they lie.
#pragma unroll 1
          for (int c0 = 0; c0 < kKeys; c0 += 32) {
            float x[32];
            tmem_ld32(tS + c0, reinterpret_cast<uint32_t*>(x));
            const uint32_t see = row_sees(a, sg, in, tok, pos0 + c0);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 32; ++c) x[c] = (see >> c & 1u) ? (TOKEN ? x[c] * ksc[c0 + c] : x[c]) : -INFINITY;
            tmem_st32(tS + c0, *reinterpret_cast<const uint32_t(*)[32]>(x));
          }
          tmem_wait_st();
          ksc = s_ones;
        }
        // 64 scores from column c0 on. They are read twice, for the maximum and for the weights, in loops and not
        // unrolled: a CTA that has two tiles of a unit runs this code twice, and instructions that are not in the
        // cache yet take seven clocks each.
        auto scores = [&](float* x, int c0) {
          tmem_ld32(tS + c0, reinterpret_cast<uint32_t*>(x));
          tmem_ld32(tS + c0 + 32, reinterpret_cast<uint32_t*>(x) + 32);
          tmem_wait_ld();
          if constexpr (TOKEN) {
#pragma unroll
            for (int c = 0; c < 64; c += 4) {
              const float4 f = *reinterpret_cast<const float4*>(ksc + c0 + c);
              f2_unpack(f2_mul(f2_pack(x[c], x[c + 1]), f2_pack(f.x, f.y)), x[c], x[c + 1]);
              f2_unpack(f2_mul(f2_pack(x[c + 2], x[c + 3]), f2_pack(f.z, f.w)), x[c + 2], x[c + 3]);
            }
          }
        };
        float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll 1
        for (int c0 = 0; c0 < kKeys; c0 += 64) {
          float x[64];
          scores(x, c0);
#pragma unroll
          for (int c = 0; c < 64; c += 4) {
            m0 = max3(m0, x[c], x[c + 1]);
            m1 = max3(m1, x[c + 2], x[c + 3]);
          }
        }
        const float mx = fmaxf(m0, m1) * sl2;
        float f = 1.f;
        if (mx > ref + kSlack) {
          f = exp2_fast(ref - mx);
          ref = mx;
          l *= f;
          lu *= f;
        }
        [[maybe_unused]] float to_v = 1.f;
        if constexpr (TOKEN) {
          const int at = (tn + i) % kLogs;
          ok = mbar_wait<true>(log_full + at, (uint32_t)((tn + i) / kLogs) & 1u, abort_flag, g.status, FP_DEV_TIMEOUT);
          if (!ok) break;
          f = 1.f;
          // The tile's largest scale bounds x + log2(v_scale): the exact maxima are only formed where some row's reference
          // may have to rise, which they decide (a half more than covers the roundings; formed for every tile: 255 us where
          // this takes 223 us, 64 tokens of 8 query heads over 128K keys).
          const float most = mx + scale_log2(__uint_as_float(max(s_vmax[at * 2], s_vmax[at * 2 + 1])));
          if (__any_sync(0xffffffffu, most + 0.5f > vref + kSlack)) {
            float v0 = -INFINITY, v1 = -INFINITY;
#pragma unroll 1
            for (int c0 = 0; c0 < kKeys; c0 += 16) {
              float x[16];
              tmem_ld16(tS + c0, reinterpret_cast<uint32_t(&)[16]>(x));
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < 16; c += 4) {
                const float4 k = *reinterpret_cast<const float4*>(ksc + c0 + c);
                const float4 lg = *reinterpret_cast<const float4*>(s_vlog + at * kKeys + c0 + c);
                v0 = max3(v0, fmaf(x[c] * k.x, sl2, lg.x), fmaf(x[c + 1] * k.y, sl2, lg.y));
                v1 = max3(v1, fmaf(x[c + 2] * k.z, sl2, lg.z), fmaf(x[c + 3] * k.w, sl2, lg.w));
              }
            }
            const float vmx = fmaxf(v0, v1);
            if (vmx > vref + kSlack) {
              f = exp2_fast(vref - vmx);
              vref = vmx;
            }
          }
          to_v = products_factor(ref, vref);
        }
        if (i > first && __any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            uint32_t r16[16];
            tmem_ld16(tO + c * 16, r16);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) r16[e] = __float_as_uint(__uint_as_float(r16[e]) * f);
            tmem_st16(tO + c * 16, r16);
          }
        }
        const float neg = ref == -INFINITY ? 0.f : (E4M3 ? kShift - ref : -ref);
        const uint64_t sl2x2 = f2_pack(sl2, sl2), negx2 = f2_pack(neg, neg);
        [[maybe_unused]] const uint64_t to_vx2 = f2_pack(to_v, to_v);
        uint64_t sum0 = 0, sum1 = 0, used0 = 0, used1 = 0;  // (pairs of float32 zeros)
        const float* vsc = s_vsc + (tn + i) % kScales * kKeys;
        // P goes out in two halves of the keys; O += P V starts on the first while the second is computed
#pragma unroll 1
        for (int hf = 0; hf < 2; ++hf) {
          float x[64];
          uint32_t p16[32];
          scores(x, hf * 64);
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float p0, p1;
            f2_unpack(f2_fma(f2_pack(x[2 * e], x[2 * e + 1]), sl2x2, negx2), p0, p1);
            p0 = exp2_fast(p0);
            p1 = exp2_fast(p1);
            const uint64_t p = f2_pack(p0, p1);
            if (e & 1) sum1 = f2_add(sum1, p);
            else sum0 = f2_add(sum0, p);
            if constexpr (TOKEN) {
              const float2 vs = *reinterpret_cast<const float2*>(vsc + hf * 64 + 2 * e);
              f2_unpack(f2_mul(f2_mul(p, f2_pack(vs.x, vs.y)), to_vx2), p0, p1);
            }
            p16[e] = pack2<E4M3>(p0, p1);
            if constexpr (!E4M3) {
              const uint64_t q = f2_pack(__uint_as_float(p16[e] << 16), __uint_as_float(p16[e] & 0xffff0000u));
              if (e & 1) used1 = f2_add(used1, q);
              else used0 = f2_add(used0, q);
            }
          }
          tmem_st32(tS + hf * 32, p16);
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(p_full + 2 * w + hf);
        }
        float a0, a1, a2, a3;
        f2_unpack(sum0, a0, a1);
        f2_unpack(sum1, a2, a3);
        l += (a0 + a1) + (a2 + a3);
        if constexpr (!E4M3) {
          f2_unpack(used0, a0, a1);
          f2_unpack(used1, a2, a3);
          lu += (a0 + a1) + (a2 + a3);
        }
      }
      if (E4M3) lu = l;
      if (!ok) break;
      ok = mbar_wait<true>(o_full + w, (uint32_t)on & 1u, abort_flag, g.status, FP_DEV_TIMEOUT);
      if (!ok) break;
      ++on;
      tc_fence_after();

      // ---- the segment's rows
      const bool whole = sg.whole();
      const long long part = 2 * blockIdx.x + (segment == 0 ? 0 : 1);
      auto flagged = [&](volatile int* f) {
        const int s1 = segment + 1;
        return E4M3 ? f[0] == s1 || f[1] == s1 || f[2] == s1 || f[3] == s1 : f[0] == s1;
      };
      const bool odd = sg.t1 * kKeys > sg.base && flagged(s_odd + segment % kFlags * 4);
      // This lane's fragments: rows lane / 4 + 8 k of the warp's (k = 0 .. 3), columns 2 (lane % 4) + {0, 1} of eight.
      // Where they go, in bytes. (A thread that stored its own row wrote 32 lines per store, which took 9000 clocks.)
      const int fr = lane >> 2, fc = 2 * (lane & 3);
      uint8_t* to[4];
      int row_tok[4];
      {
        uint8_t* mine = whole ? reinterpret_cast<uint8_t*>(a.o + ((long long)(sg.off + tok) * a.Hq + sg.head * a.G + h) * D)
                              : reinterpret_cast<uint8_t*>(a.part_o + (part * a.rows + lr) * D);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const unsigned long long there = __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), 8 * k + fr);
          to[k] = 8 * k + fr < rows_in ? reinterpret_cast<uint8_t*>(there) : nullptr;
          row_tok[k] = __shfl_sync(0xffffffffu, tok, 8 * k + fr);
        }
      }
      // columns c0 .. c0 + 15 of 16 rows (half hf) with their rows' factors applied
      auto store16 = [&](float* f, int hf, int c0) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint8_t* at = hf ? to[2 + k] : to[k];
          if (at == nullptr) continue;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float2 v = make_float2(f[4 * j + 2 * k], f[4 * j + 2 * k + 1]);
            const int d = c0 + 8 * j + fc;
            if (odd) {
              const float2 add = odd_values<E4M3, TOKEN, D>(a, sg.r, sg.off, sg.head, sg.base, sg.t0,
                                                            min(sg.kv, sg.t1 * kKeys), hf ? row_tok[2 + k] : row_tok[k], d);
              v = make_float2(v.x + add.x, v.y + add.y);
            }
            if (whole) *reinterpret_cast<uint32_t*>(at + 2 * d) = pack2<false>(v.x, v.y);
            else *reinterpret_cast<float2*>(at + 4 * d) = v;
          }
        }
      };
      auto store_lse = [&](float top, float sum) {
        if (!in) return;
        // the weights' factor (e4m3) comes off the logarithm
        const float lse2 = sum == 0.f ? -INFINITY : (top == -INFINITY ? 0.f : top) + log2f(sum) - (E4M3 ? kShift : 0.f);
        if (!whole) a.part_lse[part * a.rows + lr] = lse2;
        else if (a.lse)
          a.lse[(long long)(sg.head * a.G + h) * g.total_tokens + sg.off + tok] = lse2 * 0.69314718055994531f;
      };
      if (PAIR || nt == 1) {
        if ((PAIR || first == 0) && any_rows) {
          const float f = TOKEN ? products_back(ref, vref, l) : lu == 0.f ? 0.f : v_mul / lu;
#pragma unroll 1
          for (int hf = 0; hf < 2; ++hf) {
            if (hf * 16 >= rows_in) break;
            const float f0 = __shfl_sync(0xffffffffu, f, hf * 16 + fr), f1 = __shfl_sync(0xffffffffu, f, hf * 16 + 8 + fr);
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
              float o[16];
              tmem_ld_frag16(tO + (hf << 20) + c0, o);
              tmem_ld_frag16(tO + (hf << 20) + c0 + 16, o + 8);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float fe = (e & 2) ? f1 : f0;
                o[e] = TOKEN ? o[e] * fe * fe : o[e] * fe;
              }
              store16(o, hf, c0);
              store16(o + 8, hf, c0 + 16);
            }
          }
          store_lse(ref, l);
        }
      } else {
        // Either warpgroup finishes half of the columns: the other's O comes through Q's place (its products are over)
        // in rounds of COLS columns, every thread's fragments to the same thread of the other.
        s_half[w * 128 + row] = make_float4(ref, l, TOKEN ? vref : v_mul, lu);
        float* box = reinterpret_cast<float*>(sQ) + (threadIdx.x & 127) * 4;  // [2][COLS / 4 pieces][128][4]
        constexpr int PIECES = C::COLS / 4;
        float top = 0.f, sum = 0.f, mine = 0.f, theirs = 0.f;
        float fm[4], ft[4];  // factors of this lane's rows
#pragma unroll 1
        for (int c0 = 0; c0 < D / 2; c0 += C::COLS) {
          const int give = (1 - w) * (D / 2) + c0, keep = w * (D / 2) + c0;
          if (any_rows) {
#pragma unroll
            for (int c = 0; c < C::COLS; c += 16)
#pragma unroll
              for (int hf = 0; hf < 2; ++hf) {
                if (hf * 16 >= rows_in) continue;
                float o[8];
                tmem_ld_frag16(tO + (hf << 20) + give + c, o);
                tmem_wait_ld();
                float* at = box + ((1 - w) * PIECES + c / 4 + hf * 2) * 512;
                *reinterpret_cast<float4*>(at) = make_float4(o[0], o[1], o[2], o[3]);
                *reinterpret_cast<float4*>(at + 512) = make_float4(o[4], o[5], o[6], o[7]);
              }
          }
          mbar_arrive(half_full);
          ok = mbar_wait<true>(half_full, (uint32_t)hn & 1u, abort_flag, g.status, FP_DEV_TIMEOUT);
          if (!ok) break;
          if (c0 == 0) {
            const float4 y = s_half[(1 - w) * 128 + row];
            top = fmaxf(ref, y.x);
            const float e0 = top == -INFINITY ? 1.f : exp2_fast(ref - top);
            const float e1 = top == -INFINITY ? 1.f : exp2_fast(y.x - top);
            sum = l * e0 + y.y * e1;
            const float used = lu * e0 + y.w * e1;
            if constexpr (TOKEN) {  // (NaN where neither has a maximum: then so is `used`, or zero)
              mine = products_back(top, vref, used);
              theirs = products_back(top, y.z, used);
            } else {
              mine = used == 0.f ? 0.f : e0 * v_mul / used;
              theirs = used == 0.f ? 0.f : e1 * y.z / used;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              fm[k] = __shfl_sync(0xffffffffu, mine, 8 * k + fr);
              ft[k] = __shfl_sync(0xffffffffu, theirs, 8 * k + fr);
            }
          }
          if (any_rows) {
#pragma unroll
            for (int c = 0; c < C::COLS; c += 16)
#pragma unroll
              for (int hf = 0; hf < 2; ++hf) {
                if (hf * 16 >= rows_in) continue;
                float o[8];
                tmem_ld_frag16(tO + (hf << 20) + keep + c, o);
                const float* at = box + (w * PIECES + c / 4 + hf * 2) * 512;
                const float4 y0 = *reinterpret_cast<const float4*>(at), y1 = *reinterpret_cast<const float4*>(at + 512);
                const float y[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const float f = fm[2 * hf + ((e >> 1) & 1)], g = ft[2 * hf + ((e >> 1) & 1)];
                  o[e] = TOKEN ? o[e] * f * f + y[e] * g * g : o[e] * f + y[e] * g;
                }
                store16(o, hf, keep + c);
              }
          }
          // both go on when the boxes are read: they are filled again, or with the next segment's Q
          mbar_arrive(half_empty);
          ok = mbar_wait<true>(half_empty, (uint32_t)hn & 1u, abort_flag, g.status, FP_DEV_TIMEOUT);
          if (!ok) break;
          ++hn;
        }
        if (!ok) break;
        if (w == 0) store_lse(top, sum);
      }
      tc_fence_before();
      tn += nt;
      ++segment;
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

template <bool E4M3, bool TOKEN, int D, bool PAIR>
cudaError_t run(const TreeArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t s) {
  using C = Cfg<E4M3, D, PAIR>;
  auto kern = wide_kernel<E4M3, TOKEN, D, PAIR>;
  // more than half of the SM's shared memory: one CTA per SM, so that the
  // 512-column TMEM allocation never waits for a co-resident CTA
  const int want = C::SMEM_FIXED + axis_bytes(a.g.R), smem = want > 120 * 1024 ? want : 120 * 1024;
  static std::atomic<unsigned long long> prepared{0};
  const cudaError_t e = prepare(kern, (int)Roles<E4M3>::LAUNCH_REGS, prepared);
  if (e != cudaSuccess) return e;
  kern<<<a.grid, Roles<E4M3>::THREADS, smem, s>>>(mk, mv, a);
  return cudaGetLastError();
}

template <bool E4M3, bool TOKEN, int D>
cudaError_t run_rows(const TreeArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t s) {
  return a.rows > 128 ? run<E4M3, TOKEN, D, true>(a, mk, mv, s) : run<E4M3, TOKEN, D, false>(a, mk, mv, s);
}

}  // namespace

cudaError_t launch_wide(const TreeArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t s) {
  if (a.g.e4m3) return a.g.token_scale ? run_rows<true, true, 128>(a, mk, mv, s) : run_rows<true, false, 128>(a, mk, mv, s);
  return a.g.d == 128 ? run_rows<false, false, 128>(a, mk, mv, s) : run_rows<false, false, 64>(a, mk, mv, s);
}

}  // namespace tree
}  // namespace fp
