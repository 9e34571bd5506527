// C ABI of the paged cache and the attention over it: argument validation and
// launches on the caller's stream.
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>

#include "cache.cuh"

namespace fp {

namespace {

constexpr int kMaxRequests = 4096;
constexpr int kMaxHeads = 256;
constexpr int kMaxNewTokens = 1024;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

fp_status_t cuda_fail(const char* step, cudaError_t e) {
  set_last_error(step, (int)e, cudaGetErrorString(e));
  return FP_ERR_CUDA;
}

// Everything about the cache that needs no device.
fp_status_t validate_cache(const fp_cache_t* c) {
  if (!c) return FP_ERR_INVALID_ARG;
  if (c->dtype != FP_BF16 && c->dtype != FP_E4M3) return FP_ERR_INVALID_ARG;
  if (c->scale != FP_SCALE_NONE && c->scale != FP_SCALE_HEAD && c->scale != FP_SCALE_TOKEN) return FP_ERR_INVALID_ARG;
  if ((c->dtype == FP_BF16) != (c->scale == FP_SCALE_NONE)) return FP_ERR_INVALID_ARG;
  if (c->batch < 1 || c->hkv < 1 || c->num_pages < 1 || c->max_pages_per_req < 1) return FP_ERR_INVALID_ARG;
  if (c->batch > kMaxRequests || c->hkv > kMaxHeads) return FP_ERR_UNSUPPORTED;
  if (c->head_dim != 128 && !(c->head_dim == 64 && c->dtype == FP_BF16)) return FP_ERR_UNSUPPORTED;
  const int P = c->page_size;
  if (P < 16 || P > 65536 || (P & (P - 1)) != 0) return FP_ERR_UNSUPPORTED;
  if ((long long)c->max_pages_per_req * P > INT_MAX) return FP_ERR_UNSUPPORTED;  // int positions
  if (!c->k_pool || !c->v_pool || !c->page_table || !c->kv_lens) return FP_ERR_INVALID_ARG;
  if (c->dtype == FP_E4M3 && (!c->k_scale || !c->v_scale)) return FP_ERR_INVALID_ARG;
  if (!aligned(c->k_pool, 16) || !aligned(c->v_pool, 16) || !aligned(c->k_scale, 16) || !aligned(c->v_scale, 16) ||
      !aligned(c->page_table, 4) || !aligned(c->kv_lens, 4))
    return FP_ERR_ALIGNMENT;
  return FP_OK;
}

fp_status_t validate_new_tokens(const int32_t* cu_tokens, int total_tokens) {
  if (!cu_tokens || total_tokens < 0) return FP_ERR_INVALID_ARG;
  return aligned(cu_tokens, 4) ? FP_OK : FP_ERR_ALIGNMENT;
}

// Packed K and V rows of fp_cache_write / fp_cache_read.
fp_status_t validate_rows(const fp_cache_t* c, const void* k, long long k_stride, const void* v, long long v_stride) {
  const long long row = (long long)c->hkv * c->head_dim;
  if (!k || !v || k_stride < row || v_stride < row) return FP_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || k_stride % 8 != 0 || v_stride % 8 != 0) return FP_ERR_ALIGNMENT;
  return FP_OK;
}

CacheGeometry geometry(const fp_cache_t* c, const int32_t* cu_tokens, int total_tokens) {
  CacheGeometry g;
  g.R = c->batch;
  g.Hkv = c->hkv;
  g.d = c->head_dim;
  g.e4m3 = c->dtype == FP_E4M3;
  g.token_scale = c->scale == FP_SCALE_TOKEN;
  g.page_size = c->page_size;
  g.page_shift = 0;
  while ((1 << g.page_shift) < g.page_size) ++g.page_shift;
  g.max_pages = c->max_pages_per_req;
  g.num_pages = c->num_pages;
  g.k_pool = static_cast<uint8_t*>(c->k_pool);
  g.v_pool = static_cast<uint8_t*>(c->v_pool);
  g.k_scale = c->k_scale;
  g.v_scale = c->v_scale;
  g.table = c->page_table;
  g.kv_lens = c->kv_lens;
  g.cu = cu_tokens;
  g.total_tokens = total_tokens;
  g.status = nullptr;
  return g;
}

fp_status_t validate_tree(const fp_cache_t* c, const fp_tree_t* t) {
  if (!t) return FP_ERR_INVALID_ARG;
  if (t->hq < 1 || t->hq % c->hkv != 0 || t->total_tokens < 0 || t->max_tokens < 1) return FP_ERR_INVALID_ARG;
  if (!std::isfinite(t->softmax_scale) || t->softmax_scale < 0.f) return FP_ERR_INVALID_ARG;
  const int G = t->hq / c->hkv;
  if (!(G <= 8 || G == 16) || t->max_tokens > kMaxNewTokens) return FP_ERR_UNSUPPORTED;
  if ((long long)t->total_tokens * t->hq > INT_MAX) return FP_ERR_UNSUPPORTED;
  // positions are rounded up to whole tiles in an int
  if ((long long)c->max_pages_per_req * c->page_size > INT_MAX - 1024) return FP_ERR_UNSUPPORTED;
  // the axis of all tiles (and up to 8 places before a unit's) is counted in an int
  const long long tiles = ((long long)c->max_pages_per_req * c->page_size + 127) / 128 + 8;
  const long long units = ((long long)t->max_tokens * G + 15) / 16 * c->hkv * c->batch;
  if (tiles > (INT_MAX / 2) / units) return FP_ERR_UNSUPPORTED;
  if (t->mask && t->mask_words < (t->max_tokens + 31) / 32) return FP_ERR_INVALID_ARG;
  if (t->q_stride != 0) {
    if (t->q_stride < (long long)t->hq * c->head_dim) return FP_ERR_INVALID_ARG;
    if (t->q_stride % 8 != 0) return FP_ERR_ALIGNMENT;
  }
  return FP_OK;
}

}  // namespace

int sm_count() {
  static std::atomic<int> counts[64];  // per device, 0: not asked yet
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (dev < 64 && (n = counts[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 148;
  n = n < 256 ? n : 256;
  if (dev < 64) counts[dev].store(n, std::memory_order_relaxed);
  return n;
}

}  // namespace fp

using namespace fp;

extern "C" {

fp_status_t fp_cache_write(const fp_cache_t* c, const int32_t* cu_tokens, int total_tokens, const void* k,
                           long long k_stride, const void* v, long long v_stride, void* stream) {
  fp_status_t st = validate_cache(c);
  if (st == FP_OK) st = validate_new_tokens(cu_tokens, total_tokens);
  if (st != FP_OK) return st;
  if (total_tokens == 0) return FP_OK;
  if ((st = validate_rows(c, k, k_stride, v, v_stride)) != FP_OK) return st;
  CacheGeometry g = geometry(c, cu_tokens, total_tokens);
  if (!(g.status = status_ptr())) return cuda_fail("device status symbol", cudaGetLastError());
  const cudaError_t e = launch_cache_write(g, k, k_stride, v, v_stride, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FP_OK : cuda_fail("cache write launch", e);
}

fp_status_t fp_cache_read(const fp_cache_t* c, const int32_t* cu_tokens, int total_tokens, const int32_t* starts,
                          void* k, long long k_stride, void* v, long long v_stride, void* stream) {
  fp_status_t st = validate_cache(c);
  if (st == FP_OK) st = validate_new_tokens(cu_tokens, total_tokens);
  if (st != FP_OK) return st;
  if (starts && !aligned(starts, 4)) return FP_ERR_ALIGNMENT;
  if (total_tokens == 0) return FP_OK;
  if ((st = validate_rows(c, k, k_stride, v, v_stride)) != FP_OK) return st;
  CacheGeometry g = geometry(c, cu_tokens, total_tokens);
  if (!(g.status = status_ptr())) return cuda_fail("device status symbol", cudaGetLastError());
  const cudaError_t e = launch_cache_read(g, starts, k, k_stride, v, v_stride, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FP_OK : cuda_fail("cache read launch", e);
}

fp_status_t fp_cache_commit(const fp_cache_t* c, const int32_t* cu_tokens, int total_tokens, const int32_t* accept,
                            const int32_t* num_accept, int max_accept, int32_t* new_lens, void* stream) {
  fp_status_t st = validate_cache(c);
  if (st == FP_OK) st = validate_new_tokens(cu_tokens, total_tokens);
  if (st != FP_OK) return st;
  if (!num_accept || !new_lens || max_accept < 0 || (max_accept > 0 && !accept)) return FP_ERR_INVALID_ARG;
  if (max_accept > kMaxNewTokens) return FP_ERR_UNSUPPORTED;
  if (!aligned(accept, 4) || !aligned(num_accept, 4) || !aligned(new_lens, 4)) return FP_ERR_ALIGNMENT;
  CacheGeometry g = geometry(c, cu_tokens, total_tokens);
  if (!(g.status = status_ptr())) return cuda_fail("device status symbol", cudaGetLastError());
  const cudaError_t e =
      launch_cache_commit(g, accept, num_accept, max_accept, new_lens, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FP_OK : cuda_fail("cache commit launch", e);
}

size_t fp_tree_workspace_size(const fp_cache_t* c, const fp_tree_t* t) {
  if (validate_cache(c) != FP_OK || validate_tree(c, t) != FP_OK) return 0;
  return tree_workspace(geometry(c, nullptr, 0), t->hq, t->max_tokens);
}

fp_status_t fp_tree_attention(const fp_cache_t* c, const fp_tree_t* t, const void* q, void* o, float* lse,
                              void* workspace, size_t ws_bytes, void* stream) {
  fp_status_t st = validate_cache(c);
  if (st == FP_OK) st = validate_tree(c, t);
  if (st == FP_OK) st = validate_new_tokens(t->cu_tokens, t->total_tokens);
  if (st != FP_OK) return st;
  if (t->total_tokens == 0) return FP_OK;
  if (!q || !o) return FP_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(t->mask, 4) || !aligned(lse, 4)) return FP_ERR_ALIGNMENT;
  CacheGeometry g = geometry(c, t->cu_tokens, t->total_tokens);
  if (!workspace || !aligned(workspace, 256) || ws_bytes < tree_workspace(g, t->hq, t->max_tokens))
    return FP_ERR_WORKSPACE;
  // CTAs write rows of o while others still read q
  const long long row = (long long)t->hq * c->head_dim, rows = t->total_tokens - 1;
  const uintptr_t q0 = reinterpret_cast<uintptr_t>(q), o0 = reinterpret_cast<uintptr_t>(o);
  const uintptr_t q_bytes = 2 * (rows * (t->q_stride ? t->q_stride : row) + row), o_bytes = 2 * (rows + 1) * row;
  if (o0 < q0 + q_bytes && q0 < o0 + o_bytes) return FP_ERR_INVALID_ARG;
  if (!(g.status = status_ptr())) return cuda_fail("device status symbol", cudaGetLastError());
  return launch_tree(g, *t, q, o, lse, workspace, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
