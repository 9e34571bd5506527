// Internal definitions of the paged cache and the decoding steps over it.
#pragma once

#include "internal.cuh"

namespace fp {

// The status word (FP_DEV_*) of the current device; nullptr on a runtime error.
unsigned* status_ptr();

// SMs of the current device (at most 256: the combining kernel's registers).
int sm_count();

// encode_tiled with another L2 promotion than 256 bytes.
bool encode_tiled(CUtensorMap* map, CUtensorMapDataType type, int rank, const void* base, const cuuint64_t* dims,
                  const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapL2promotion promotion);

// Validated geometry of a paged cache (fp_cache_t).
struct CacheGeometry {
  int R, Hkv, d;
  int e4m3;        // pools hold e4m3 codes (else bf16)
  int token_scale; // FP_SCALE_TOKEN
  int page_size, page_shift, max_pages, num_pages;
  uint8_t* k_pool;
  uint8_t* v_pool;
  float* k_scale;
  float* v_scale;
  const int32_t* table;
  const int32_t* kv_lens;
  const int32_t* cu;   // cu_tokens
  int total_tokens;
  unsigned* status;
};

// Rows, new tokens and cached length of request r; false (n = 0) when the
// request's arrays do not fit, with FP_DEV_BAD_SEQLENS set.
// READ_ONLY: the kernel does not write kv_lens (fp_cache_commit may).
template <bool READ_ONLY = false>
__device__ __forceinline__ bool cache_span(const CacheGeometry& g, int r, int& off, int& n, int& kv) {
  const int a = __ldg(g.cu + r), b = __ldg(g.cu + r + 1);
  kv = READ_ONLY ? __ldg(g.kv_lens + r) : __ldcg(g.kv_lens + r);
  off = a;
  n = b - a;
  if (a < 0 || n < 0 || b > g.total_tokens || n > kv || kv > (long long)g.max_pages * g.page_size) {
    atomicOr(g.status, FP_DEV_BAD_SEQLENS);
    n = 0;
    return false;
  }
  return true;
}

cudaError_t launch_cache_write(const CacheGeometry& g, const void* k, long long k_stride, const void* v,
                               long long v_stride, cudaStream_t s);
cudaError_t launch_cache_read(const CacheGeometry& g, const int32_t* starts, void* k, long long k_stride, void* v,
                              long long v_stride, cudaStream_t s);
cudaError_t launch_cache_commit(const CacheGeometry& g, const int32_t* accept, const int32_t* num_accept,
                                int max_accept, int32_t* new_lens, cudaStream_t s);
size_t tree_workspace(const CacheGeometry& g, int hq, int max_tokens);
fp_status_t launch_tree(const CacheGeometry& g, const fp_tree_t& t, const void* q, void* o, float* lse, void* ws,
                        cudaStream_t s);

}  // namespace fp
