// swa_cache_kernels.h — launch interface between the cache calls of the C ABI (swa_cache_api.cu) and
// their kernels, and the device helpers those kernels share.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "swa_attn.h"
#include "swa_cache.h"
#include "swa_kernels.h"

namespace swa {

// Capability check and error-word address of the current device (swa_api.cu).
swa_status device_error_word(unsigned** err);

constexpr int kMaxCacheQueries = 64;  // T of swa_cache_attn

// Exponent range of a block's scale.  Its ends bound every product of a code and a ratio of two
// scales (2^88) times 2^20 tokens below fp32's range, and 448 * 2^40 is far above any activation.
constexpr int kScaleMinExp = -48;
constexpr int kScaleMaxExp = 40;

// The cache and the tables that lead into it, as every cache kernel sees them.
struct CacheView {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  float* weight;  // may be null
  int pages, Hkv, page, D;
  const int* table;  // [B, max_pages]
  int max_pages;
  const int* lens;      // [B], tokens cached before the step
  const int* new_lens;  // [B] or null (every sequence has T)
  int B, T;
  unsigned* err;
};

#ifdef __CUDACC__

__device__ __forceinline__ void raise_index_error(const CacheView& c) {
  atomicOr(c.err, kErrIndex);
}

// Tokens cached before and new tokens of sequence b; false (and the error bit) when they do not fit
// the table.
__device__ __forceinline__ bool sequence_of(const CacheView& c, int b, int* len, int* n) {
  const int l = c.lens[b];
  const int m = c.new_lens ? c.new_lens[b] : c.T;
  *len = l;
  *n = m;
  const bool ok = l >= 0 && m >= 0 && m <= c.T &&
                  static_cast<long long>(l) + m <= static_cast<long long>(c.max_pages) * c.page;
  if (!ok) raise_index_error(c);
  return ok;
}

// Page of block `i` of sequence b, or -1 (and the error bit) when the table names none; i must be
// inside the table.
__device__ __forceinline__ int page_of(const CacheView& c, const int* table, int b, int i,
                                       int max_pages) {
  const int p = table[static_cast<size_t>(b) * max_pages + i];
  if (p >= 0 && p < c.pages) return p;
  raise_index_error(c);
  return -1;
}

#endif  // __CUDACC__

cudaError_t launch_cache_append(const CacheView& c, const void* k, const void* v,
                                const float* weight, int dtype, cudaStream_t stream);

struct CacheAttnArgs {
  const void* q;
  void* o;
  float* lse;
  int Hq, window;
  float scale;
  int accumulate, dtype;
  void* workspace;
};
size_t cache_attn_workspace_bytes(int B, int Hq, int Hkv, int T, int D, int max_pages, int page,
                                  int accumulate);
cudaError_t launch_cache_attn(const CacheView& c, const CacheAttnArgs& a, cudaStream_t stream);

struct CacheEvictArgs {
  const int* dst_table;
  int dst_pages, budget, recent;
  int* kept;
  int* lens_out;
};
cudaError_t launch_cache_evict(const CacheView& c, const CacheEvictArgs& a, cudaStream_t stream);

size_t key_weights_workspace_bytes(const Problem& pb);
cudaError_t launch_key_weights(const Problem& pb, const void* q, const void* k, const float* lse,
                               float* w, void* workspace, cudaStream_t stream);

}  // namespace swa
