// swa_cache_kernels.h — launch interface between the cache calls of the C ABI (swa_cache_api.cu) and
// their kernels, and the device helpers those kernels share.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "swa_attn.h"
#include "swa_cache.h"
#include "swa_kernels.h"
#ifdef __CUDACC__
#include "swa_ptx.cuh"
#endif

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
// the table.  kL2: as load_global (swa_ptx.cuh).
template <bool kL2 = false>
__device__ __forceinline__ bool sequence_of(const CacheView& c, int b, int* len, int* n) {
  const int l = load_global<kL2>(c.lens + b);
  const int m = c.new_lens ? load_global<kL2>(c.new_lens + b) : c.T;
  *len = l;
  *n = m;
  const bool ok = l >= 0 && m >= 0 && m <= c.T &&
                  static_cast<long long>(l) + m <= static_cast<long long>(c.max_pages) * c.page;
  if (!ok) raise_index_error(c);
  return ok;
}

// Page of block `i` of sequence b, or -1 (and the error bit) when the table names none; i must be
// inside the table.
template <bool kL2 = false>
__device__ __forceinline__ int page_of(const CacheView& c, const int* table, int b, int i,
                                       int max_pages) {
  const int p = load_global<kL2>(table + static_cast<size_t>(b) * max_pages + i);
  if (p >= 0 && p < c.pages) return p;
  raise_index_error(c);
  return -1;
}

// Four e4m3 codes times `ratio` (two equal halves), a power of two of at most 1, rounded to nearest
// even.  fp16 holds codes exactly, and a product that it rounds (below 2^-20) is zero as a code; a
// ratio that it rounds to zero takes every code below half the least one.
__device__ __forceinline__ uint32_t e4m3x4_times(uint32_t codes, uint32_t ratio) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\t.reg .b32 x, y;\n\t"
      "mov.b32 {a, b}, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 x, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 y, b;\n\t"
      "mul.rn.f16x2 x, x, %2;\n\t"
      "mul.rn.f16x2 y, y, %2;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 a, x;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 b, y;\n\t"
      "mov.b32 %0, {a, b};\n\t}"
      : "=r"(r)
      : "r"(codes), "r"(ratio));
  return r;
}
// Codes 0, 1 (low half) and 2, 3 (high half) of a word as two fp16 pairs.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ uint32_t half2_of(float x) {
  const __half2 h = __float2half2_rn(x);
  return *reinterpret_cast<const uint32_t*>(&h);
}

#endif  // __CUDACC__

cudaError_t launch_cache_append(const CacheView& c, const void* k, const void* v,
                                const float* weight, int dtype, cudaStream_t stream);

struct CacheAttnArgs {
  const void* q;
  void* o;
  float* lse;
  int Hq, window, sinks;
  int base;  // slots of the shared prefix
  float scale;
  int accumulate, dtype;
  void* workspace;
};
size_t cache_attn_workspace_bytes(int B, int Hq, int Hkv, int T, int D, int max_pages, int page,
                                  int window, int sinks, int base, int accumulate);
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
