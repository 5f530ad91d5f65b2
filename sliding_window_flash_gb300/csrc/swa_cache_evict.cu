// swa_cache_evict.cu — cuts a paged cache to a budget by accumulated attention weight.
//
// Two kernels.  The first chooses, one block per (sequence, kv head): the (budget - recent)-th
// largest weight of the older tokens by a radix selection over the weights' ordered bits (four
// passes of 8 bits, a histogram each), then the survivors in slot order by a running count: all
// above the threshold, the recent ones, and the first of those equal to it.  The second moves: one
// block per (destination page, kv head, sequence), whose scales are the largest of its tokens'.
#include <cuda_fp8.h>

#include "swa_cache_kernels.h"
#include "swa_ptx.cuh"

namespace swa {
namespace {

constexpr int kSelectThreads = 1024;
constexpr int kMoveThreads = 256;

// Bits that order like the floats: negatives reversed, -0 as 0, NaN on top (its sign is ignored).
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kSelectThreads)
    swa_evict_select_kernel(const CacheView c, const CacheEvictArgs a) {
  __shared__ unsigned s_hist[256];
  __shared__ unsigned s_pick, s_want;
  __shared__ int s_warp[32];
  const int h = static_cast<int>(blockIdx.x), b = static_cast<int>(blockIdx.y);
  const int tid = static_cast<int>(threadIdx.x);
  int* kept = a.kept + (static_cast<size_t>(b) * c.Hkv + h) * a.budget;
  int len, n;
  const bool ok = sequence_of(c, b, &len, &n);
  if (!ok) len = 0;
  const int m = min(len, a.budget);
  if (h == 0 && tid == 0) a.lens_out[b] = m;
  for (int i = m + tid; i < a.budget; i += kSelectThreads) kept[i] = -1;
  if (len <= a.budget) {
    for (int i = tid; i < len; i += kSelectThreads) kept[i] = i;
    return;
  }
  const int old = len - a.recent;            // tokens that compete
  unsigned want = static_cast<unsigned>(a.budget - a.recent);  // of which this many stay
  auto key_of = [&](int s) -> uint32_t {
    const int page = page_of(c, c.table, b, s / c.page, c.max_pages);
    if (page < 0) return 0u;
    return ordered(c.weight[(static_cast<size_t>(page) * c.Hkv + h) * c.page + s % c.page]);
  };
  uint32_t prefix = 0, mask = 0;
  if (want > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += kSelectThreads) s_hist[i] = 0;
      __syncthreads();
      for (int s = tid; s < old; s += kSelectThreads) {
        const uint32_t k = key_of(s);
        if ((k & mask) == prefix) atomicAdd(&s_hist[(k >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (tid == 0) {
        unsigned left = want;
        int i = 255;
        while (i > 0 && s_hist[i] < left) left -= s_hist[i--];
        s_pick = static_cast<unsigned>(i);
        s_want = left;
      }
      __syncthreads();
      prefix |= s_pick << shift;
      mask |= 255u << shift;
      want = s_want;
      __syncthreads();
    }
  }
  // `prefix` is the smallest key that stays; of the tokens that have it, the first `want`.
  int done = 0, ties = 0;
  const int warp = tid >> 5, lane = tid & 31;
  for (int s0 = 0; s0 < len; s0 += kSelectThreads) {
    const int s = s0 + tid;
    const bool late = s >= old && s < len;
    const uint32_t k = s < old ? key_of(s) : 0u;
    const bool some = a.budget > a.recent;
    const bool above = s < old && some && k > prefix, tie = s < old && some && k == prefix;
    const unsigned tb = __ballot_sync(0xffffffffu, tie);
    if (lane == 0) s_warp[warp] = __popc(tb);
    __syncthreads();
    int before = ties, all = 0;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) before += s_warp[w];
      all += s_warp[w];
    }
    before += __popc(tb & ((1u << lane) - 1u));
    ties += all;
    __syncthreads();
    const bool stay = late || above || (tie && before < static_cast<int>(want));
    const unsigned sb = __ballot_sync(0xffffffffu, stay);
    if (lane == 0) s_warp[warp] = __popc(sb);
    __syncthreads();
    int at = done;
    all = 0;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) at += s_warp[w];
      all += s_warp[w];
    }
    at += __popc(sb & ((1u << lane) - 1u));
    done += all;
    __syncthreads();
    if (stay && at < a.budget) kept[at] = s;
  }
}

__device__ __forceinline__ uint32_t rescale4(uint32_t u, float r) {
  float x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half_raw hr = __nv_cvt_fp8_to_halfraw(
        static_cast<__nv_fp8_storage_t>((u >> (8 * i)) & 0xffu), __NV_E4M3);
    x[i] = __half2float(*reinterpret_cast<const __half*>(&hr)) * r;
  }
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[0], x[1]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[2], x[3]), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

__global__ void __launch_bounds__(kMoveThreads)
    swa_evict_move_kernel(const CacheView c, const CacheEvictArgs a) {
  __shared__ long long s_row[128];       // source row (token) of the pool, or -1
  __shared__ float s_k[128], s_v[128];   // its scales, then their ratio to the block's
  const int h = static_cast<int>(blockIdx.y), b = static_cast<int>(blockIdx.z);
  const int j0 = static_cast<int>(blockIdx.x) * c.page;
  const int m = min(a.lens_out[b], a.budget);
  const int rows = min(c.page, m - j0);
  if (rows <= 0) return;
  const int to = page_of(c, a.dst_table, b, static_cast<int>(blockIdx.x), a.dst_pages);
  if (to < 0) return;
  const size_t block = static_cast<size_t>(to) * c.Hkv + h;
  const int* kept = a.kept + (static_cast<size_t>(b) * c.Hkv + h) * a.budget + j0;
  const int tid = static_cast<int>(threadIdx.x);
  if (tid < rows) {
    const int s = kept[tid];
    const int page = page_of(c, c.table, b, s / c.page, c.max_pages);
    const size_t from = static_cast<size_t>(max(page, 0)) * c.Hkv + h;
    s_row[tid] = page < 0 ? -1 : static_cast<long long>(from * c.page + s % c.page);
    s_k[tid] = page < 0 ? 0.f : c.k_scale[from];
    s_v[tid] = page < 0 ? 0.f : c.v_scale[from];
  }
  __syncthreads();
  float ks = 0.f, vs = 0.f;
  for (int i = 0; i < rows; ++i) {
    ks = fmaxf(ks, s_k[i]);
    vs = fmaxf(vs, s_v[i]);
  }
  if (tid == 0 && ks > 0.f) {
    c.k_scale[block] = ks;
    c.v_scale[block] = vs;
  }
  if (tid < rows && s_row[tid] >= 0) c.weight[block * c.page + tid] = c.weight[s_row[tid]];
  const int units = c.D / 16;
  for (int i = tid; i < rows * units; i += kMoveThreads) {
    const int r = i / units, u = i % units;
    if (s_row[r] < 0) continue;
    const size_t from = static_cast<size_t>(s_row[r]) * c.D + u * 16;
    const size_t out = (block * c.page + r) * c.D + u * 16;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const float ratio = w == 0 ? s_k[r] / ks : s_v[r] / vs;
      uint4 x = *reinterpret_cast<const uint4*>((w == 0 ? c.k : c.v) + from);
      if (ratio != 1.f) {
        x.x = rescale4(x.x, ratio);
        x.y = rescale4(x.y, ratio);
        x.z = rescale4(x.z, ratio);
        x.w = rescale4(x.w, ratio);
      }
      *reinterpret_cast<uint4*>((w == 0 ? c.k : c.v) + out) = x;
    }
  }
}

}  // namespace

cudaError_t launch_cache_evict(const CacheView& c, const CacheEvictArgs& a, cudaStream_t stream) {
  swa_evict_select_kernel<<<dim3(static_cast<unsigned>(c.Hkv), static_cast<unsigned>(c.B)),
                            kSelectThreads, 0, stream>>>(c, a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>((a.budget + c.page - 1) / c.page),
                  static_cast<unsigned>(c.Hkv), static_cast<unsigned>(c.B));
  swa_evict_move_kernel<<<grid, kMoveThreads, 0, stream>>>(c, a);
  return cudaGetLastError();
}

}  // namespace swa
