// swa_cache_append.cu — quantises new keys and values into the paged e4m3 cache.
//
// One block of threads owns one (sequence, page, kv head): it alone writes that block's codes,
// scales and weights.  It finds the largest |x| of the new keys and of the new values, takes
//   scale = max(old scale if older tokens share the block, least 2^e with max |x| <= 448 2^e),
// rounds the older codes to a raised scale, and writes the new codes x / scale (both scales are
// powers of two, so every product below is exact and each code is rounded once).
//
// Bandwidth-bound: 2 or 4 bytes in and one byte out per element.  Each lane takes 8 consecutive
// elements, D / 8 lanes a token's row, whose largest |x| is a shuffle reduction; the elements are
// read again from the L2 for the conversion.
#include <cuda_fp8.h>

#include "swa_cache_kernels.h"
#include "swa_ptx.cuh"

namespace swa {
namespace {

constexpr int kAppendThreads = 256;

// Eight elements as fp32.
template <int kDtype>
struct Load8 {
  static __device__ __forceinline__ void get(const void* base, size_t i, float (&x)[8]) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + i));
    const uint32_t r[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = Elem<kDtype == SWA_FP16>::unpack(r[j]);
      x[2 * j] = f.x;
      x[2 * j + 1] = f.y;
    }
  }
};
template <>
struct Load8<SWA_FP32> {
  static __device__ __forceinline__ void get(const void* base, size_t i, float (&x)[8]) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
};

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// 2^e for the least e in range with amax <= 448 2^e = 1.75 2^(e + 8); `bits` is amax as fp32 bits.
__device__ __forceinline__ float scale_for(uint32_t bits) {
  int e = static_cast<int>(bits >> 23) - 127 - 8;  // subnormal amax: far below the range's end
  if ((bits & 0x7fffffu) > 0x600000u) ++e;         // mantissa above 1.75
  e = max(kScaleMinExp, min(kScaleMaxExp, e));
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// |x| above this (448 * 2^40), infinite or NaN: as fp32 bits of |x|, which order like the values
// with infinity and NaN on top.
constexpr uint32_t kLargestBits = (static_cast<uint32_t>(127 + 8 + kScaleMaxExp) << 23) | 0x600000u;

template <int D, int kDtype>
__global__ void __launch_bounds__(kAppendThreads)
    swa_cache_append_kernel(const CacheView c, const void* __restrict__ k,
                            const void* __restrict__ v, const float* __restrict__ weight) {
  constexpr int kLanes = D / 8;  // lanes of a row
  constexpr int kRows = kAppendThreads / kLanes;
  __shared__ uint32_t s_k[128], s_v[128];  // each new token's largest |x|, as bits
  __shared__ float s_scale[4];             // new scale and old / new ratio, of k and of v
  const int b = static_cast<int>(blockIdx.z), h = static_cast<int>(blockIdx.y);
  int len, n;
  if (!sequence_of(c, b, &len, &n) || n == 0) return;
  const int blk = len / c.page + static_cast<int>(blockIdx.x);
  const int slot0 = blk * c.page;
  const int first = max(len, slot0) - slot0;             // first new row of the block
  const int last = min(len + n - slot0, c.page);         // one past the last
  if (first >= last) return;
  const int page = page_of(c, c.table, b, blk, c.max_pages);
  if (page < 0) return;
  const size_t block = static_cast<size_t>(page) * c.Hkv + h;
  // element offset of the block's row 0 in k and v, if it were a new token
  const long long src = ((static_cast<long long>(b) * c.Hkv + h) * c.T + slot0 - len) * D;
  const int sub = static_cast<int>(threadIdx.x) % kLanes, row0 = static_cast<int>(threadIdx.x) / kLanes;

  for (int r0 = first; r0 < last; r0 += kRows) {
    const int r = r0 + row0;
    uint32_t mk = 0, mv = 0;
    if (r < last) {
      float x[8];
      Load8<kDtype>::get(k, static_cast<size_t>(src + static_cast<long long>(r) * D + sub * 8), x);
#pragma unroll
      for (int j = 0; j < 8; ++j) mk = max(mk, __float_as_uint(x[j]) & 0x7fffffffu);
      Load8<kDtype>::get(v, static_cast<size_t>(src + static_cast<long long>(r) * D + sub * 8), x);
#pragma unroll
      for (int j = 0; j < 8; ++j) mv = max(mv, __float_as_uint(x[j]) & 0x7fffffffu);
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) {
      mk = max(mk, __shfl_xor_sync(0xffffffffu, mk, o));
      mv = max(mv, __shfl_xor_sync(0xffffffffu, mv, o));
    }
    if (sub == 0 && r < last) {
      s_k[r] = mk;
      s_v[r] = mv;
    }
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    uint32_t mk = 0, mv = 0;
    for (int r = first + static_cast<int>(threadIdx.x); r < last; r += 32) {
      if (max(s_k[r], s_v[r]) <= kLargestBits) {
        mk = max(mk, s_k[r]);
        mv = max(mv, s_v[r]);
      }
    }
    mk = __reduce_max_sync(0xffffffffu, mk);
    mv = __reduce_max_sync(0xffffffffu, mv);
    if (threadIdx.x < 2) {
      float* held = threadIdx.x == 0 ? c.k_scale + block : c.v_scale + block;
      float now = scale_for(threadIdx.x == 0 ? mk : mv), ratio = 1.f;
      if (first > 0) {
        const float old = *held;
        now = fmaxf(now, old);
        ratio = old / now;
      }
      if (first == 0 || ratio != 1.f) *held = now;
      s_scale[threadIdx.x] = now;
      s_scale[2 + threadIdx.x] = ratio;
    }
  }
  __syncthreads();
  const float kinv = 1.f / s_scale[0], vinv = 1.f / s_scale[1];

#pragma unroll
  for (int w = 0; w < 2; ++w) {  // older codes, where the scale rose
    const float ratio = s_scale[2 + w];
    if (ratio == 1.f) continue;
    uint32_t* codes = reinterpret_cast<uint32_t*>((w == 0 ? c.k : c.v) + block * c.page * D);
    for (int i = static_cast<int>(threadIdx.x); i < first * D / 4; i += kAppendThreads) {
      codes[i] = e4m3x4_times(codes[i], half2_of(ratio));
    }
  }
  for (int r = first + row0; r < last; r += kRows) {
    const bool bad = max(s_k[r], s_v[r]) > kLargestBits;
    float x[8];
    const size_t at = static_cast<size_t>(src + static_cast<long long>(r) * D + sub * 8);
    uint2 ck = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu), cv = make_uint2(0u, 0u);
    if (!bad) {
      Load8<kDtype>::get(k, at, x);
      ck = make_uint2(e4m3x4(x[0] * kinv, x[1] * kinv, x[2] * kinv, x[3] * kinv),
                      e4m3x4(x[4] * kinv, x[5] * kinv, x[6] * kinv, x[7] * kinv));
      Load8<kDtype>::get(v, at, x);
      cv = make_uint2(e4m3x4(x[0] * vinv, x[1] * vinv, x[2] * vinv, x[3] * vinv),
                      e4m3x4(x[4] * vinv, x[5] * vinv, x[6] * vinv, x[7] * vinv));
    }
    const size_t out = (block * c.page + r) * D + sub * 8;
    *reinterpret_cast<uint2*>(c.k + out) = ck;
    *reinterpret_cast<uint2*>(c.v + out) = cv;
  }
  if (c.weight != nullptr) {
    const long long wsrc = (static_cast<long long>(b) * c.Hkv + h) * c.T + slot0 - len;
    for (int r = first + static_cast<int>(threadIdx.x); r < last; r += kAppendThreads)
      c.weight[block * c.page + r] = weight != nullptr ? weight[wsrc + r] : 0.f;
  }
}

template <int D>
cudaError_t launch_d(const CacheView& c, const void* k, const void* v, const float* weight,
                     int dtype, cudaStream_t stream) {
  // T tokens touch at most this many pages of a sequence.
  const dim3 grid(static_cast<unsigned>((c.T + c.page - 2) / c.page + 1),
                  static_cast<unsigned>(c.Hkv), static_cast<unsigned>(c.B));
  if (dtype == SWA_BF16)
    swa_cache_append_kernel<D, SWA_BF16><<<grid, kAppendThreads, 0, stream>>>(c, k, v, weight);
  else if (dtype == SWA_FP16)
    swa_cache_append_kernel<D, SWA_FP16><<<grid, kAppendThreads, 0, stream>>>(c, k, v, weight);
  else
    swa_cache_append_kernel<D, SWA_FP32><<<grid, kAppendThreads, 0, stream>>>(c, k, v, weight);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_append(const CacheView& c, const void* k, const void* v,
                                const float* weight, int dtype, cudaStream_t stream) {
  if (c.D == 64) return launch_d<64>(c, k, v, weight, dtype, stream);
  if (c.D == 128) return launch_d<128>(c, k, v, weight, dtype, stream);
  return launch_d<256>(c, k, v, weight, dtype, stream);
}

}  // namespace swa
