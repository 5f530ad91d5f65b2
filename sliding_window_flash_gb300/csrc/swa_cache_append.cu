// swa_cache_append.cu — quantises new keys and values into the paged e4m3 cache.
//
// One block of threads owns one (sequence, page, kv head): it alone writes that block's codes,
// scales and weights.  It finds the largest |x| of the new keys and of the new values, takes
//   scale = max(old scale if older tokens share the block, least 2^e with max |x| <= 448 2^e),
// rounds the older codes to a raised scale, and writes the new codes x / scale (both scales are
// powers of two, so every product below is exact and each code is rounded once).
//
// Bandwidth-bound: 2 or 4 bytes in and one byte out per element.  Each lane takes 8 consecutive
// elements of four rows a quarter of a page apart, of keys and values, all on their way together, and
// keeps them until the scale is known; D / 8 lanes share a row, whose largest |x| is a shuffle
// reduction.  Elements of 16 bits are compared and multiplied two at a time: element by element the
// instructions bound it (77 us for 30,553 tokens, 16 heads, D = 128, bf16, where this takes 65 us,
// 5.8 TB/s).
#include <cuda_fp8.h>

#include "swa_cache_kernels.h"
#include "swa_ptx.cuh"

namespace swa {
namespace {

constexpr int kHeld = 4;  // rows that a lane holds; a block has page D / 32 threads

// Eight elements as they are stored, and as fp32.
template <int kDtype>
struct Eight {
  uint4 u;
  __device__ __forceinline__ void load(const void* base, size_t i) {
    u = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + i));
  }
  __device__ __forceinline__ void clear() { u = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
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
struct Eight<SWA_FP32> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* base, size_t i) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
    a = __ldcs(p);
    b = __ldcs(p + 1);
  }
  __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
};

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The largest |x| of a row's keys and of its values, as fp32 bits, in every lane of the row.  The bits
// of |x| order like the values, with infinity and NaN on top, in every type; 16-bit types are compared
// two at a time, keys and values in one word for the reduction across lanes.
template <int kDtype, int kLanes>
__device__ __forceinline__ uint2 largest(const Eight<kDtype>& k, const Eight<kDtype>& v) {
  if constexpr (kDtype == SWA_FP32) {
    float x[8], y[8];
    k.get(x);
    v.get(y);
    uint32_t mk = 0, mv = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      mk = max(mk, __float_as_uint(x[j]) & 0x7fffffffu);
      mv = max(mv, __float_as_uint(y[j]) & 0x7fffffffu);
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) {
      mk = max(mk, __shfl_xor_sync(0xffffffffu, mk, o));
      mv = max(mv, __shfl_xor_sync(0xffffffffu, mv, o));
    }
    return make_uint2(mk, mv);
  } else {
    const uint32_t m = 0x7fff7fffu;
    const uint32_t mk = max_u16x2(max_u16x2(k.u.x & m, k.u.y & m), max_u16x2(k.u.z & m, k.u.w & m));
    const uint32_t mv = max_u16x2(max_u16x2(v.u.x & m, v.u.y & m), max_u16x2(v.u.z & m, v.u.w & m));
    uint32_t both = max_u16x2(__byte_perm(mk, mv, 0x5410), __byte_perm(mk, mv, 0x7632));
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1)
      both = max_u16x2(both, __shfl_xor_sync(0xffffffffu, both, o));
    const float2 f = Elem<kDtype == SWA_FP16>::unpack(both);
    return make_uint2(__float_as_uint(f.x), __float_as_uint(f.y));
  }
}

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

// Eight elements times `inv`, a power of two that brings them to at most 448, as codes.  bf16 elements
// are multiplied as pairs, exactly.  fp16 ones as well while inv is within fp16's normal numbers
// (`direct`): a product that fp16 rounds is below 2^-14, and zero as a code either way.
template <int kDtype>
__device__ __forceinline__ uint2 quantise(const Eight<kDtype>& v, float inv, uint32_t inv2,
                                          bool direct) {
  if constexpr (kDtype != SWA_FP32) {
    const uint32_t r[4] = {v.u.x, v.u.y, v.u.z, v.u.w};
    uint32_t out[4];
    if (kDtype == SWA_FP16 && direct) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        asm("{\n\t.reg .b32 x;\n\t.reg .b16 a;\n\t"
            "mul.rn.f16x2 x, %1, %2;\n\t"
            "cvt.rn.satfinite.e4m3x2.f16x2 a, x;\n\t"
            "cvt.u32.u16 %0, a;\n\t}"
            : "=r"(out[j])
            : "r"(r[j]), "r"(inv2));
      return make_uint2(out[0] | out[1] << 16, out[2] | out[3] << 16);
    }
    if (kDtype == SWA_BF16) {
      float x[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t y;
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(r[j]), "r"(inv2));
        x[2 * j] = __uint_as_float(y << 16);
        x[2 * j + 1] = __uint_as_float(y & 0xffff0000u);
      }
      return make_uint2(e4m3x4(x[0], x[1], x[2], x[3]), e4m3x4(x[4], x[5], x[6], x[7]));
    }
  }
  float x[8];
  v.get(x);
  return make_uint2(e4m3x4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv),
                    e4m3x4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv));
}

// A power of two as a pair of the element type, and whether fp16 products with it are exact enough.
template <int kDtype>
__device__ __forceinline__ uint32_t pair_of(float x) {
  return Elem<kDtype == SWA_FP16>::pack(x, x);
}

// kKeep: the elements stay in registers; without it (fp32 in blocks of more than 512 threads, which
// have 64 registers each) they are read again when the scale is known.
template <int D, int kDtype, bool kKeep>
__global__ void __launch_bounds__(kKeep && kDtype == SWA_FP32 ? 512 : D * 4,
                                  kDtype == SWA_FP32 ? 1 : 256 / D)
    swa_cache_append_kernel(const CacheView c, const void* __restrict__ k,
                            const void* __restrict__ v, const float* __restrict__ weight) {
  constexpr int kLanes = D / 8;  // lanes of a row
  __shared__ uint32_t s_k[128], s_v[128];  // each new token's largest |x|, as bits
  __shared__ float s_scale[4];             // new scale and old / new ratio, of k and of v
  const int b = static_cast<int>(blockIdx.z), h = static_cast<int>(blockIdx.y);
  const int tid = static_cast<int>(threadIdx.x), threads = static_cast<int>(blockDim.x);
  int len, n;
  if (!sequence_of(c, b, &len, &n) || n == 0) return;
  const int blk = len / c.page + static_cast<int>(blockIdx.x);
  if (blk >= c.max_pages) return;  // behind the table, where slots may pass 31 bits
  const int slot0 = blk * c.page;
  const int first = max(len, slot0) - slot0;      // first new row of the block
  const int last = min(len + n - slot0, c.page);  // one past the last
  if (first >= last) return;
  // element offset of the block's row 0 in k and v, if it were a new token
  const long long src = ((static_cast<long long>(b) * c.Hkv + h) * c.T + slot0 - len) * D;
  const int sub = tid % kLanes, row0 = tid / kLanes, step = c.page / kHeld;
  const long long own = src + static_cast<long long>(row0) * D + sub * 8;
  Eight<kDtype> xk[kHeld], xv[kHeld];
#pragma unroll
  for (int e = 0; e < kHeld; ++e) {
    const int r = row0 + e * step;
    xk[e].clear();
    xv[e].clear();
    if (r >= first && r < last) {
      xk[e].load(k, static_cast<size_t>(own + e * step * D));
      xv[e].load(v, static_cast<size_t>(own + e * step * D));
    }
  }
  const int page = page_of(c, c.table, b, blk, c.max_pages);
  if (page < 0) return;
  const size_t block = static_cast<size_t>(page) * c.Hkv + h;
#pragma unroll
  for (int e = 0; e < kHeld; ++e) {
    const uint2 m = largest<kDtype, kLanes>(xk[e], xv[e]);
    if (sub == 0) {
      s_k[row0 + e * step] = m.x;
      s_v[row0 + e * step] = m.y;
    }
  }
  __syncthreads();
  if (tid < 32) {
    uint32_t mk = 0, mv = 0;
    for (int r = first + tid; r < last; r += 32) {
      if (max(s_k[r], s_v[r]) <= kLargestBits) {
        mk = max(mk, s_k[r]);
        mv = max(mv, s_v[r]);
      }
    }
    mk = __reduce_max_sync(0xffffffffu, mk);
    mv = __reduce_max_sync(0xffffffffu, mv);
    if (tid < 2) {
      float* held = tid == 0 ? c.k_scale + block : c.v_scale + block;
      float now = scale_for(tid == 0 ? mk : mv), ratio = 1.f;
      if (first > 0) {
        const float old = *held;
        now = fmaxf(now, old);
        ratio = old / now;
      }
      if (first == 0 || ratio != 1.f) *held = now;
      s_scale[tid] = now;
      s_scale[2 + tid] = ratio;
    }
  }
  __syncthreads();
  const float kinv = 1.f / s_scale[0], vinv = 1.f / s_scale[1];
  const uint32_t kinv2 = pair_of<kDtype>(kinv), vinv2 = pair_of<kDtype>(vinv);
  const bool direct = fminf(kinv, vinv) >= 0x1p-14f && fmaxf(kinv, vinv) <= 0x1p15f;
#pragma unroll
  for (int e = 0; e < kHeld; ++e) {
    const int r = row0 + e * step;
    if (r < first || r >= last) continue;
    const bool bad = max(s_k[r], s_v[r]) > kLargestBits;
    if (!kKeep) {
      xk[e].load(k, static_cast<size_t>(own + e * step * D));
      xv[e].load(v, static_cast<size_t>(own + e * step * D));
    }
    const size_t out = (block * c.page + r) * D + sub * 8;
    *reinterpret_cast<uint2*>(c.k + out) =
        bad ? make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu) : quantise(xk[e], kinv, kinv2, direct);
    *reinterpret_cast<uint2*>(c.v + out) = bad ? make_uint2(0u, 0u) : quantise(xv[e], vinv, vinv2, direct);
  }
#pragma unroll
  for (int w = 0; w < 2; ++w) {  // older codes, where the scale rose
    const float ratio = s_scale[2 + w];
    if (ratio == 1.f) continue;
    const uint32_t times = half2_of(ratio);
    uint4* codes = reinterpret_cast<uint4*>((w == 0 ? c.k : c.v) + block * c.page * D);
    for (int i = tid; i < first * D / 16; i += threads) {
      const uint4 u = codes[i];
      codes[i] = make_uint4(e4m3x4_times(u.x, times), e4m3x4_times(u.y, times),
                            e4m3x4_times(u.z, times), e4m3x4_times(u.w, times));
    }
  }
  if (c.weight != nullptr) {
    const long long wsrc = (static_cast<long long>(b) * c.Hkv + h) * c.T + slot0 - len;
    for (int r = first + tid; r < last; r += threads)
      c.weight[block * c.page + r] = weight != nullptr ? weight[wsrc + r] : 0.f;
  }
}

template <int D>
cudaError_t launch_d(const CacheView& c, const void* k, const void* v, const float* weight,
                     int dtype, cudaStream_t stream) {
  // T tokens touch at most this many pages of a sequence.
  const dim3 grid((static_cast<unsigned>(c.T) + c.page - 2) / c.page + 1,
                  static_cast<unsigned>(c.Hkv), static_cast<unsigned>(c.B));
  const unsigned threads = static_cast<unsigned>(c.page * D / (8 * kHeld));
  if (dtype == SWA_BF16)
    swa_cache_append_kernel<D, SWA_BF16, true><<<grid, threads, 0, stream>>>(c, k, v, weight);
  else if (dtype == SWA_FP16)
    swa_cache_append_kernel<D, SWA_FP16, true><<<grid, threads, 0, stream>>>(c, k, v, weight);
  else if (threads <= 512)
    swa_cache_append_kernel<D, SWA_FP32, true><<<grid, threads, 0, stream>>>(c, k, v, weight);
  else
    swa_cache_append_kernel<D, SWA_FP32, false><<<grid, threads, 0, stream>>>(c, k, v, weight);
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
