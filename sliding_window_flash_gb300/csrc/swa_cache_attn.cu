// swa_cache_attn.cu — attention of a few tokens per sequence over the paged e4m3 cache, and the
// accumulation of the weight each cached token received.
//
// First form: one block per (query, head, sequence); its warps take the visible slots in turn with
// an online softmax each, and join their sums in shared memory.
#include <cuda_fp8.h>

#include "swa_cache_kernels.h"
#include "swa_ptx.cuh"

namespace swa {
namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ float e4m3_value(uint32_t code) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(code), __NV_E4M3);
  return __half2float(*reinterpret_cast<const __half*>(&h));
}

template <int D, bool F16>
__device__ __forceinline__ float q_value(const void* q, size_t i) {
  const uint16_t u = static_cast<const uint16_t*>(q)[i];
  return Elem<F16>::unpack(u).x;
}

template <int D, bool F16>
__global__ void __launch_bounds__(kWarps * 32)
    swa_cache_attn_kernel(const CacheView c, const CacheAttnArgs a) {
  constexpr int E = D / 32;
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][D];
  const int t = static_cast<int>(blockIdx.x), hq = static_cast<int>(blockIdx.y);
  const int b = static_cast<int>(blockIdx.z);
  const int h = hq / (a.Hq / c.Hkv);
  const int warp = static_cast<int>(warp_id()), lane = static_cast<int>(lane_id());
  const size_t row = (static_cast<size_t>(b) * a.Hq + hq) * c.T + t;
  int len, n;
  const bool ok = sequence_of(c, b, &len, &n) && t < n;
  const int hi = ok ? len + t : -1, lo = max(0, hi - a.window + 1);
  float q[E], o[E] = {}, m = SWA_NEG_INF, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) q[e] = q_value<D, F16>(a.q, row * D + lane * E + e);
  for (int s = lo + warp; s <= hi; s += kWarps) {
    const int page = page_of(c, c.table, b, s / c.page, c.max_pages);
    if (page < 0) continue;
    const size_t block = static_cast<size_t>(page) * c.Hkv + h;
    const size_t at = (block * c.page + s % c.page) * D + lane * E;
    float x = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) x = fmaf(q[e], e4m3_value(c.k[at + e]), x);
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) x += __shfl_xor_sync(0xffffffffu, x, i);
    x *= a.scale * c.k_scale[block];
    const float top = fmaxf(m, x);  // NaN scores leave m and make the sum NaN below
    const float keep = m == top ? 1.f : expf(m - top), p = expf(x - top);
    const float pv = p * c.v_scale[block];
    l = l * keep + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * keep + pv * e4m3_value(c.v[at + e]);
    m = top;
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = o[e];
  __syncthreads();
  float top = SWA_NEG_INF, sum = 0.f;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w]);
  float f[kWarps];
  for (int w = 0; w < kWarps; ++w) {
    f[w] = s_l[w] == 0.f ? 0.f : (s_m[w] == top ? 1.f : expf(s_m[w] - top));
    sum += s_l[w] * f[w];
  }
  for (int d = static_cast<int>(threadIdx.x); d < D; d += kWarps * 32) {
    float acc = 0.f;
    for (int w = 0; w < kWarps; ++w) acc += s_o[w][d] * f[w];
    const float r = sum == 0.f ? 0.f : acc / sum;
    static_cast<uint16_t*>(a.o)[row * D + d] =
        static_cast<uint16_t>(Elem<F16>::pack(r, 0.f) & 0xffffu);
  }
  if (threadIdx.x == 0) a.lse[row] = sum == 0.f ? SWA_NEG_INF : top + logf(sum);
}

template <int D, bool F16>
__global__ void __launch_bounds__(128)
    swa_cache_weights_kernel(const CacheView c, const CacheAttnArgs a) {
  const int h = static_cast<int>(blockIdx.y), b = static_cast<int>(blockIdx.z);
  int len, n;
  if (!sequence_of(c, b, &len, &n) || n == 0) return;
  const int G = a.Hq / c.Hkv;
  const long long at = static_cast<long long>(blockIdx.x) * 128 + threadIdx.x +
                       max(0, len - a.window + 1) / 32 * 32;
  if (at >= len + n) return;
  const int s = static_cast<int>(at);
  if (s + a.window <= len) return;  // no query sees it
  const int page = page_of(c, c.table, b, s / c.page, c.max_pages);
  if (page < 0) return;
  const size_t block = static_cast<size_t>(page) * c.Hkv + h;
  const uint8_t* key = c.k + (block * c.page + s % c.page) * D;
  const float scale = a.scale * c.k_scale[block];
  float add = 0.f;
  for (int r = 0; r < G * n; ++r) {
    const int g = r / n, t = r % n;
    if (s > len + t || s + a.window <= len + t) continue;
    const size_t row = (static_cast<size_t>(b) * a.Hq + h * G + g) * c.T + t;
    float x = 0.f;
    for (int d = 0; d < D; ++d) x = fmaf(q_value<D, F16>(a.q, row * D + d), e4m3_value(key[d]), x);
    add += expf(x * scale - a.lse[row]);
  }
  c.weight[block * c.page + s % c.page] += add;
}

template <int D, bool F16>
cudaError_t launch_d(const CacheView& c, const CacheAttnArgs& a, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(c.T), static_cast<unsigned>(a.Hq),
                  static_cast<unsigned>(c.B));
  swa_cache_attn_kernel<D, F16><<<grid, kWarps * 32, 0, stream>>>(c, a);
  if (a.accumulate) {
    const long long most = static_cast<long long>(c.max_pages) * c.page;
    const long long span = most < a.window + c.T + 32ll ? most : a.window + c.T + 32ll;
    const dim3 wgrid(static_cast<unsigned>((span + 127) / 128), static_cast<unsigned>(c.Hkv),
                     static_cast<unsigned>(c.B));
    swa_cache_weights_kernel<D, F16><<<wgrid, 128, 0, stream>>>(c, a);
  }
  return cudaGetLastError();
}

}  // namespace

size_t cache_attn_workspace_bytes(int, int, int, int, int, int, int, int) { return 0; }

cudaError_t launch_cache_attn(const CacheView& c, const CacheAttnArgs& a, cudaStream_t stream) {
  const bool f16 = a.dtype == SWA_FP16;
  if (c.D == 64) return f16 ? launch_d<64, true>(c, a, stream) : launch_d<64, false>(c, a, stream);
  if (c.D == 128)
    return f16 ? launch_d<128, true>(c, a, stream) : launch_d<128, false>(c, a, stream);
  return f16 ? launch_d<256, true>(c, a, stream) : launch_d<256, false>(c, a, stream);
}

}  // namespace swa
