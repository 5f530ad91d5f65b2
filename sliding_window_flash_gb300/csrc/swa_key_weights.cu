// swa_key_weights.cu — the attention weight every key received: for key j of kv head hk,
//   w[j] = sum over the group's query heads and the queries i that see j of
//          exp(scale <q_i, k_j> - lse_i).
//
// First form: one thread per key, the key's row in shared memory, the queries of its window read a
// tile at a time.
#include "swa_cache_kernels.h"
#include "swa_ptx.cuh"

namespace swa {
namespace {

constexpr int kKeys = 64, kQueries = 16;

template <int D, bool F16>
__global__ void __launch_bounds__(kKeys)
    swa_key_weights_kernel(const uint16_t* __restrict__ q, const uint16_t* __restrict__ k,
                           const float* __restrict__ lse, float* __restrict__ w, int Hq, int Hkv,
                           Span sp, float scale) {
  __shared__ uint32_t s_k[kKeys][D / 2 + 1];
  __shared__ uint32_t s_q[kQueries][D / 2];
  const int h = static_cast<int>(blockIdx.y), b = static_cast<int>(blockIdx.z);
  const int tid = static_cast<int>(threadIdx.x), k0 = static_cast<int>(blockIdx.x) * kKeys;
  const size_t kv = static_cast<size_t>(b) * Hkv + h;
  const uint32_t* kk = reinterpret_cast<const uint32_t*>(k) + kv * sp.Lk * (D / 2);
  for (int i = tid; i < kKeys * D / 2; i += kKeys) {
    const int r = i / (D / 2), d = i % (D / 2);
    s_k[r][d] = k0 + r < sp.Lk ? kk[static_cast<size_t>(k0 + r) * (D / 2) + d] : 0u;
  }
  const int key = k0 + tid, last_key = min(k0 + kKeys, sp.Lk) - 1;
  const int lo = max(0, k0 + sp.dmin - sp.off);
  const long long hi = min(static_cast<long long>(sp.Lq) - 1,
                           static_cast<long long>(last_key) + sp.dmax - sp.off);
  float sum = 0.f;
  const int G = Hq / Hkv;
  for (int g = 0; g < G; ++g) {
    const size_t row0 = (static_cast<size_t>(b) * Hq + h * G + g) * sp.Lq;
    const uint32_t* qq = reinterpret_cast<const uint32_t*>(q) + row0 * (D / 2);
    for (int i0 = lo; i0 <= hi; i0 += kQueries) {
      __syncthreads();
      for (int i = tid; i < kQueries * D / 2; i += kKeys) {
        const int r = i / (D / 2), d = i % (D / 2);
        s_q[r][d] = i0 + r < sp.Lq ? qq[static_cast<size_t>(i0 + r) * (D / 2) + d] : 0u;
      }
      __syncthreads();
      float x[kQueries] = {};
      for (int d = 0; d < D / 2; ++d) {
        const float2 kd = Elem<F16>::unpack(s_k[tid][d]);
#pragma unroll
        for (int r = 0; r < kQueries; ++r) {
          const float2 qd = Elem<F16>::unpack(s_q[r][d]);
          x[r] = fmaf(kd.x, qd.x, fmaf(kd.y, qd.y, x[r]));
        }
      }
#pragma unroll
      for (int r = 0; r < kQueries; ++r) {
        const int i = i0 + r, d = i + sp.off - key;
        if (i < sp.Lq && d >= sp.dmin && d <= sp.dmax) sum += expf(x[r] * scale - lse[row0 + i]);
      }
    }
  }
  if (key < sp.Lk) w[kv * sp.Lk + key] = sum;
}

template <int D, bool F16>
cudaError_t launch_d(const Problem& pb, const void* q, const void* k, const float* lse, float* w,
                     cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((pb.span.Lk + kKeys - 1) / kKeys),
                  static_cast<unsigned>(pb.Hkv), static_cast<unsigned>(pb.B));
  swa_key_weights_kernel<D, F16><<<grid, kKeys, 0, stream>>>(
      static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k), lse, w, pb.Hq, pb.Hkv,
      pb.span, pb.scale);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_key_weights(const Problem& pb, const void* q, const void* k, const float* lse,
                               float* w, cudaStream_t stream) {
  if (pb.D == 64)
    return pb.f16 ? launch_d<64, true>(pb, q, k, lse, w, stream)
                  : launch_d<64, false>(pb, q, k, lse, w, stream);
  if (pb.D == 128)
    return pb.f16 ? launch_d<128, true>(pb, q, k, lse, w, stream)
                  : launch_d<128, false>(pb, q, k, lse, w, stream);
  return pb.f16 ? launch_d<256, true>(pb, q, k, lse, w, stream)
                : launch_d<256, false>(pb, q, k, lse, w, stream);
}

}  // namespace swa
