// swa_bwd_sinks.cu — dK and dV of the sinks: the sums that the parts of their walks left
// (swa_bwd_dkdv.cu, swa_d256_dkdv_pair.cu), added in order, dK scaled, rounded once, and written over
// the sinks' rows.  Every float of the parts is read once, four a thread; with 4 sinks that is a megabyte or
// less, and its latency is most of its 2.5 us (129 sinks: 3.3).  The kernel is launched behind dQ, which
// begins while the parts are still walked, and waits for both.
#include "swa_kernels.h"
#include "swa_ptx.cuh"

namespace swa {
namespace {

template <bool F16>
__global__ void __launch_bounds__(256)
    swa_sink_join_kernel(const float* part, uint16_t* dk, uint16_t* dv, int splits, int heads,
                         int sinks, int Lk, int D, float scale) {
  wait_predecessor();
  launch_dependents();
  const long long quads = static_cast<long long>(heads) * 2 * sinks * (D / 4);
  const size_t step = sink_part_offset(1, heads, 0, 0, sinks, 0, D);
  for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < quads;
       i += static_cast<long long>(gridDim.x) * 256) {
    const float* src = part + 4 * i;
    float4 sum = *reinterpret_cast<const float4*>(src);
#pragma unroll 4
    for (int s = 1; s < splits; ++s) {
      const float4 x = *reinterpret_cast<const float4*>(src + s * step);
      sum.x += x.x;
      sum.y += x.y;
      sum.z += x.z;
      sum.w += x.w;
    }
    const long long row = i / (D / 4);
    const int col = static_cast<int>(i - row * (D / 4)) * 4;
    const long long hw = row / sinks;  // 2 bhk + (dV: 1)
    const int key = static_cast<int>(row - hw * sinks);
    const float mul = hw & 1 ? 1.f : scale;
    uint16_t* dst = (hw & 1 ? dv : dk) + (static_cast<size_t>(hw >> 1) * Lk + key) * D + col;
    *reinterpret_cast<uint2*>(dst) = make_uint2(Elem<F16>::pack(sum.x * mul, sum.y * mul),
                                                Elem<F16>::pack(sum.z * mul, sum.w * mul));
  }
}

}  // namespace

cudaError_t launch_sink_join(const Problem& pb, void* dk, void* dv, cudaStream_t stream) {
  const int heads = pb.B * pb.Hkv;
  const long long quads = static_cast<long long>(heads) * 2 * pb.sinks * (pb.D / 4);
  const long long blocks = (quads + 255) / 256, most = 16ll * sm_count();
  auto kern = pb.f16 ? swa_sink_join_kernel<true> : swa_sink_join_kernel<false>;
  return launch_early(kern, static_cast<unsigned>(blocks < most ? blocks : most), 256, 0, stream,
                      pb.sink_part, static_cast<uint16_t*>(dk), static_cast<uint16_t*>(dv),
                      sink_plan(pb).splits, heads, pb.sinks, pb.span.Lk, pb.D, pb.scale);
}

}  // namespace swa
