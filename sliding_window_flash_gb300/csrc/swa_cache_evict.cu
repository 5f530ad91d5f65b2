// swa_cache_evict.cu — cuts a paged cache to a budget by accumulated attention weight.
//
// Two kernels.  The first chooses, one cluster of 1 to 8 CTAs per (sequence, kv head), each with a
// slice of the older tokens: their weights, as bits that order like the floats, are read once into
// shared memory; up to three passes of a radix selection (11, 11 and 10 bits) find the smallest weight
// that stays.  Each CTA adds the bins it filled to its first neighbour's histogram through distributed
// shared memory, which finds the bin and tells all of them (reading every histogram from every CTA
// instead: 59 us in all where this takes 20, one sequence of 30,553 tokens with 16 heads).  Then every
// CTA knows how many of its tokens stay and where they go, and its warps write the survivors in slot
// order by ballots: all above the threshold, and the first of those equal to it.
// The second moves, a destination block (page and kv head) at a time, whose scales are the largest of
// its tokens': 8 warps copy one block while 4 look up where the next one's tokens are, a chain of four
// dependent reads that otherwise every block waits for.  It reads and writes 2 D + 4 bytes a survivor,
// which bounds it.
#include "swa_cache_kernels.h"
#include "swa_ptx.cuh"

namespace swa {
namespace {

constexpr int kSelectThreads = 512;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 2048;
constexpr int kMaxHeld = 48 * 1024;  // weights of a slice held in shared memory; more are read again
constexpr int kMoveThreads = 256;  // that copy
constexpr int kLookThreads = 128;  // that look up the next block's sources, one for each row

static_assert(kMaxHeld % 4 == 0, "held in fours");

// Bits that order like the floats: negatives reversed, -0 as 0, NaN on top (its sign is ignored).
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Accesses to the 32-bit word of CTA `rank`'s shared memory that is at `saddr` in this CTA's.
__device__ __forceinline__ uint32_t cluster_at(uint32_t saddr, uint32_t rank) {
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(saddr), "r"(rank));
  return remote;
}
__device__ __forceinline__ unsigned cluster_ld(uint32_t saddr, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_at(saddr, rank)) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_st(uint32_t saddr, uint32_t rank, unsigned v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_at(saddr, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_add(uint32_t saddr, uint32_t rank, unsigned v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(cluster_at(saddr, rank)),
               "r"(v)
               : "memory");
}

struct alignas(16) SelectShared {
  unsigned hist[3][kBins];  // one for each pass; the first CTA's become the cluster's
  unsigned warp[2][kSelectWarps];
  unsigned count[2];        // this CTA's tokens above the threshold, and equal to it
  unsigned pick[3][3];      // each pass's bin, how many of its tokens stay, whether that is all of them
};
static_assert(sizeof(SelectShared) % 16 == 0, "the held weights behind it are read 16 bytes at a time");

// Four consecutive tokens of a slice: their keys, and which of them exist (a bit each).
struct Quad {
  uint32_t k[4];
  unsigned real;
};

__global__ void __launch_bounds__(kSelectThreads, 2)
    swa_evict_select_kernel(const CacheView c, const CacheEvictArgs a, int ctas, int page_log2) {
  extern __shared__ __align__(16) uint8_t smem[];
  SelectShared& sh = *reinterpret_cast<SelectShared*>(smem);
  uint32_t* held = reinterpret_cast<uint32_t*>(smem + sizeof(SelectShared));
  const int rank = static_cast<int>(blockIdx.x) % ctas, h = static_cast<int>(blockIdx.x) / ctas;
  const int b = static_cast<int>(blockIdx.y);
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int* kept = a.kept + (static_cast<size_t>(b) * c.Hkv + h) * a.budget;
  int len, n;
  if (!sequence_of(c, b, &len, &n)) len = 0;
  const int m = min(len, a.budget);
  const int me = rank * kSelectThreads + tid, all = ctas * kSelectThreads;
  for (int i = m + me; i < a.budget; i += all) kept[i] = -1;
  // Where nothing is chosen the whole cluster leaves: the same for all of its CTAs.
  if (len <= a.budget) {
    for (int i = me; i < len; i += all) kept[i] = i;
    return;
  }
  const int old = len - a.recent;         // tokens that compete
  const int chosen = a.budget - a.recent; // of which this many stay
  for (int i = me; i < a.recent; i += all) kept[chosen + i] = old + i;
  if (chosen == 0) return;

  // This CTA's slice, and each warp's consecutive part of it; a lane takes four tokens at a time.
  constexpr int kStep = 128;  // tokens of a warp's step
  const int part = ((old + ctas - 1) / ctas + kSelectWarps * kStep - 1) / (kSelectWarps * kStep) * kStep;
  const int slice = part * kSelectWarps;
  const long long first = static_cast<long long>(rank) * slice;
  const int mine = static_cast<int>(max(0ll, min(static_cast<long long>(slice), old - first)));
  const bool hold = mine <= kMaxHeld;
  const int w0 = warp * part, w1 = min(mine, w0 + part);  // of the slice
  auto fetch = [&](int i) -> Quad {  // i is a multiple of 4, and so is every page's length
    Quad q = {{0u, 0u, 0u, 0u}, 0u};
    if (i >= w1) return q;
    const int s = static_cast<int>(first) + i;
    const int page = page_of(c, c.table, b, s >> page_log2, c.max_pages);
    q.real = (1u << min(4, w1 - i)) - 1u;
    if (page < 0) return q;
    const size_t at = (static_cast<size_t>(page) * c.Hkv + h) * c.page + (s & (c.page - 1));
    const float4 x = *reinterpret_cast<const float4*>(c.weight + at);
    q.k[0] = ordered(x.x);
    q.k[1] = ordered(x.y);
    q.k[2] = ordered(x.z);
    q.k[3] = ordered(x.w);
    return q;
  };
  auto get = [&](int i) -> Quad {
    if (!hold) return fetch(i);
    Quad q = {{0u, 0u, 0u, 0u}, 0u};
    if (i < w1) {
      const uint4 x = *reinterpret_cast<const uint4*>(held + i);
      q.k[0] = x.x, q.k[1] = x.y, q.k[2] = x.z, q.k[3] = x.w;
      q.real = (1u << min(4, w1 - i)) - 1u;
    }
    return q;
  };
  auto sync_all = [&]() {
    if (ctas == 1)
      __syncthreads();
    else
      cluster_sync_all();
  };
  for (int i = tid; i < 3 * kBins; i += kSelectThreads) (&sh.hist[0][0])[i] = 0u;
  if (hold) {
#pragma unroll 4
    for (int i = w0 + 4 * lane; i < w1; i += kStep) {
      const Quad q = fetch(i);
      *reinterpret_cast<uint4*>(held + i) = make_uint4(q.k[0], q.k[1], q.k[2], q.k[3]);
    }
  }
  sync_all();  // every histogram is zero

  uint32_t prefix = 0, mask = 0;
  unsigned left = static_cast<unsigned>(chosen);
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t digit = pass == 2 ? 1023u : 2047u;
#pragma unroll 2
    for (int i = w0 + 4 * lane; i < w1; i += kStep) {
      const Quad q = get(i);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if ((q.real >> j & 1u) && (q.k[j] & mask) == prefix)
          atomicAdd(&sh.hist[pass][(q.k[j] >> shift) & digit], 1u);
    }
    if (rank != 0) {
      __syncthreads();
      for (int i = tid; i < kBins; i += kSelectThreads) {
        const unsigned v = sh.hist[pass][i];
        if (v != 0) cluster_add(smem_u32(&sh.hist[pass][i]), 0, v);
      }
    }
    sync_all();
    if (rank == 0) {
      // Four bins a thread, counted from the top down.
      constexpr int kMine = kBins / kSelectThreads;
      static_assert(kMine == 4, "bins of a thread");
      const int top = kBins - 4 - 4 * tid;
      const uint4 x = *reinterpret_cast<const uint4*>(&sh.hist[pass][top]);
      const unsigned bins[4] = {x.w, x.z, x.y, x.x};
      const unsigned sum = x.x + x.y + x.z + x.w;
      unsigned scan = sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const unsigned up = __shfl_up_sync(0xffffffffu, scan, d);
        if (lane >= d) scan += up;
      }
      if (lane == 31) sh.warp[0][warp] = scan;
      __syncthreads();
      // keys in bins above this thread's
      const unsigned before = lane < warp ? sh.warp[0][lane] : 0u;
      unsigned above = scan - sum + __reduce_add_sync(0xffffffffu, before);
      if (above < left && left <= above + sum) {
        int j = 0;
        while (above + bins[j] < left) above += bins[j++];
        for (int r = 0; r < ctas; ++r) {
          cluster_st(smem_u32(&sh.pick[pass][0]), r, static_cast<unsigned>(top + 3 - j));
          cluster_st(smem_u32(&sh.pick[pass][1]), r, left - above);
          cluster_st(smem_u32(&sh.pick[pass][2]), r, bins[j] == left - above ? 1u : 0u);
        }
      }
    }
    sync_all();
    prefix |= sh.pick[pass][0] << shift;
    mask |= digit << shift;
    left = sh.pick[pass][1];
    if (sh.pick[pass][2] != 0) {  // the whole bin stays: everything from its first key on
      --prefix;  // not 0: some token does not stay
      left = 0;
      break;
    }
  }

  // Every token above `prefix` stays, and of those equal to it the first `left`.
  unsigned n_above = 0, n_tie = 0;
  for (int i = w0; i < w1; i += kStep) {
    const Quad q = get(i + 4 * lane);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool real = q.real >> j & 1u;
      n_above += __popc(__ballot_sync(0xffffffffu, real && q.k[j] > prefix));
      n_tie += __popc(__ballot_sync(0xffffffffu, real && q.k[j] == prefix));
    }
  }
  // Each warp's numbers, then how many come before it: in its CTA, and in the CTAs before.
  if (lane == 0) {
    sh.warp[0][warp] = n_above;
    sh.warp[1][warp] = n_tie;
  }
  __syncthreads();
  if (warp < 2) {
    const unsigned x = lane < kSelectWarps ? sh.warp[warp][lane] : 0u;
    unsigned scan = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const unsigned up = __shfl_up_sync(0xffffffffu, scan, d);
      if (lane >= d) scan += up;
    }
    if (lane < kSelectWarps) sh.warp[warp][lane] = scan - x;
    if (lane == 31) sh.count[warp] = scan;
  }
  sync_all();
  if (warp < 2) {
    const unsigned x = lane < rank ? cluster_ld(smem_u32(&sh.count[warp]), lane) : 0u;
    const unsigned sum = __reduce_add_sync(0xffffffffu, x);
    if (lane < kSelectWarps) sh.warp[warp][lane] += sum;
  }
  sync_all();  // the counts have been read: a CTA may leave
  unsigned at_above = sh.warp[0][warp], at_tie = sh.warp[1][warp];  // of the tokens before this warp's
  const unsigned below = (1u << lane) - 1u;
  for (int i = w0; i < w1; i += kStep) {
    const Quad q = get(i + 4 * lane);
    unsigned ob[4], tb[4], above = at_above, ties = at_tie;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool real = q.real >> j & 1u;
      ob[j] = __ballot_sync(0xffffffffu, real && q.k[j] > prefix);
      tb[j] = __ballot_sync(0xffffffffu, real && q.k[j] == prefix);
      above += __popc(ob[j] & below);
      ties += __popc(tb[j] & below);
      at_above += __popc(ob[j]);
      at_tie += __popc(tb[j]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool over = ob[j] >> lane & 1u, tie = tb[j] >> lane & 1u;
      if (over || (tie && ties < left)) {
        const unsigned to = above + min(ties, left);
        if (to < static_cast<unsigned>(chosen))
          kept[to] = static_cast<int>(first) + i + 4 * lane + j;
      }
      above += over;
      ties += tie;
    }
  }
}

// What the copying threads need to know of one destination block.
struct MoveBlock {
  long long row[128];  // source row (token) of the pool, or -1
  float scale[2][128]; // its scales, of keys and of values
  long long block;     // destination page and head, or -1: nothing to do
};

template <int D>
__global__ void __launch_bounds__(kMoveThreads + kLookThreads, 4)
    swa_evict_move_kernel(const CacheView c, const CacheEvictArgs a, int pages, int64_t tasks) {
  __shared__ MoveBlock s_block[2];
  const int tid = static_cast<int>(threadIdx.x);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // Task t is destination page t % pages of head (t / pages) % Hkv of a sequence.
  auto look = [&](int64_t t, MoveBlock& to_do) {
    const int i = tid - kMoveThreads;
    const int64_t bh = t / pages;
    const int j = static_cast<int>(t - bh * pages);
    const int b = static_cast<int>(bh / c.Hkv), h = static_cast<int>(bh - static_cast<int64_t>(b) * c.Hkv);
    // lens_out may be lens: cutting a length twice is cutting it once, so it does not matter whether
    // another block has written it yet.
    int len, n;
    if (!sequence_of(c, b, &len, &n)) len = 0;
    const int m = min(len, a.budget);
    if (h == 0 && j == 0 && i == 0) a.lens_out[b] = m;
    const int rows = min(c.page, m - j * c.page);
    const int to = rows > 0 ? page_of(c, a.dst_table, b, j, a.dst_pages) : -1;
    if (i == 0) to_do.block = to < 0 ? -1 : static_cast<long long>(to) * c.Hkv + h;
    long long row = -1;
    float ks = 0.f, vs = 0.f;
    if (i < rows && to >= 0) {
      const int s = a.kept[static_cast<size_t>(bh) * a.budget + j * c.page + i];
      const int page = page_of(c, c.table, b, s / c.page, c.max_pages);
      if (page >= 0) {
        const size_t from = static_cast<size_t>(page) * c.Hkv + h;
        row = static_cast<long long>(from * c.page + s % c.page);
        ks = c.k_scale[from];
        vs = c.v_scale[from];
        c.weight[(static_cast<size_t>(to) * c.Hkv + h) * c.page + i] = c.weight[row];
      }
    }
    to_do.row[i] = row;
    to_do.scale[0][i] = ks;
    to_do.scale[1][i] = vs;
  };
  if (tid >= kMoveThreads && blockIdx.x < tasks) look(blockIdx.x, s_block[0]);
  __syncthreads();
  int cur = 0;
  for (int64_t t = blockIdx.x; t < tasks; t += gridDim.x, cur ^= 1) {
    if (tid >= kMoveThreads) {
      if (t + gridDim.x < tasks) look(t + gridDim.x, s_block[cur ^ 1]);
    } else if (s_block[cur].block >= 0) {
      const MoveBlock& m = s_block[cur];
      const size_t block = static_cast<size_t>(m.block);
      // The block's scales, found by every warp for itself.
      float top[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        top[0] = fmaxf(top[0], m.scale[0][lane_id() + 32 * i]);
        top[1] = fmaxf(top[1], m.scale[1][lane_id() + 32 * i]);
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) {
        top[0] = fmaxf(top[0], __shfl_xor_sync(0xffffffffu, top[0], d));
        top[1] = fmaxf(top[1], __shfl_xor_sync(0xffffffffu, top[1], d));
      }
      if (tid == 0 && top[0] > 0.f) {
        c.k_scale[block] = top[0];
        c.v_scale[block] = top[1];
      }
      // 16 bytes at a time, four of them on their way together: a row's keys, then its values.
      constexpr int kUnits = D / 16;
      const int units = c.page * 2 * kUnits;
      for (int i0 = tid; i0 < units; i0 += 4 * kMoveThreads) {
        uint4 x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = i0 + e * kMoveThreads;
          const long long row = i < units ? m.row[i / (2 * kUnits)] : -1;
          if (row >= 0)
            x[e] = __ldcs(reinterpret_cast<const uint4*>((i / kUnits & 1 ? c.v : c.k) +
                                                         static_cast<size_t>(row) * D + i % kUnits * 16));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = i0 + e * kMoveThreads, r = i / (2 * kUnits), w = i / kUnits & 1;
          if (i >= units || m.row[r] < 0) continue;
          uint4 y = x[e];
          if (m.scale[w][r] != top[w]) {
            const uint32_t ratio = half2_of(m.scale[w][r] / top[w]);
            y = make_uint4(e4m3x4_times(y.x, ratio), e4m3x4_times(y.y, ratio),
                           e4m3x4_times(y.z, ratio), e4m3x4_times(y.w, ratio));
          }
          *reinterpret_cast<uint4*>((w ? c.v : c.k) + (block * c.page + r) * D + i % kUnits * 16) = y;
        }
      }
    }
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_cache_evict(const CacheView& c, const CacheEvictArgs& a, cudaStream_t stream) {
  // CTAs of a cluster: as many as there are SMs for, with at least 2048 slots each; two for each SM where
  // they have 12,288 (8 sequences of 32,768 tokens, 8 heads: 45 us, 50 otherwise; 16 of 8,192: 24, or 27
  // with two for each SM there too).
  const long long slots = static_cast<long long>(c.max_pages) * c.page;
  const long long heads = static_cast<long long>(c.B) * c.Hkv;
  int ctas = 1;
  while (ctas < kMaxCluster && ((heads * ctas * 2 <= sm_count() && slots > 2048ll * ctas) ||
                                (heads * ctas <= sm_count() && slots > 12288ll * ctas)))
    ctas *= 2;
  const long long slice = (slots + ctas - 1) / ctas + kSelectWarps * 128;
  const int held = static_cast<int>(slice < kMaxHeld ? slice : kMaxHeld);
  const int bytes = static_cast<int>(sizeof(SelectShared)) + held * 4;
  cudaError_t e = allow_smem<swa_evict_select_kernel>(static_cast<int>(sizeof(SelectShared)) +
                                                      kMaxHeld * 4);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(c.Hkv * ctas), static_cast<unsigned>(c.B));
  cfg.blockDim = dim3(kSelectThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(bytes);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, swa_evict_select_kernel, c, a, ctas,
                              c.page == 32 ? 5 : c.page == 64 ? 6 : 7)) != cudaSuccess) return e;
  // The move may be scheduled while the choice ends (it waits for it before it reads).
  const int pages = (a.budget + c.page - 1) / c.page;
  const int64_t tasks = heads * pages, most = 4ll * sm_count();
  auto move = c.D == 64    ? swa_evict_move_kernel<64>
              : c.D == 128 ? swa_evict_move_kernel<128>
                           : swa_evict_move_kernel<256>;
  return launch_early(move, static_cast<unsigned>(tasks < most ? tasks : most), kMoveThreads + kLookThreads, 0, stream,
                      c, a, pages, tasks);
}

}  // namespace swa
