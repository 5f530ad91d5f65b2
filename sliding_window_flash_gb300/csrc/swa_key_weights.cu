// swa_key_weights.cu — the attention weight every key received: for key j of kv head hk,
//   w[j] = sum over the group's query heads and the queries i that see j of
//          exp(scale <q_i, k_j> - lse_i) = sum 2^(c s_ij - lse_i / ln 2),  c = scale / ln 2.
//
// One product per visible pair (2 D flops) and one exponential: at D = 128 a 128 x 128 tile takes the
// tensor core ~512 cycles and the exponential unit ~546, so both have to run all the time.  The scores
// are taken transposed, S^T = K Q^T, which puts a key on a TMEM lane: its sum stays in the registers
// of the threads that own the lane, and nothing is reduced across threads until the end.
//   * A task is 256 keys (two 128-row tiles) of one (batch, kv head) with the walk over its query
//     tiles of every query head of the group: each query tile loaded is used for two products, which
//     halves the traffic into shared memory (30 bytes a cycle and SM at D = 128).
//   * Persistent CTAs, one per SM, take tasks longest first, there and back again (task i of a round
//     from the left, then from the right), so that walks of unequal length even out.  With few tasks
//     each walk is cut into `pieces` equal parts whose sums a second kernel adds in order.
//   * 20 warps: 16 take the exponentials (a quarter of the lanes, a key tile and half of a tile's
//     columns each), and one each loads Q, loads K, issues the products, and keeps -lse / ln 2 of the
//     next query tiles in shared memory.  Four score tiles in TMEM, two per key tile.
//   * Masked tiles select; whatever a query outside the window holds does not reach the sum.  A tile's
//     64 terms are added in fp32, tiles with a compensated sum (Kahan), so the error does not grow
//     with the walk.
#include "swa_cache_kernels.h"
#include "swa_ptx.cuh"
#include "swa_tmap.h"

namespace swa {
namespace {

constexpr int kTaskKeys = 256;
constexpr int kEpiWarps = 16;
constexpr int kWarpQ = kEpiWarps, kWarpK = kEpiWarps + 1, kWarpMma = kEpiWarps + 2,
              kWarpLse = kEpiWarps + 3;
constexpr int kKwThreads = 32 * (kEpiWarps + 4);
constexpr int kLseSlots = 3;

template <int D>
struct KwCfg {
  static constexpr int kCols = D < 128 ? D : 128;       // columns of a piece of a tile
  static constexpr int kHalves = D / kCols;             // pieces of a tile
  static constexpr int kPieceBytes = 128 * kCols * 2;
  static constexpr int kChunks = kCols / 64;
  static constexpr int kChunkBytes = 128 * 128;
  static constexpr int kKSets = D == 256 ? 1 : 2;       // tasks whose keys are held
  static constexpr int kKPieces = kKSets * 2 * kHalves; // 4
  static constexpr int kQStages = D == 64 ? 6 : 3;      // pieces
  static constexpr int kOffQ = kKPieces * kPieceBytes;
  static constexpr int kOffLse = kOffQ + kQStages * kPieceBytes;
  static constexpr int kOffRed = kOffLse + kLseSlots * 512;  // a half's sums, per key tile
  static constexpr int kOffBar = kOffRed + 2 * 512;
  static constexpr int kKFull = 0;
  static constexpr int kKEmpty = kKFull + kKSets;
  static constexpr int kQFull = kKEmpty + kKSets;
  static constexpr int kQEmpty = kQFull + kQStages;
  static constexpr int kSFull = kQEmpty + kQStages;   // [tile][buffer]
  static constexpr int kSEmpty = kSFull + 4;
  static constexpr int kLFull = kSEmpty + 4;
  static constexpr int kLEmpty = kLFull + kLseSlots;
  static constexpr int kDrain = kLEmpty + kLseSlots;
  static constexpr int kNumBars = kDrain + 1;
  static constexpr int kSmemBytes = kOffBar + kNumBars * 8 + 16;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");
};

struct KwArgs {
  const float* lse;
  float* w;        // [pieces][B Hkv][Lk] when pieces > 1, else the output
  int BHK, Hq, Hkv, G, pieces;
  int64_t tasks;   // key blocks x pieces x B Hkv
  Span span;
  float scale_log2;
  unsigned* err;
};

// A task's walk: units [u0, u1) of (query head, query tile) pairs, head-major.
struct Walk {
  int k0, bhk, piece, qb_lo, nq, u0, u1;
};

struct Schedule {
  int64_t tasks;
  int round = 0;
  // Index of this CTA's next task, or -1.
  __device__ __forceinline__ int64_t next() {
    const int64_t grid = gridDim.x;
    const int64_t at = (round & 1) ? grid - 1 - blockIdx.x : blockIdx.x;
    const int64_t i = round++ * grid + at;
    if (i < tasks) return i;
    return -1;
  }
  __device__ __forceinline__ bool over() const { return round * static_cast<int64_t>(gridDim.x) >= tasks; }
};

__device__ __forceinline__ Walk walk_of(const KwArgs& a, int64_t task) {
  Walk w;
  const int kbp = static_cast<int>(task / a.BHK);
  w.bhk = static_cast<int>(task - static_cast<int64_t>(kbp) * a.BHK);
  w.piece = kbp % a.pieces;
  w.k0 = kbp / a.pieces * kTaskKeys;
  w.qb_lo = a.span.first_qblock(w.k0);
  const int last = w.k0 + kBlockN < a.span.Lk ? w.k0 + kBlockN : w.k0;
  w.nq = max(0, a.span.last_qblock(last) - w.qb_lo + 1);
  const int64_t all = static_cast<int64_t>(a.G) * w.nq;
  w.u0 = static_cast<int>(all * w.piece / a.pieces);
  w.u1 = static_cast<int>(all * (w.piece + 1) / a.pieces);
  return w;
}

// Whether key tile `tile` of the walk's block is seen by query tile qb at all.
struct TileSpan {
  int lo, hi;
};
__device__ __forceinline__ TileSpan tile_span(const KwArgs& a, int k0, int tile) {
  const int k = k0 + tile * kBlockN;
  TileSpan t = {0, -1};
  if (k < a.span.Lk) {
    t.lo = a.span.first_qblock(k);
    t.hi = a.span.last_qblock(k);
  }
  return t;
}

template <int D, bool F16>
__global__ void __launch_bounds__(kKwThreads, 1)
    swa_key_weights_kernel(const __grid_constant__ CUtensorMap tm_q,
                           const __grid_constant__ CUtensorMap tm_k, const KwArgs a) {
  using C = KwCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (!smem_base_ok(smem, a.err)) return;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kNumBars);
  int& abort_flag = *reinterpret_cast<int*>(tmem_slot + 1);
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  const uint32_t sK = smem_u32(smem), sQ = smem_u32(smem + C::kOffQ);
  const uint32_t warp = warp_id(), lane = lane_id();
  const Span sp = a.span;
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < C::kKSets; ++i) {
      mbar_init(bar(C::kKFull + i), 1);
      mbar_init(bar(C::kKEmpty + i), 1);
    }
    for (int i = 0; i < C::kQStages; ++i) {
      mbar_init(bar(C::kQFull + i), 1);
      mbar_init(bar(C::kQEmpty + i), 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar(C::kSFull + i), 1);
      mbar_init(bar(C::kSEmpty + i), kEpiWarps / 2);
    }
    for (int i = 0; i < kLseSlots; ++i) {
      mbar_init(bar(C::kLFull + i), 1);
      mbar_init(bar(C::kLEmpty + i), kEpiWarps);
    }
    mbar_init(bar(C::kDrain), 1);
    fence_barrier_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Schedule sched = {a.tasks};

  if (warp == kWarpQ) {
    // ------------------------------------------------------------------ Q pieces
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      int s = 0;
      uint32_t phase = 1;  // of the empty barriers: the first round does not wait
      bool ok = true;
      int64_t issued = 0;
      while (ok && !sched.over()) {
        const int64_t task = sched.next();
        if (task < 0) continue;
        const Walk w = walk_of(a, task);
        const int bhq0 = w.bhk / a.Hkv * a.Hq + w.bhk % a.Hkv * a.G;
        int gi = w.nq > 0 ? w.u0 / w.nq : 0, qi = w.nq > 0 ? w.u0 % w.nq : 0;
        for (int u = w.u0; ok && u < w.u1; ++u) {
          for (int h = 0; h < C::kHalves; ++h) {
            if (!(ok = mbar_wait(bar(C::kQEmpty + s), phase, &abort_flag, a.err))) break;
            mbar_arrive_expect_tx(bar(C::kQFull + s), C::kPieceBytes);
            for (int x = 0; x < C::kChunks; ++x)
              tma_load_3d(sQ + s * C::kPieceBytes + x * C::kChunkBytes, &tm_q, bar(C::kQFull + s),
                          128 * h + 64 * x, (w.qb_lo + qi) * kBlockM, bhq0 + gi);
            ++issued;
            if (++s == C::kQStages) {
              s = 0;
              phase ^= 1u;
            }
          }
          if (++qi == w.nq) {
            qi = 0;
            ++gi;
          }
        }
      }
      // every copy of this warp has landed before the CTA ends
      for (int64_t i = issued > C::kQStages ? issued - C::kQStages : 0; i < issued; ++i)
        drain_wait(bar(C::kQFull + static_cast<int>(i % C::kQStages)),
                   static_cast<uint32_t>(i / C::kQStages) & 1u, a.err);
    }
  } else if (warp == kWarpK) {
    // ------------------------------------------------------------------ K tiles
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      int64_t n = 0;
      bool ok = true;
      while (ok && !sched.over()) {
        const int64_t task = sched.next();
        if (task < 0) continue;
        const Walk w = walk_of(a, task);
        if (w.u0 == w.u1) continue;
        const int set = static_cast<int>(n % C::kKSets);
        if (!(ok = mbar_wait(bar(C::kKEmpty + set), (static_cast<uint32_t>(n / C::kKSets) & 1u) ^ 1u,
                             &abort_flag, a.err)))
          break;
        mbar_arrive_expect_tx(bar(C::kKFull + set), 2 * C::kHalves * C::kPieceBytes);
        for (int tile = 0; tile < 2; ++tile)
          for (int x = 0; x < C::kHalves * C::kChunks; ++x)
            tma_load_3d(sK + ((set * 2 + tile) * C::kHalves) * C::kPieceBytes + x * C::kChunkBytes,
                        &tm_k, bar(C::kKFull + set), 64 * x, w.k0 + tile * kBlockN, w.bhk);
        ++n;
      }
      for (int64_t i = n > C::kKSets ? n - C::kKSets : 0; i < n; ++i)
        drain_wait(bar(C::kKFull + static_cast<int>(i % C::kKSets)),
                   static_cast<uint32_t>(i / C::kKSets) & 1u, a.err);
    }
  } else if (warp == kWarpMma) {
    // ------------------------------------------------------------------ products
    constexpr uint32_t kId = idesc_f16kind(Elem<F16>::kMmaFmt, kBlockN, kBlockM, false, false);
    int s = 0;
    uint32_t qphase = 0;
    int64_t n = 0;
    uint32_t used[2] = {0, 0};  // score tiles issued for each key tile
    bool ok = true;
    while (ok && !sched.over()) {
      const int64_t task = sched.next();
      if (task < 0) continue;
      const Walk w = walk_of(a, task);
      if (w.u0 == w.u1) continue;
      const int set = static_cast<int>(n % C::kKSets);
      const TileSpan ts0 = tile_span(a, w.k0, 0), ts1 = tile_span(a, w.k0, 1);
      if (!(ok = warp_wait(bar(C::kKFull + set), static_cast<uint32_t>(n / C::kKSets) & 1u,
                           &abort_flag, a.err)))
        break;
      int qi = w.u0 % w.nq;
      for (int u = w.u0; ok && u < w.u1; ++u) {
        const int qb = w.qb_lo + qi;
        const bool on[2] = {qb >= ts0.lo && qb <= ts0.hi, qb >= ts1.lo && qb <= ts1.hi};
#pragma unroll
        for (int h = 0; h < C::kHalves; ++h) {
          if (!(ok = warp_wait(bar(C::kQFull + s), qphase, &abort_flag, a.err))) break;
#pragma unroll
          for (int tile = 0; tile < 2; ++tile) {
            if (!ok || !on[tile]) continue;
            const uint32_t buf = used[tile] & 1u;
            if (h == 0 && !(ok = warp_wait(bar(C::kSEmpty + 2 * tile + buf),
                                           ((used[tile] >> 1) & 1u) ^ 1u, &abort_flag, a.err)))
              continue;
            tc_fence_after();
            umma_ss_kmajor_d<C::kCols>(
                tmem + (2 * tile + buf) * 128u,
                smem_desc_sw128(sK + ((set * 2 + tile) * C::kHalves + h) * C::kPieceBytes, 16, 1024),
                smem_desc_sw128(sQ + s * C::kPieceBytes, 16, 1024), kId, h > 0 ? 1u : 0u);
            if (h == C::kHalves - 1) {
              umma_commit_w(bar(C::kSFull + 2 * tile + buf));
              ++used[tile];
            }
          }
          if (!ok) break;
          umma_commit_w(bar(C::kQEmpty + s));
          if (++s == C::kQStages) {
            s = 0;
            qphase ^= 1u;
          }
        }
        if (++qi == w.nq) qi = 0;
      }
      if (!ok) break;
      umma_commit_w(bar(C::kKEmpty + set));
      ++n;
    }
    umma_commit_w(bar(C::kDrain));
    warp_drain_wait(bar(C::kDrain), 0, a.err);
  } else if (warp == kWarpLse) {
    // ------------------------------------------------------------------ -lse / ln 2, a slot per query tile
    float* s_lse = reinterpret_cast<float*>(smem + C::kOffLse);
    int s = 0;
    uint32_t phase = 1;
    bool ok = true;
    while (ok && !sched.over()) {
      const int64_t task = sched.next();
      if (task < 0) continue;
      const Walk w = walk_of(a, task);
      const int bhq0 = w.bhk / a.Hkv * a.Hq + w.bhk % a.Hkv * a.G;
      int gi = w.nq > 0 ? w.u0 / w.nq : 0, qi = w.nq > 0 ? w.u0 % w.nq : 0;
      for (int u = w.u0; u < w.u1; ++u) {
        float y[4];
        const int q0 = (w.qb_lo + qi) * kBlockM + static_cast<int>(lane);
        const float* row = a.lse + static_cast<size_t>(bhq0 + gi) * sp.Lq;
#pragma unroll
        for (int i = 0; i < 4; ++i)  // queries past the end weigh nothing
          y[i] = q0 + 32 * i < sp.Lq ? -kLog2e * __ldg(row + q0 + 32 * i) : SWA_NEG_INF;
        if (!(ok = warp_wait(bar(C::kLEmpty + s), phase, &abort_flag, a.err))) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) s_lse[s * 128 + 32 * i + lane] = y[i];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::kLFull + s));
        if (++s == kLseSlots) {
          s = 0;
          phase ^= 1u;
        }
        if (++qi == w.nq) {
          qi = 0;
          ++gi;
        }
      }
    }
  } else {
    // ------------------------------------------------------------------ exponentials and sums
    const int tile = static_cast<int>(warp >> 2) & 1, half = static_cast<int>(warp >> 3);
    const int r = static_cast<int>((warp & 3u) * 32 + lane);  // key row of the tile
    const uint32_t lane_base = ((warp & 3u) * 32u) << 16;
    const float* s_lse = reinterpret_cast<const float*>(smem + C::kOffLse) + 64 * half;
    float* s_red = reinterpret_cast<float*>(smem + C::kOffRed) + 128 * tile;
    const float2 c2 = make_float2(a.scale_log2, a.scale_log2);
    int s = 0;
    uint32_t lphase = 0, used = 0;
    bool ok = true;
    while (!sched.over()) {  // to the end even after a wait ran out: the barriers below count on it
      const int64_t task = sched.next();
      if (task < 0) continue;
      const Walk w = walk_of(a, task);
      const TileSpan ts = tile_span(a, w.k0, tile);
      const int key = w.k0 + tile * kBlockN + r;
      const int vis_lo = key + sp.dmin - sp.off;
      const int vis_hi = static_cast<int>(
          min(static_cast<long long>(key) + sp.dmax - sp.off, static_cast<long long>(sp.Lq)));
      const int k0t = w.k0 + tile * kBlockN;
      // A query tile at q0 needs no mask iff q_int_lo <= q0 <= q_int_hi.
      const int q_int_lo = k0t + kBlockN - 1 + sp.dmin - sp.off;
      const long long q_int_hi = static_cast<long long>(k0t) + sp.dmax - sp.off - (kBlockM - 1);
      float sum = 0.f, comp = 0.f;
      int qi = w.nq > 0 ? w.u0 % w.nq : 0;
      for (int u = w.u0; ok && u < w.u1; ++u) {
        const int qb = w.qb_lo + qi;
        if (!(ok = warp_wait(bar(C::kLFull + s), lphase, &abort_flag, a.err))) break;
        if (qb >= ts.lo && qb <= ts.hi) {
          const uint32_t buf = used & 1u;
          if (!(ok = warp_wait(bar(C::kSFull + 2 * tile + buf), (used >> 1) & 1u, &abort_flag,
                               a.err)))
            break;
          tc_fence_after();
          uint32_t rr[2][32];
          const uint32_t col = tmem + lane_base + (2 * tile + buf) * 128u + 64u * half;
          tmem_ld32(col, rr[0]);
          tmem_ld32(col + 32u, rr[1]);
          tmem_wait_ld_all();
          reg_fence(rr[0]);
          reg_fence(rr[1]);
          warp_arrive(bar(C::kSEmpty + 2 * tile + buf));
          ++used;
          const float4* l4 = reinterpret_cast<const float4*>(s_lse + s * 128);
          float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
          const int q0 = qb * kBlockM;
          if (q0 >= q_int_lo && q0 <= q_int_hi) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float4 l = l4[i];
              const uint32_t* src = &rr[i >> 3][(4 * i) & 31];
              const float2 x0 = __ffma2_rn(make_float2(__uint_as_float(src[0]), __uint_as_float(src[1])),
                                           c2, make_float2(l.x, l.y));
              const float2 x1 = __ffma2_rn(make_float2(__uint_as_float(src[2]), __uint_as_float(src[3])),
                                           c2, make_float2(l.z, l.w));
              acc0 = __fadd2_rn(acc0, make_float2(ex2(x0.x), ex2(x0.y)));
              acc1 = __fadd2_rn(acc1, make_float2(ex2(x1.x), ex2(x1.y)));
            }
          } else {
            const int base = q0 + 64 * half;
            const int lo = vis_lo - base, hi = vis_hi - base;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float4 l = l4[i];
              const uint32_t* src = &rr[i >> 3][(4 * i) & 31];
              const float2 x0 = __ffma2_rn(make_float2(__uint_as_float(src[0]), __uint_as_float(src[1])),
                                           c2, make_float2(l.x, l.y));
              const float2 x1 = __ffma2_rn(make_float2(__uint_as_float(src[2]), __uint_as_float(src[3])),
                                           c2, make_float2(l.z, l.w));
              float2 p0, p1;
              p0.x = 4 * i >= lo && 4 * i <= hi ? ex2(x0.x) : 0.f;
              p0.y = 4 * i + 1 >= lo && 4 * i + 1 <= hi ? ex2(x0.y) : 0.f;
              p1.x = 4 * i + 2 >= lo && 4 * i + 2 <= hi ? ex2(x1.x) : 0.f;
              p1.y = 4 * i + 3 >= lo && 4 * i + 3 <= hi ? ex2(x1.y) : 0.f;
              acc0 = __fadd2_rn(acc0, p0);
              acc1 = __fadd2_rn(acc1, p1);
            }
          }
          const float2 both = __fadd2_rn(acc0, acc1);
          const float add = __fsub_rn(__fadd_rn(both.x, both.y), comp);
          const float next = __fadd_rn(sum, add);
          comp = __fsub_rn(__fsub_rn(next, sum), add);
          sum = next;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::kLEmpty + s));
        if (++s == kLseSlots) {
          s = 0;
          lphase ^= 1u;
        }
        if (++qi == w.nq) qi = 0;
      }
      // The two column halves of a key meet.
      if (half == 1) s_red[r] = sum;
      named_barrier_sync(1 + tile, 256);
      if (half == 0 && key < sp.Lk)
        a.w[(static_cast<size_t>(w.piece) * a.BHK + w.bhk) * sp.Lk + key] = sum + s_red[r];
      named_barrier_sync(1 + tile, 256);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// out[i] = the pieces' sums in order.
__global__ void __launch_bounds__(256)
    swa_key_weights_join_kernel(const float* __restrict__ parts, float* __restrict__ out,
                                int64_t n, int pieces) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t stride = static_cast<int64_t>(gridDim.x) * 256;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += stride) {
    float sum = 0.f;
#pragma unroll 4
    for (int p = 0; p < pieces; ++p) sum += parts[p * n + i];
    out[i] = sum;
  }
}

// Pieces that each walk is cut into: eight tasks for every SM even out walks of unequal length, and a
// piece has at least one (query head, query tile) pair.
int pieces_of(const Problem& pb) {
  const int64_t blocks =
      static_cast<int64_t>((pb.span.Lk + kTaskKeys - 1) / kTaskKeys) * pb.B * pb.Hkv;
  const int64_t want = (8ll * sm_count() + blocks - 1) / blocks;
  // queries that a block of keys can see
  const int64_t reach = static_cast<int64_t>(pb.span.dmax) - pb.span.dmin + kTaskKeys;
  const int64_t tiles = ((reach < pb.span.Lq ? reach : pb.span.Lq) + kBlockM - 1) / kBlockM;
  const int64_t most = tiles * (pb.Hq / pb.Hkv);
  return static_cast<int>(want < most ? want : most);
}

template <int D, bool F16>
cudaError_t launch_d(const Problem& pb, const void* q, const void* k, const float* lse, float* w,
                     float* workspace, cudaStream_t stream) {
  using C = KwCfg<D>;
  CUtensorMap tq, tk;
  const uint64_t bhk = static_cast<uint64_t>(pb.B) * pb.Hkv;
  if (!make_tmap_3d(&tq, q, static_cast<uint64_t>(pb.B) * pb.Hq, pb.span.Lq, D, kBlockM, F16) ||
      !make_tmap_3d(&tk, k, bhk, pb.span.Lk, D, kBlockN, F16))
    return cudaErrorInvalidValue;
  auto kern = swa_key_weights_kernel<D, F16>;
  cudaError_t e = allow_smem<swa_key_weights_kernel<D, F16>>(C::kSmemBytes);
  if (e != cudaSuccess) return e;
  KwArgs a;
  a.lse = lse;
  a.BHK = static_cast<int>(bhk);
  a.Hq = pb.Hq;
  a.Hkv = pb.Hkv;
  a.G = pb.Hq / pb.Hkv;
  a.pieces = pieces_of(pb);
  a.w = a.pieces > 1 ? workspace : w;
  a.tasks = static_cast<int64_t>((pb.span.Lk + kTaskKeys - 1) / kTaskKeys) * a.pieces * a.BHK;
  a.span = pb.span;
  a.scale_log2 = pb.scale * kLog2e;
  a.err = pb.err;
  const int64_t sms = sm_count();
  const unsigned grid = static_cast<unsigned>(a.tasks < sms ? a.tasks : sms);
  kern<<<grid, kKwThreads, C::kSmemBytes, stream>>>(tq, tk, a);
  if ((e = cudaGetLastError()) != cudaSuccess || a.pieces == 1) return e;
  const int64_t n = static_cast<int64_t>(a.BHK) * pb.span.Lk;
  const int64_t blocks = (n + 255) / 256;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks < sms * 8 ? blocks : sms * 8));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, swa_key_weights_join_kernel, static_cast<const float*>(workspace),
                            w, n, a.pieces);
}

}  // namespace

size_t key_weights_workspace_bytes(const Problem& pb) {
  const int pieces = pieces_of(pb);
  if (pieces == 1) return 0;
  const size_t bytes = static_cast<size_t>(pieces) * pb.B * pb.Hkv * pb.span.Lk * sizeof(float);
  return (bytes + 255) & ~static_cast<size_t>(255);
}

cudaError_t launch_key_weights(const Problem& pb, const void* q, const void* k, const float* lse,
                               float* w, void* workspace, cudaStream_t stream) {
  float* ws = static_cast<float*>(workspace);
  if (pb.D == 64)
    return pb.f16 ? launch_d<64, true>(pb, q, k, lse, w, ws, stream)
                  : launch_d<64, false>(pb, q, k, lse, w, ws, stream);
  if (pb.D == 128)
    return pb.f16 ? launch_d<128, true>(pb, q, k, lse, w, ws, stream)
                  : launch_d<128, false>(pb, q, k, lse, w, ws, stream);
  return pb.f16 ? launch_d<256, true>(pb, q, k, lse, w, ws, stream)
                : launch_d<256, false>(pb, q, k, lse, w, ws, stream);
}

}  // namespace swa
