// swa_key_weights.cu — the attention weight every key received: for key j of kv head hk,
//   w[j] = sum over the group's query heads and the queries i that see j of
//          exp(scale <q_i, k_j> - lse_i) = sum 2^(c s_ij - lse_i / ln 2),  c = scale / ln 2.
//
// One product per visible pair (2 D flops) and one exponential: at D = 128 a 128 x 128 tile takes the
// tensor core ~512 cycles and the exponential unit ~546, so both have to run all the time.  The scores
// are taken transposed, S^T = K Q^T, which puts a key on a TMEM lane: its sum stays in the registers
// of the threads that own the lane, and little is reduced across threads at the end.
//   * CTA pairs: a task is 256 keys (128 a CTA) of one (batch, kv head) with the walk over 256 queries
//     at a time of every query head of the group.  Each CTA loads its keys and its half of the
//     queries; rank 0 issues M = 256, N = 256 products for both.  An SM then reads 64 bytes of operands
//     a cycle from shared memory; single CTAs with 128 x 128 products read 128, all there is.
//     Products alone take the pairs 0.169 ms and single CTAs 0.207, the whole 0.235 and 0.288 or more
//     (N = 32,768, W = 1,024, 32 / 16 heads, D = 128).  Units of 128 queries in four buffers, in turn
//     for two groups of warps, take 0.282: their products alone take 0.200.
//   * Persistent pairs take tasks longest first, there and back again (task i of a round from the
//     left, then from the right), so that walks of unequal length even out.  With few tasks each walk
//     is cut into `pieces` equal parts whose sums a second kernel adds in order.
//   * 20 warps a CTA: 16 take the exponentials (32 keys and 64 of a unit's 256 queries each; a part
//     that the window hides is skipped), and one each loads Q, loads K, issues the products (rank 0)
//     or forwards the arrival of its copies (rank 1), and keeps -lse / ln 2 of the next queries in
//     shared memory, announced by the same barrier as their scores (0.036 ms less than with each
//     warp fetching its own).  Two score buffers of 256 columns fill TMEM.
//   * What bounds it: the instructions of the 16 exponential warps, in step with one another for the
//     wait on the same scores.  Of the time over the products', reading the scores from TMEM is 0.006 ms,
//     the log-sum-exps from shared memory 0.016, masks 0.009, exponentials 0.04.
//   * Masked parts select; whatever a query outside the window holds does not reach the sum.  64 terms
//     are added in fp32, then into a compensated sum (Kahan), so the error does not grow with the walk.
#include <type_traits>

#include "swa_cache_kernels.h"
#include "swa_ptx.cuh"
#include "swa_tmap.h"

namespace swa {
namespace {

constexpr int kTaskKeys = 256;
constexpr int kUnitQueries = 256;
constexpr int kEpiWarps = 16;
constexpr int kWarpQ = kEpiWarps, kWarpK = kEpiWarps + 1, kWarpMma = kEpiWarps + 2,
              kWarpLse = kEpiWarps + 3;
constexpr int kKwThreads = 32 * (kEpiWarps + 4);
constexpr int kLseSlots = 4;

template <int D>
struct KwCfg {
  static constexpr int kCols = D < 128 ? D : 128;       // columns of a piece of a tile
  static constexpr int kHalves = D / kCols;             // pieces of a tile
  static constexpr int kPieceBytes = 128 * kCols * 2;
  static constexpr int kChunks = kCols / 64;
  static constexpr int kChunkBytes = 128 * 128;
  static constexpr int kTileBytes = kHalves * kPieceBytes;
  static constexpr int kKSets = D == 256 ? 1 : 2;       // tasks whose keys are held
  static constexpr int kQStages = D == 64 ? 6 : 4;      // pieces
  static constexpr int kOffQ = kKSets * kTileBytes;
  static constexpr int kOffLse = kOffQ + kQStages * kPieceBytes;
  static constexpr int kOffRed = kOffLse + kLseSlots * kUnitQueries * 4;  // three groups' sums
  static constexpr int kOffBar = kOffRed + 3 * 512;
  static constexpr int kKFull = 0;
  static constexpr int kKEmpty = kKFull + kKSets;
  static constexpr int kQFull = kKEmpty + kKSets;
  static constexpr int kQEmpty = kQFull + kQStages;
  static constexpr int kSFull = kQEmpty + kQStages;   // 2 buffers
  static constexpr int kSEmpty = kSFull + 2;          // rank 0's: both CTAs' warps have read
  static constexpr int kLEmpty = kSEmpty + 2;
  static constexpr int kRFull = kLEmpty + kLseSlots;
  static constexpr int kREmpty = kRFull + 1;
  static constexpr int kDrain = kREmpty + 1;
  static constexpr int kNumBars = kDrain + 1;
  static constexpr int kSmemBytes = kOffBar + kNumBars * 8 + 16;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");
};

struct KwArgs {
  const float* lse;
  float* w;        // [pieces][B Hkv][Lk] when pieces > 1, else the output
  int BHK, Hq, G;
  uint32_t tasks;  // key blocks x pieces x B Hkv
  FastDiv div_bhk, div_pieces, div_hkv;
  Span span;
  float scale_log2;
  unsigned* err;
};

// A task's walk: units [u0, u1) of (query head, 256 queries) pairs, head-major; np per head.
struct Walk {
  int k0, bhk, bhq0, piece, q_lo, np, u0, u1;
};

// The tasks of this pair, in order.
struct Schedule {
  uint32_t tasks, round;
  __device__ __forceinline__ bool over() const { return round * (gridDim.x >> 1) >= tasks; }
  // The walk of the next task that has one; false when there is none left.
  __device__ __forceinline__ bool next(const KwArgs& a, Walk* w) {
    const uint32_t pairs = gridDim.x >> 1, mine = blockIdx.x >> 1;
    while (!over()) {
      const uint32_t task = round * pairs + ((round & 1u) ? pairs - 1u - mine : mine);
      ++round;
      if (task >= tasks) continue;
      const uint32_t kbp = a.div_bhk.div(task);
      w->bhk = static_cast<int>(task - kbp * a.div_bhk.d);
      const uint32_t kb = a.div_pieces.div(kbp);
      w->piece = static_cast<int>(kbp - kb * a.div_pieces.d);
      const uint32_t batch = a.div_hkv.div(static_cast<uint32_t>(w->bhk));
      w->bhq0 = static_cast<int>(batch) * a.Hq +
                (w->bhk - static_cast<int>(batch * a.div_hkv.d)) * a.G;
      w->k0 = static_cast<int>(kb) * kTaskKeys;
      const int qb_lo = a.span.first_qblock(w->k0);
      const int last = w->k0 + kBlockN < a.span.Lk ? w->k0 + kBlockN : w->k0;
      w->q_lo = qb_lo * kBlockM;
      w->np = (max(0, a.span.last_qblock(last) - qb_lo + 1) + 1) / 2;
      // pieces are as equal as the units allow, the longer ones first
      const uint32_t all = static_cast<uint32_t>(a.G) * w->np;
      const uint32_t len = a.div_pieces.div(all), extra = all - len * a.div_pieces.d;
      const uint32_t p = static_cast<uint32_t>(w->piece);
      w->u0 = static_cast<int>(p * len + min(p, extra));
      w->u1 = static_cast<int>(w->u0 + len + (p < extra ? 1u : 0u));
      return true;
    }
    return false;
  }
};

// A walk's position: query head of the group and first query of the unit.
struct UnitPos {
  int gi, pi;
  __device__ __forceinline__ explicit UnitPos(const Walk& w)
      : gi(w.np > 0 ? w.u0 / w.np : 0), pi(w.np > 0 ? w.u0 % w.np : 0) {}
  __device__ __forceinline__ void advance(const Walk& w) {
    if (++pi == w.np) {
      pi = 0;
      ++gi;
    }
  }
  __device__ __forceinline__ int q0(const Walk& w) const { return w.q_lo + pi * kUnitQueries; }
};

// Pair products over kCols of the contraction: each CTA holds 128 rows of A and 128 of B, K-major in
// 64-column chunks 16 KB apart (K-step ks starts 32 bytes further inside a chunk).
template <int kCols>
__device__ __forceinline__ void umma2_ss_rows128(uint32_t d, uint64_t a, uint64_t b, uint32_t id,
                                                 uint32_t accumulate) {
  static_assert(kCols == 64 || kCols == 128, "columns");
  if constexpr (kCols == 128) {
    asm volatile(
        "{\n\t.reg .pred e, p, t;\n\t.reg .b64 ra, rb;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.eq.b32 t, %3, %3;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t"
        "add.s64 ra, %1, 2;\n\tadd.s64 rb, %2, 2;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], ra, rb, %3, t;\n\t"
        "add.s64 ra, %1, 4;\n\tadd.s64 rb, %2, 4;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], ra, rb, %3, t;\n\t"
        "add.s64 ra, %1, 6;\n\tadd.s64 rb, %2, 6;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], ra, rb, %3, t;\n\t"
        "add.s64 ra, %1, 1024;\n\tadd.s64 rb, %2, 1024;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], ra, rb, %3, t;\n\t"
        "add.s64 ra, %1, 1026;\n\tadd.s64 rb, %2, 1026;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], ra, rb, %3, t;\n\t"
        "add.s64 ra, %1, 1028;\n\tadd.s64 rb, %2, 1028;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], ra, rb, %3, t;\n\t"
        "add.s64 ra, %1, 1030;\n\tadd.s64 rb, %2, 1030;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], ra, rb, %3, t;\n\t"
        "}" ::"r"(d), "l"(a), "l"(b), "r"(id), "r"(accumulate)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred e, p, t;\n\t.reg .b64 ra, rb;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.eq.b32 t, %3, %3;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t"
        "add.s64 ra, %1, 2;\n\tadd.s64 rb, %2, 2;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], ra, rb, %3, t;\n\t"
        "add.s64 ra, %1, 4;\n\tadd.s64 rb, %2, 4;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], ra, rb, %3, t;\n\t"
        "add.s64 ra, %1, 6;\n\tadd.s64 rb, %2, 6;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], ra, rb, %3, t;\n\t"
        "}" ::"r"(d), "l"(a), "l"(b), "r"(id), "r"(accumulate)
        : "memory");
  }
}

template <int D, bool F16>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kKwThreads, 1)
    swa_key_weights_kernel(const __grid_constant__ CUtensorMap tm_q,
                           const __grid_constant__ CUtensorMap tm_k, const KwArgs a) {
  using C = KwCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  // Both CTAs of the pair always reach the cluster barriers and the collective TMEM allocation; a
  // misaligned window only disables the work (and is reported).
  const bool smem_ok = (smem_u32(smem) & 1023u) == 0u;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kNumBars);
  int& abort_flag = *reinterpret_cast<int*>(tmem_slot + 1);
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  const uint32_t sK = smem_u32(smem), sQ = smem_u32(smem + C::kOffQ);
  const uint32_t warp = warp_id(), lane = lane_id();
  const uint32_t rank = cluster_rank();
  const bool lead = rank == 0u;
  const Span sp = a.span;
  if (threadIdx.x == 0) {
    abort_flag = smem_ok ? 0 : 1;
    if (!smem_ok) atomicOr(a.err, kErrSmemLayout);
    const uint32_t full_count = lead ? 2u : 1u;  // rank 0: own copy and rank 1's relay
    for (int i = 0; i < C::kKSets; ++i) {
      mbar_init(bar(C::kKFull + i), full_count);
      mbar_init(bar(C::kKEmpty + i), 1);
    }
    for (int i = 0; i < C::kQStages; ++i) {
      mbar_init(bar(C::kQFull + i), full_count);
      mbar_init(bar(C::kQEmpty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(C::kSFull + i), 2);  // the product, and its queries' log-sum-exps
      mbar_init(bar(C::kSEmpty + i), 2 * kEpiWarps);
    }
    for (int i = 0; i < kLseSlots; ++i) mbar_init(bar(C::kLEmpty + i), kEpiWarps);
    mbar_init(bar(C::kRFull), kEpiWarps * 3 / 4);
    mbar_init(bar(C::kREmpty), kEpiWarps / 4);
    mbar_init(bar(C::kDrain), 1);
    fence_barrier_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc_pair(smem_u32(tmem_slot), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Schedule sched = {a.tasks, 0u};

  if (!smem_ok) {
    // nothing to do: fall through to the final barrier and the collective release
  } else if (warp == kWarpQ) {
    // ------------------------------------------------------------------ this CTA's half of Q
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      int s = 0;
      uint32_t phase = 1;  // of the empty barriers: the first round does not wait
      bool ok = true;
      int64_t issued = 0;
      Walk w;
      while (ok && sched.next(a, &w)) {
        UnitPos pos(w);
        for (int u = w.u0; ok && u < w.u1; ++u, pos.advance(w)) {
          for (int h = 0; h < C::kHalves; ++h) {
            if (!(ok = mbar_wait(bar(C::kQEmpty + s), phase, &abort_flag, a.err))) break;
            mbar_arrive_expect_tx(bar(C::kQFull + s), C::kPieceBytes);
            for (int x = 0; x < C::kChunks; ++x)
              tma_load_3d(sQ + s * C::kPieceBytes + x * C::kChunkBytes, &tm_q, bar(C::kQFull + s),
                          128 * h + 64 * x, pos.q0(w) + kBlockM * static_cast<int>(rank),
                          w.bhq0 + pos.gi);
            ++issued;
            if (++s == C::kQStages) {
              s = 0;
              phase ^= 1u;
            }
          }
        }
      }
      // every copy of this warp has landed before the CTA ends
      for (int64_t i = issued > C::kQStages ? issued - C::kQStages : 0; i < issued; ++i)
        drain_wait(bar(C::kQFull + static_cast<int>(i % C::kQStages)),
                   static_cast<uint32_t>(i / C::kQStages) & 1u, a.err);
    }
  } else if (warp == kWarpK) {
    // ------------------------------------------------------------------ this CTA's keys
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      int64_t n = 0;
      Walk w;
      while (sched.next(a, &w)) {
        if (w.u0 == w.u1) continue;
        const int set = static_cast<int>(n % C::kKSets);
        if (!mbar_wait(bar(C::kKEmpty + set), (static_cast<uint32_t>(n / C::kKSets) & 1u) ^ 1u,
                       &abort_flag, a.err))
          break;
        mbar_arrive_expect_tx(bar(C::kKFull + set), C::kTileBytes);
        for (int x = 0; x < C::kHalves * C::kChunks; ++x)
          tma_load_3d(sK + set * C::kTileBytes + x * C::kChunkBytes, &tm_k, bar(C::kKFull + set),
                      64 * x, w.k0 + kBlockN * static_cast<int>(rank), w.bhk);
        ++n;
      }
      for (int64_t i = n > C::kKSets ? n - C::kKSets : 0; i < n; ++i)
        drain_wait(bar(C::kKFull + static_cast<int>(i % C::kKSets)),
                   static_cast<uint32_t>(i / C::kKSets) & 1u, a.err);
    }
  } else if (warp == kWarpMma) {
    // ------------------------------------------------------------------ products / relay
    constexpr uint32_t kId =
        idesc_f16kind(Elem<F16>::kMmaFmt, 2 * kBlockN, kUnitQueries, false, false);
    // Rank 1 forwards each of its copies, in the order rank 0 takes them, to rank 0's barrier.
    auto arrived = [&](int idx, uint32_t parity) -> bool {
      if (lead) return warp_wait_cluster(bar(idx), parity, &abort_flag, a.err);
      if (!warp_wait(bar(idx), parity, &abort_flag, a.err)) return false;
      if (lane == 0) mbar_arrive_cluster(mapa_rank0(bar(idx)));
      __syncwarp();
      return true;
    };
    int s = 0;
    uint32_t qphase = 0, used = 0;
    int64_t n = 0;
    bool ok = true;
    Walk w;
    while (ok && sched.next(a, &w)) {
      if (w.u0 == w.u1) continue;
      const int set = static_cast<int>(n % C::kKSets);
      if (!(ok = arrived(C::kKFull + set, static_cast<uint32_t>(n / C::kKSets) & 1u))) break;
      for (int u = w.u0; ok && u < w.u1; ++u) {
        const uint32_t buf = used & 1u;
        if (lead && !(ok = warp_wait_cluster(bar(C::kSEmpty + buf), ((used >> 1) & 1u) ^ 1u,
                                             &abort_flag, a.err)))
          break;
#pragma unroll
        for (int h = 0; h < C::kHalves; ++h) {
          if (!(ok = arrived(C::kQFull + s, qphase))) break;
          if (lead) {
            tc_fence_after();
            umma2_ss_rows128<C::kCols>(
                tmem + buf * 256u,
                smem_desc_sw128(sK + set * C::kTileBytes + h * C::kPieceBytes, 16, 1024),
                smem_desc_sw128(sQ + s * C::kPieceBytes, 16, 1024), kId, h > 0 ? 1u : 0u);
            if (h == C::kHalves - 1) umma2_commit_w(bar(C::kSFull + buf));
            umma2_commit_w(bar(C::kQEmpty + s));
          }
          if (++s == C::kQStages) {
            s = 0;
            qphase ^= 1u;
          }
        }
        ++used;
      }
      if (!ok) break;
      if (lead) umma2_commit_w(bar(C::kKEmpty + set));
      ++n;
    }
    if (lead) {
      umma2_commit_w(bar(C::kDrain));
      warp_drain_wait(bar(C::kDrain), 0, a.err);
    }
  } else if (warp == kWarpLse) {
    // ------------------------------------------------------------------ -lse / ln 2, a slot per unit
    // Slot n mod 4 holds unit n; the two S full barriers alternate, so unit n's is announced only when
    // unit n - 2's score buffer has been handed back by everyone (its phase has then completed).
    float* s_lse = reinterpret_cast<float*>(smem + C::kOffLse);
    uint32_t n = 0;
    bool ok = true;
    Walk w;
    while (ok && sched.next(a, &w)) {
      UnitPos pos(w);
      float y[8];  // the next unit's, on their way while this one's slot is waited for
      auto fetch = [&]() {
        const int q0 = pos.q0(w) + static_cast<int>(lane);
        const float* row = a.lse + static_cast<size_t>(w.bhq0 + pos.gi) * sp.Lq;
#pragma unroll
        for (int i = 0; i < 8; ++i)  // queries past the end weigh nothing
          y[i] = q0 + 32 * i < sp.Lq ? __ldg(row + q0 + 32 * i) : SWA_POS_INF;
      };
      if (w.u0 < w.u1) fetch();
      for (int u = w.u0; u < w.u1; ++u, ++n) {
        const int s = static_cast<int>(n % kLseSlots);
        if (!(ok = warp_wait(bar(C::kLEmpty + s), ((n / kLseSlots) & 1u) ^ 1u, &abort_flag, a.err)))
          break;
#pragma unroll
        for (int i = 0; i < 8; ++i) s_lse[s * kUnitQueries + 32 * i + lane] = -kLog2e * y[i];
        pos.advance(w);
        if (u + 1 < w.u1) fetch();
        __syncwarp();
        // S full of unit n - 2 must be over before this arrival counts for unit n.
        if (n >= 2 && !(ok = warp_wait(bar(C::kSFull + (n & 1u)), ((n >> 1) & 1u) ^ 1u, &abort_flag,
                                       a.err)))
          break;
        if (lane == 0) mbar_arrive(bar(C::kSFull + (n & 1u)));
      }
    }
  } else {
    // ------------------------------------------------------------------ exponentials and sums
    const int group = static_cast<int>(warp >> 2);            // 64 of a unit's 256 queries
    const int r = static_cast<int>((warp & 3u) * 32 + lane);  // key row of the CTA's tile
    const uint32_t col0 = tmem + (((warp & 3u) * 32u) << 16) + 64u * group;
    const float* s_lse = reinterpret_cast<const float*>(smem + C::kOffLse) + 64 * group;
    float* s_red = reinterpret_cast<float*>(smem + C::kOffRed);
    const float2 c2 = make_float2(a.scale_log2, a.scale_log2);
    uint32_t n = 0, rphase = 0;  // units walked so far
    Walk w;
    bool ok = true;
    while (ok && sched.next(a, &w)) {
      const int key = w.k0 + kBlockN * static_cast<int>(rank) + r;
      // This lane's key sees queries vis_lo .. vis_hi; some key of the warp sees vis_lo - lane ..
      // vis_hi - lane + 31, every one vis_lo - lane + 31 .. vis_hi - lane.
      const int vis_lo = key + sp.dmin - sp.off;
      // (vis_hi - lane is cut off behind the last query, the same for the whole warp.)
      const int key0 = key - static_cast<int>(lane);
      const int vis_hi = static_cast<int>(lane) +
                         (key0 < sp.Lk
                              ? static_cast<int>(min(static_cast<long long>(key0) + sp.dmax - sp.off,
                                                     static_cast<long long>(sp.Lq) + 63))
                              : -64);  // a warp without keys: everything is skipped
      float sum = 0.f, comp = 0.f;
      UnitPos pos(w);
      for (int u = w.u0; u < w.u1; ++u, ++n) {
        const uint32_t buf = n & 1u;
        const int qw = pos.q0(w) + 64 * group;
        const int slot = static_cast<int>(n % kLseSlots);
        if (!(ok = warp_wait(bar(C::kSFull + buf), (n >> 1) & 1u, &abort_flag, a.err))) break;
        const int rel_lo = vis_lo - qw, rel_hi = vis_hi - qw;
        if (rel_hi - static_cast<int>(lane) + 31 < 0 || rel_lo - static_cast<int>(lane) > 63) {
          warp_arrive_rank0(bar(C::kSEmpty + buf));
          if (lane == 0) mbar_arrive(bar(C::kLEmpty + slot));
          pos.advance(w);
          continue;
        }
        tc_fence_after();
        const uint32_t col = col0 + buf * 256u;
        const float4* l4 = reinterpret_cast<const float4*>(s_lse + slot * kUnitQueries);
        // Sum of the part's exponentials.  At the window's edges (at_edge) the queries that this key does
        // not see are masked.  Two copies: a branch around the masks alone keeps the two halves of a part
        // without any from interleaving (0.254 and 0.202 ms where this takes 0.235 and 0.195), and
        // comparing with one bound at a time takes 0.254 here too.
        auto part = [&](auto at_edge) -> float {
          constexpr bool kEdge = decltype(at_edge)::value;
          uint32_t raw[32];  // 32 scores at a time: registers for more of them would spill
          tmem_ld32(col, raw);
          float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            tmem_wait_ld(raw);
            if (c == 1) warp_arrive_rank0(bar(C::kSEmpty + buf));
            float2 x[16];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 l = l4[8 * c + i];
              x[2 * i] = __ffma2_rn(
                  make_float2(__uint_as_float(raw[4 * i]), __uint_as_float(raw[4 * i + 1])), c2,
                  make_float2(l.x, l.y));
              x[2 * i + 1] = __ffma2_rn(
                  make_float2(__uint_as_float(raw[4 * i + 2]), __uint_as_float(raw[4 * i + 3])), c2,
                  make_float2(l.z, l.w));
            }
            if constexpr (kEdge) {
              // lo <= i <= hi as one unsigned comparison; a part that is not skipped has lo <= hi
              const uint32_t lo = static_cast<uint32_t>(rel_lo - 32 * c);
              const uint32_t n = static_cast<uint32_t>(rel_hi - rel_lo);
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                x[i].x = 2u * i - lo <= n ? x[i].x : SWA_NEG_INF;
                x[i].y = 2u * i + 1u - lo <= n ? x[i].y : SWA_NEG_INF;
              }
            }
            if (c == 0) tmem_ld32(col + 32u, raw);
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              acc0 = __fadd2_rn(acc0, make_float2(ex2(x[i].x), ex2(x[i].y)));
              acc1 = __fadd2_rn(acc1, make_float2(ex2(x[i + 1].x), ex2(x[i + 1].y)));
            }
          }
          const float2 both = __fadd2_rn(acc0, acc1);
          return __fadd_rn(both.x, both.y);
        };
        const bool edge = rel_lo - static_cast<int>(lane) + 31 > 0 || rel_hi - static_cast<int>(lane) < 63;
        const float add = edge ? part(std::true_type{}) : part(std::false_type{});
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::kLEmpty + slot));
        pos.advance(w);
        const float term = __fsub_rn(add, comp);
        const float next = __fadd_rn(sum, term);
        comp = __fsub_rn(__fsub_rn(next, sum), term);
        sum = next;
      }
      if (!ok) break;
      // The four groups of a key's sum meet at the first's threads.
      if (group != 0) {
        if (!(ok = warp_wait(bar(C::kREmpty), rphase ^ 1u, &abort_flag, a.err))) break;
        s_red[(group - 1) * 128 + r] = sum;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::kRFull));
      } else {
        if (!(ok = warp_wait(bar(C::kRFull), rphase, &abort_flag, a.err))) break;
        sum = (sum + s_red[r]) + (s_red[128 + r] + s_red[256 + r]);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::kREmpty));
        if (key < sp.Lk)
          a.w[(static_cast<size_t>(w.piece) * a.BHK + w.bhk) * sp.Lk + key] = sum;
      }
      rphase ^= 1u;
    }
  }

  // Every cross-CTA arrival and every pair product (rank 0 waited for its drain) is complete once both
  // CTAs are here; then the pair releases its TMEM together.
  tc_fence_before();
  cluster_sync_all();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
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

// Pieces that each walk is cut into: eight tasks for every pair of SMs even out walks of unequal
// length, and a piece has at least one unit.
int pieces_of(const Problem& pb) {
  const int64_t blocks =
      static_cast<int64_t>((pb.span.Lk + kTaskKeys - 1) / kTaskKeys) * pb.B * pb.Hkv;
  const int64_t want = (8ll * (sm_count() / 2) + blocks - 1) / blocks;
  // queries that a block of keys can see
  const int64_t reach = static_cast<int64_t>(pb.span.dmax) - pb.span.dmin + kTaskKeys;
  const int64_t units =
      ((reach < pb.span.Lq ? reach : pb.span.Lq) + kUnitQueries - 1) / kUnitQueries;
  const int64_t most = units * (pb.Hq / pb.Hkv);
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
  a.G = pb.Hq / pb.Hkv;
  const int pieces = pieces_of(pb);
  a.w = pieces > 1 ? workspace : w;
  const int64_t tasks = static_cast<int64_t>((pb.span.Lk + kTaskKeys - 1) / kTaskKeys) * pieces * a.BHK;
  // Task indices (and rounds of them) stay below 2^31: B Hkv Lk < 2^31 keys make at most 2^23 blocks
  // of full walks, and pieces are only cut while there are fewer tasks than that.
  if (tasks >= (1ll << 30)) return cudaErrorInvalidValue;
  a.tasks = static_cast<uint32_t>(tasks);
  a.div_bhk = FastDiv(static_cast<uint32_t>(a.BHK));
  a.div_pieces = FastDiv(static_cast<uint32_t>(pieces));
  a.div_hkv = FastDiv(static_cast<uint32_t>(pb.Hkv));
  a.span = pb.span;
  a.scale_log2 = pb.scale * kLog2e;
  a.err = pb.err;
  const int64_t sms = sm_count();
  const int64_t pairs = max_pair_clusters<swa_key_weights_kernel<D, F16>>(kKwThreads, C::kSmemBytes);
  const unsigned grid = static_cast<unsigned>(2 * (a.tasks < pairs ? a.tasks : pairs));
  kern<<<grid, kKwThreads, C::kSmemBytes, stream>>>(tq, tk, a);
  if ((e = cudaGetLastError()) != cudaSuccess || pieces == 1) return e;
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
                            w, n, pieces);
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
