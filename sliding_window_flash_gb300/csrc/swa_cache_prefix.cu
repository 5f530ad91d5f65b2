// swa_cache_prefix.cu — attention of a batch over the prefix whose pages all its sequences share: the
// prefix is walked once for the rows of all sequences instead of once for each sequence.
//
// The B G T query rows of a kv head meet the same keys, so this is a product of matrices again: 4 D
// flops for each row and slot against 2 D bytes a slot, which the memory bounds up to some 150 rows and
// the tensor cores beyond.  A CTA takes 128 rows of a kv head and a part of their chunks (128 keys, 64 at
// D = 256), on tcgen05:
//   * 2 warps turn keys and 4 values into fp16 operands: codes are read from global memory a chunk ahead
//     into registers, converted (exact, cvt.f16x2.e4m3x2) and stored in the swizzled layouts of the tensor
//     core, keys K-major, values MN-major, which is how tokens lie anyway.
//   * One warp issues S = Q K^T two chunks ahead of O += P V; P goes back to TMEM as the A operand.
//   * 8 warps are the softmax, 16 whole rows each (four threads a row), against a running maximum that moves
//     only when a chunk's sum calls for it.
//   * Where 128 chunks lie, their pages and their scales, is looked up by all threads at once and kept in
//     shared memory, which leaves the loops few registers to hold: what spills would miss the little L1
//     that operands of 200 KB leave.  A chunk has slots of up to four pages, and a tile rows of sequences of
//     different lengths, so of each 32 slots it is known which some row's sequence sees: of others neither
//     table entry nor scale is read, and their values count as zero.
// q is taken as fp16 after scaling each row by a power of two, as in swa_cache_attn.cu.  Keys carry their
// block's scale into the scores' factor; values are scaled by theirs relative to the largest of the item's
// chunks, exactly while a scale is at least 2^-15 of it (a code is a multiple of 2^-9, an fp16 value of 2^-24).
// Parts leave fp32 partial results; swa_cache_attn.cu joins them with those of the slots behind the prefix.
//
// What bounds it: the softmax warps, two to a scheduler.  A chunk of 128 keys takes them some 2,200 cycles
// (about 900 the exponentials, 260 reading scores, 190 the vote whether they stand, the rest waits and the
// loop), its two products 1,024 and its operands less than that beside them; without the products or the
// conversions the kernel takes the same time within 8 %.  A part's beginning and end, run once, take 13 us
// of instructions to fetch and waits one behind the other.  64 sequences, 32 / 8 heads, D = 128, a prefix of
// 32,768: 48-51 us alone (34 GFLOP, 67 MB); 12 sequences, 5 tokens, 32 / 16 heads, D = 256, a prefix of 4,096: 28.
// It begins while the walk over the sequences' own slots ends, and the join while it ends: 79-80 and 71 us in
// all.  The first item's rows come while its chunks are looked up (1 us of the smallest calls' 15 to 17, large
// ones the same).  Tried: operands fetched register by register while they are converted (90 us), more
// than 16 warps (96 registers each, which spill), masks in the passes instead of in TMEM (spilled), the next
// chunk's first scores read while the warp judges this one's (a few spills; 87 us).
#include <climits>
#include <type_traits>

#include "swa_cache_prefix.h"
#include "swa_ptx.cuh"

namespace swa {
namespace {

constexpr float kRescaleThreshold = 8.0f;  // the maximum moves past 2^8
constexpr float kFastSumLimit = 4096.0f;   // a chunk's one-pass sum stands up to 2^12

template <int D>
struct PrefixCfg {
  static constexpr int KT = D == 256 ? 64 : 128;  // keys of a chunk
  static constexpr int kBlock = 128;              // chunks that are looked up together
  static constexpr int kGroups = KT / 32;         // of 32 keys, each inside one page
  static constexpr int kQBytes = kPrefixRows * D * 2;
  static constexpr int kQChunk = kPrefixRows * 128;
  static constexpr int kKVBytes = KT * D * 2;
  static constexpr int kKVChunk = KT * 128;
  static constexpr int kKStages = D == 256 ? 2 : 3;
  static constexpr int kVStages = 2;
  static constexpr int kOffK = kQBytes;
  static constexpr int kOffV = kOffK + kKStages * kKVBytes;
  static constexpr int kOffFirst = kOffV + kVStages * kKVBytes;
  static constexpr int kOffRange = kOffFirst + (kPrefixTiles + 2) * 8;
  static constexpr int kOffRec = kOffRange + kPrefixTiles * 16;  // what is known about kBlock chunks
  static constexpr int kOffMax = kOffRec + kBlock * 80;          // largest value scales of their items
  static constexpr int kOffSeen = kOffMax + kBlock * 4;          // the slots that each row sees
  static constexpr int kOffSeq = kOffSeen + kPrefixRows * 8;  // and each sequence
  static constexpr int kOffBar = kOffSeq + kPrefixSeqs * 8;
  static constexpr int kQFull = 0;
  static constexpr int kKFull = 1;
  static constexpr int kKEmpty = kKFull + kKStages;
  static constexpr int kVFull = kKEmpty + kKStages;
  static constexpr int kVEmpty = kVFull + kVStages;
  static constexpr int kSFull = kVEmpty + kVStages;  // 2
  static constexpr int kPFull = kSFull + 2;          // 2
  static constexpr int kPVDone = kPFull + 2;         // 2
  static constexpr int kOEmpty = kPVDone + 2;
  static constexpr int kDrain = kOEmpty + 1;
  static constexpr int kNumBars = kDrain + 1;
  static constexpr int kSmemBytes = kOffBar + kNumBars * 8 + 16;  // + TMEM address and abort flag
  static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");
  // TMEM: two S buffers, O, two P buffers of packed pairs
  static constexpr uint32_t kColS = 0, kColO = 2 * KT, kColP = 2 * KT + D;
  static_assert(kColP + KT <= 512, "tensor memory");
  // Warps 0-7 softmax, 8 and 9 keys, 10-13 values, 14 products: more than 16 would have fewer than 128
  // registers each, and spill.
  static constexpr int kSoftmaxWarps = 8, kKeyWarps = 2, kValueWarps = 4;
  static constexpr int kKeyWarp = kSoftmaxWarps, kValueWarp = kKeyWarp + kKeyWarps;
  static constexpr int kMmaWarp = kValueWarp + kValueWarps;
  static constexpr int kThreads = 32 * (kMmaWarp + 1);
};

__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u)
      : "memory");
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The prefix slots that the rows of a tile see: the lowest length and the highest end of its sequences that
// have queries, and the same the other way round (what all of them see).
struct TileRange {
  int len_min, end_max, len_max_q, end_min;  // len_max_q: the last query's slot of the longest
};

// The chunks of a tile in order, as ChunkWalk.
struct TileWalk {
  int far, first, count;
  __device__ TileWalk(const TileRange& t, const Reach& r, int ck) {
    const int end = min(t.end_max, r.base);  // slots from here on nobody sees
    const int last = end > 0 ? (end - 1) / ck : -1;
    first = visible_lo(t.len_min, r.window) / ck;
    far = min(min((r.sinks + ck - 1) / ck, first), last + 1);
    count = far + max(0, last - first + 1);
  }
  __device__ int at(int i) const { return i < far ? i : first + (i - far); }
};

// What is known about a chunk: its item and first slot, the index in its block of its item's first chunk
// there, and for each group of 32 keys the plane (page * Hkv + head, or -1: nothing to be seen), scales, and
// which of the keys the sequences of the tile's rows see.
struct ChunkRec {
  int item, slot, origin;
  int edge;  // some row of the tile does not see some of it
  int plane[4];
  float ks[4], vs[4];
  unsigned seen[4];
};
static_assert(sizeof(ChunkRec) == 80, "kOffRec");

// Those of the 32 slots from `slot` on that lie in [lo, end), as bits.
__device__ __forceinline__ unsigned slot_bits(int slot, int lo, int end) {
  const int a = max(lo - slot, 0), z = min(end - slot, 32);
  return a < z ? (0xffffffffu << a) & (0xffffffffu >> (32 - z)) : 0u;
}
// Those that a sequence sees whose queries begin to see at `lo` and end at `end`.
__device__ __forceinline__ unsigned seen_bits(int slot, int lo, int end, int sinks) {
  return slot_bits(slot, lo, end) | slot_bits(slot, 0, min(sinks, end));
}

__device__ __forceinline__ uint4 load_codes(const uint4* p) {  // read once, and not from the L1 (load_global)
  uint4 v;
  asm volatile("ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <int D>
__global__ void __launch_bounds__(PrefixCfg<D>::kThreads, 1)
    swa_cache_prefix_kernel(const CacheView c, const PrefixDev a) {
  using C = PrefixCfg<D>;
  constexpr int KT = C::KT;
  extern __shared__ __align__(1024) uint8_t smem[];
  launch_dependents();  // (the walk ahead waited for all that is read here before it let this kernel begin)
  if (!smem_base_ok(smem, c.err)) {
    wait_predecessor();
    return;
  }
  int64_t* s_first = reinterpret_cast<int64_t*>(smem + C::kOffFirst);
  TileRange* s_range = reinterpret_cast<TileRange*>(smem + C::kOffRange);
  int2* s_seq = reinterpret_cast<int2*>(smem + C::kOffSeq);  // first slot seen (sinks aside), and the end
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kNumBars);
  int& abort_flag = *reinterpret_cast<int*>(tmem_slot + 1);
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  const uint32_t sQ = smem_u32(smem), sK0 = smem_u32(smem + C::kOffK), sV0 = smem_u32(smem + C::kOffV);
  const uint32_t warp = warp_id(), lane = lane_id();

  if (threadIdx.x == 0) {
    abort_flag = 0;
    mbar_init(bar(C::kQFull), C::kSoftmaxWarps);
    for (int s = 0; s < C::kKStages; ++s) {
      mbar_init(bar(C::kKFull + s), C::kKeyWarps);
      mbar_init(bar(C::kKEmpty + s), 1);
    }
    for (int s = 0; s < C::kVStages; ++s) {
      mbar_init(bar(C::kVFull + s), C::kValueWarps);
      mbar_init(bar(C::kVEmpty + s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar(C::kSFull + b), 1);
      mbar_init(bar(C::kPFull + b), C::kSoftmaxWarps);
      mbar_init(bar(C::kPVDone + b), 1);
    }
    mbar_init(bar(C::kOEmpty), C::kSoftmaxWarps);
    mbar_init(bar(C::kDrain), 1);
    fence_barrier_init();
  }
  // What each tile's rows see: a warp a tile, its lanes the tile's sequences.
  for (int j = static_cast<int>(warp); j < a.tiles; j += C::kThreads / 32) {
    const int b0 = static_cast<int>(a.div_r.div(static_cast<uint32_t>(j) * kPrefixRows));
    const int last = min(a.rows, (j + 1) * kPrefixRows) - 1;
    const int b1 = static_cast<int>(a.div_r.div(static_cast<uint32_t>(last)));
    int len_min = INT_MAX, end_max = 0, q_max = 0, end_min = INT_MAX;
    for (int b = b0 + static_cast<int>(lane); b <= b1; b += 32) {
      int len, n;
      const bool asks = sequence_of<true>(c, b, &len, &n) && n > 0;
      // (a sequence of two tiles gets the same from both)
      s_seq[b] = asks ? make_int2(visible_lo(len, a.reach.window), min(len + n, a.reach.base)) : make_int2(0, 0);
      if (!asks) continue;
      len_min = min(len_min, len);
      end_max = max(end_max, len + n);
      q_max = max(q_max, len + n - 1);
      end_min = min(end_min, len + 1);
    }
    len_min = __reduce_min_sync(0xffffffffu, len_min);
    end_max = __reduce_max_sync(0xffffffffu, end_max);
    q_max = __reduce_max_sync(0xffffffffu, q_max);
    end_min = __reduce_min_sync(0xffffffffu, end_min);
    if (lane == 0) s_range[j] = TileRange{end_max > 0 ? len_min : 0, end_max, q_max, end_min};
  }
  if (warp == C::kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  __syncthreads();
  if (warp == 0) {  // chunks before each tile
    int64_t sum = 0;
    for (int j0 = 0; j0 <= a.tiles; j0 += 32) {
      const int j = j0 + static_cast<int>(lane);
      const int64_t own = j < a.tiles ? TileWalk(s_range[j], a.reach, KT).count : 0;
      int64_t scan = own;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, scan, d);
        if (static_cast<int>(lane) >= d) scan += up;
      }
      if (j <= a.tiles) s_first[j] = sum + scan - own;
      sum += __shfl_sync(0xffffffffu, scan, 31);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (blockIdx.x == 0)
    for (int j = static_cast<int>(threadIdx.x); j <= a.tiles; j += C::kThreads) a.first[j] = s_first[j];

  const int64_t total = s_first[a.tiles] * c.Hkv;
  const Parts cut(total, prefix_parts(total, a.parts, a.stored, D));
  const int part = static_cast<int>(blockIdx.x);
  const int64_t begin = part < cut.parts ? cut.start(part) : total;
  const int count = part < cut.parts ? static_cast<int>(cut.start(part + 1) - begin) : 0;

  ChunkRec* s_rec = reinterpret_cast<ChunkRec*>(smem + C::kOffRec);
  unsigned* s_max = reinterpret_cast<unsigned*>(smem + C::kOffMax);
  // Which of 32 slots some sequence of tile j's rows sees.  The one whose end is the last sees all of them
  // nearly always; where it does not (an edge, a sink, or slots between two sequences' windows), all are asked.
  auto group_seen = [&](int j, int slot) -> unsigned {
    const TileRange r = s_range[j];
    const int end = min(r.end_max, a.reach.base);
    if (slot >= end) return 0u;
    if (slot + 32 <= end && slot >= visible_lo(r.len_max_q, a.reach.window)) return 0xffffffffu;
    const int b0 = static_cast<int>(a.div_r.div(static_cast<uint32_t>(j) * kPrefixRows));
    const int last = min(a.rows, (j + 1) * kPrefixRows) - 1;
    const int b1 = static_cast<int>(a.div_r.div(static_cast<uint32_t>(last)));
    unsigned bits = 0u;
#pragma unroll 1
    for (int b = b0; b <= b1; ++b) bits |= seen_bits(slot, s_seq[b].x, s_seq[b].y, a.reach.sinks);
    return bits;
  };
  // Looks up the part's chunks from i0 on, a thread a group of 32 keys.  The first block is for the warps
  // behind the softmax's, which load their first rows meanwhile and meet them at barrier 2.  Every thread of
  // the CTA comes here for every further block, whatever became of its work on the one before.
  constexpr int kFirstThread = 32 * C::kSoftmaxWarps;
  auto look_up = [&](int i0) {
    const bool all = i0 > 0;
    const int tid = static_cast<int>(threadIdx.x) - (all ? 0 : kFirstThread);
    const int threads = C::kThreads - (all ? 0 : kFirstThread);
    auto meet = [&] {
      if (all)
        __syncthreads();
      else
        named_barrier_sync(1, C::kThreads - kFirstThread);
    };
    if (all) __syncthreads();  // the block before has been read
    for (int i = tid; i < C::kBlock; i += threads) s_max[i] = 0u;
    meet();
    const int end = min(4 * C::kBlock, (4 * (count - i0) + 31) & ~31);
    for (int at = tid; at < end; at += threads) {  // whole warps
      const int rec = at / 4, group = at & 3, i = i0 + rec;
      int plane = -1;
      if (i < count) {
        const int64_t x = begin + i;
        const int j = sequence_at(s_first, a.tiles, c.Hkv, x);
        const int64_t nc = s_first[j + 1] - s_first[j], rem = x - s_first[j] * c.Hkv;
        const int h = static_cast<int>(quotient(rem, nc)), cc = static_cast<int>(rem - h * nc);
        const int slot0 = TileWalk(s_range[j], a.reach, KT).at(cc) * KT, slot = slot0 + 32 * group;
        const int origin = max(rec - cc, 0);
        float ks = 1.f, vs = 0.f;
        const unsigned seen = group < C::kGroups && slot < a.reach.base ? group_seen(j, slot) : 0u;
        if (seen != 0u) {
          const int page = page_of<true>(c, a.table, 0, slot >> a.page_log2, c.max_pages);
          if (page >= 0) {
            plane = page * c.Hkv + h;
            ks = load_global<true>(c.k_scale + plane);
            vs = load_global<true>(c.v_scale + plane);
            atomicMax(&s_max[origin], __float_as_uint(vs));
          }
        }
        ChunkRec& to = s_rec[rec];
        to.plane[group] = plane;
        to.ks[group] = ks;
        to.vs[group] = vs;
        to.seen[group] = seen;
        if (group == 0) {
          to.item = j * c.Hkv + h;
          to.slot = slot0;
          to.origin = origin;
        }
      }
      const unsigned there = __ballot_sync(0xffffffffu, plane >= 0) >> (lane & 28u);
      constexpr unsigned kAll = (1u << C::kGroups) - 1u;
      if (i < count && group == 0) {
        ChunkRec& to = s_rec[rec];
        const TileRange range = s_range[static_cast<int>(a.div_hkv.div(static_cast<uint32_t>(to.item)))];
        to.edge = (there & kAll) != kAll || to.slot + KT > min(range.end_min, a.reach.base) ||
                  (to.slot < visible_lo(range.len_max_q, a.reach.window) &&
                   to.slot + KT > a.reach.sinks);
      }
    }
    meet();
  };
  // The value reference: the largest scale of the item's chunks so far, a block of chunks at a time; it moves
  // where an item or a block begins.  Where a part's first block has nothing to be seen it is the least scale.
  constexpr float kLeastScale = 1.f / (1ll << -kScaleMinExp);
  auto reference = [&](const ChunkRec& rec, float vref, bool starts) {
    const float top = __uint_as_float(s_max[rec.origin]);
    return fmaxf(starts ? kLeastScale : vref, top);
  };

  if (warp >= C::kSoftmaxWarps) {
    look_up(0);
    named_barrier_arrive(2, C::kThreads);
  }
  if (warp >= C::kKeyWarp && warp < C::kMmaWarp) {
    // ------------------------------------------------------------------ codes to operands
    // A thread has the codes of the next chunk on their way while it converts this one's.
    int item = -1, stage = 0;
    uint32_t phase = 1;  // the first round of stages is free
    float vref = 1.f;
    auto walk = [&](auto kind) {
      constexpr bool kValues = decltype(kind)::value;
      const uint8_t* pool = kValues ? c.v : c.k;
      constexpr int kUnitsRow = D / 16;  // 16 codes each
      constexpr int kThr = 32 * (kValues ? C::kValueWarps : C::kKeyWarps), kRowsPass = kThr / kUnitsRow;
      constexpr int kPasses = KT / kRowsPass;  // units of a thread in a tile
      static_assert(32 % kRowsPass == 0, "a pass lies within a group");
      const int tid = static_cast<int>(threadIdx.x) - 32 * (kValues ? C::kValueWarp : C::kKeyWarp), cu = tid % kUnitsRow;
      // Neighbouring 64-column pieces of a row go to the same banks: every other one is taken a row on.
      const int row0 = (tid / kUnitsRow) ^ ((cu >> 2) & 1);
      const uint32_t piece = static_cast<uint32_t>(cu >> 2) * C::kKVChunk, unit = 2u * (cu & 3);
      uint4 codes[kPasses];
      auto fetch = [&](int i) {
        const ChunkRec& rec = s_rec[i];
#pragma unroll
        for (int g = 0; g < C::kGroups; ++g) {
          const int pl = rec.plane[g];
          const uint4* src = reinterpret_cast<const uint4*>(
                                 pool + (static_cast<size_t>(max(pl, 0)) * c.page +
                                         ((rec.slot + 32 * g) & (c.page - 1)) + row0) * D) + cu;
#pragma unroll
          for (int p = 0; p < 32 / kRowsPass; ++p)
            codes[g * (32 / kRowsPass) + p] =
                pl >= 0 ? load_codes(src + p * kRowsPass * kUnitsRow) : make_uint4(0u, 0u, 0u, 0u);
        }
      };
      // 16 codes as fp16, values times `ratio`, into a row of a tile
      auto put = [&](uint32_t tile, int row, uint4 w, uint32_t ratio) {
        uint32_t y[8];
        e4m3x4_to_f16(w.x, y[0], y[1]);
        e4m3x4_to_f16(w.y, y[2], y[3]);
        e4m3x4_to_f16(w.z, y[4], y[5]);
        e4m3x4_to_f16(w.w, y[6], y[7]);
        if constexpr (kValues) {
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = mul_f16x2(y[i], ratio);
        }
        const uint32_t to = tile + piece, ur = static_cast<uint32_t>(row);
        st_shared_v4(to + sw128_offset(ur, unit), y[0], y[1], y[2], y[3]);
        st_shared_v4(to + sw128_offset(ur, unit + 1), y[4], y[5], y[6], y[7]);
      };
      // Record i of `n` of a block of chunks: its codes become the operand, and those of the next one are sent
      // for.
      auto step = [&](int i, int n) -> bool {
        const ChunkRec& rec = s_rec[i];
        const bool starts = rec.item != item;
        item = rec.item;
        uint32_t ratio[C::kGroups] = {};
        if constexpr (kValues) {
          if (starts || i == 0) vref = reference(rec, vref, starts);
          const float inv = 1.f / vref;
#pragma unroll
          for (int o = 0; o < C::kGroups; ++o) ratio[o] = half2_of(rec.vs[o] * inv);
          // what nobody sees must not meet a probability of zero as infinity or NaN
          if (rec.edge) {
#pragma unroll
            for (int p = 0; p < kPasses; ++p)
              if ((rec.seen[p * kRowsPass / 32] >> (row0 + p * kRowsPass % 32) & 1u) == 0u)
                codes[p] = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        constexpr int kStages = kValues ? C::kVStages : C::kKStages;
        constexpr int kFull = kValues ? C::kVFull : C::kKFull, kEmpty = kValues ? C::kVEmpty : C::kKEmpty;
        if (!warp_wait(bar(kEmpty + stage), phase, &abort_flag, c.err)) return false;
        const uint32_t tile = (kValues ? sV0 : sK0) + static_cast<uint32_t>(stage) * C::kKVBytes;
#pragma unroll
        for (int p = 0; p < kPasses; ++p)
          put(tile, row0 + p * kRowsPass, codes[p], ratio[p * kRowsPass / 32]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kFull + stage));
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
        if (i + 1 < n) fetch(i + 1);
        return true;
      };
      bool ok = true;
      for (int i0 = 0; i0 < count; i0 += C::kBlock) {
        if (i0 > 0) look_up(i0);
        const int n = min(C::kBlock, count - i0);
        if (ok) fetch(0);
        for (int i = 0; ok && i < n; ++i) ok = step(i, n);
      }
    };
    const bool values = warp >= C::kValueWarp;
    if (values)
      walk(std::true_type{});
    else
      walk(std::false_type{});
  } else if (warp == C::kMmaWarp) {
    // ------------------------------------------------------------------ products
    constexpr uint32_t kIdS = idesc_f16kind(0u, kPrefixRows, KT, false, false);
    constexpr uint32_t kIdO = idesc_f16kind(0u, kPrefixRows, D, false, true);
    // S_g = Q K_g^T into buffer g & 1, whose scores before have become P.
    auto issue_s = [&](int g) -> bool {
      const int s = g % C::kKStages;
      if (!warp_wait(bar(C::kKFull + s), (g / C::kKStages) & 1, &abort_flag, c.err)) return false;
      tc_fence_after();
      const uint64_t da = smem_desc_sw128(sQ, 16, 1024);
      const uint64_t db = smem_desc_sw128(sK0 + s * C::kKVBytes, 16, 1024);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
        umma_ss(tmem + C::kColS + KT * (g & 1), da + (ks / 4) * (C::kQChunk >> 4) + 2 * (ks % 4),
                db + (ks / 4) * (C::kKVChunk >> 4) + 2 * (ks % 4), kIdS, ks > 0);
      umma_commit_w(bar(C::kSFull + (g & 1)));
      umma_commit_w(bar(C::kKEmpty + s));
      return true;
    };
    auto issue_pv = [&](int g, bool first) -> bool {  // O (+)= P_g V_g
      const int s = g % C::kVStages;
      if (!warp_wait(bar(C::kVFull + s), (g / C::kVStages) & 1, &abort_flag, c.err)) return false;
      if (!warp_wait(bar(C::kPFull + (g & 1)), (g >> 1) & 1, &abort_flag, c.err)) return false;
      tc_fence_after();
      const uint64_t db = smem_desc_sw128(sV0 + s * C::kKVBytes, C::kKVChunk, 1024);
#pragma unroll
      for (int ks = 0; ks < KT / 16; ++ks)
        umma_ts(tmem + C::kColO, tmem + C::kColP + KT / 2 * (g & 1) + 8 * ks, db + 128 * ks, kIdO,
                !first || ks > 0);
      umma_commit_w(bar(C::kPVDone + (g & 1)));
      umma_commit_w(bar(C::kVEmpty + s));
      return true;
    };
    // S runs up to two chunks ahead, within an item: the next one's Q takes the place of this one's.
    bool ok = true;
    int item = -1, seg = -1, ahead = 0;  // chunks whose S has been issued
    for (int i0 = 0; i0 < count; i0 += C::kBlock) {
      if (i0 > 0) look_up(i0);
      const int end = min(count, i0 + C::kBlock);
      for (int g = i0; ok && g < end; ++g) {
        const int it = s_rec[g - i0].item;
        const bool starts = it != item;
        if (starts) {
          ++seg;
          item = it;
          ok = warp_wait(bar(C::kQFull), seg & 1, &abort_flag, c.err);
        }
        while (ok && ahead < min(end, g + 2) && s_rec[ahead - i0].item == it) ok = issue_s(ahead++);
        // an item's first P V overwrites O, which the epilogue of the one before has read
        if (ok && starts && seg > 0) ok = warp_wait(bar(C::kOEmpty), (seg - 1) & 1, &abort_flag, c.err);
        if (ok) ok = issue_pv(g, starts);
      }
    }
    umma_commit_w(bar(C::kDrain));  // nothing issued is left running
    warp_drain_wait(bar(C::kDrain), 0, c.err);
  } else {
    // ------------------------------------------------------------------ softmax
    // Thread t of warp w has rows R0 = 32 (w % 4) + 16 (w / 4) + t / 4 and R1 = R0 + 8, and of every 8 columns
    // the columns 2 kq, 2 kq + 1 (kq = t % 4): the 16x256b shape of TMEM.  Four threads have a row.
    constexpr int kHalves = KT / 64;  // 64 columns at a time
    const uint32_t lane0 = 32u * (warp & 3u) + 16u * (warp >> 2), lane_base = lane0 << 16;
    const int r0 = static_cast<int>(lane0 + (lane >> 2)), kq = static_cast<int>(lane & 3u);
    auto row_max = [](float v) {
      v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
      return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
    };
    auto row_sum = [](float v) {
      v += __shfl_xor_sync(0xffffffffu, v, 1);
      return v + __shfl_xor_sync(0xffffffffu, v, 2);
    };
    int2* s_seen = reinterpret_cast<int2*>(smem + C::kOffSeen);
    int item = -1;
    bool begins = false, ok = true;
    float f[2], m[2], l[2], vref = 1.f;

    // Loads this thread's quarters of its rows of q into the Q tile, scaled.  They come there as they are, with
    // their largest magnitude, and a loop scales them: straight code for all of it is run once and takes as
    // long as its instructions take to be fetched (the start of an item 19,000 cycles at D = 256, 8,500 now).
    auto start = [&](int j, int head) {
      uint32_t top[2] = {0u, 0u};
      uint32_t place[2];
      uint4 raw[2][D / 32];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = r0 + 8 * e, rho = j * kPrefixRows + r;
        bool is = false;
        int2 seen = make_int2(0, INT_MAX);  // rows that stand for nothing need no mask
        const uint16_t* row = a.q;
        if (rho < a.rows) {
          const int b = static_cast<int>(a.div_r.div(static_cast<uint32_t>(rho)));
          const int in_seq = rho - b * a.R, t = static_cast<int>(a.div_t.mod(static_cast<uint32_t>(in_seq)));
          int len, n;
          is = sequence_of<true>(c, b, &len, &n) && t < n;
          if (is) {
            seen = make_int2(visible_lo(len + t, a.reach.window), min(len + t, a.reach.base - 1));
            row += ((static_cast<size_t>(b) * c.Hkv + head) * a.R + in_seq) * D;
          }
        }
        if (kq == 0) s_seen[r] = seen;
        // units kq and kq + 4 of every 64 columns
        place[e] = sQ + sw128_offset(static_cast<uint32_t>(r), static_cast<uint32_t>(kq));
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
          raw[e][i] = is ? __ldcg(reinterpret_cast<const uint4*>(row) + 4 * i + kq) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const uint4 y = raw[e][i];
          top[e] = __vmaxu2(top[e], __vmaxu2(__vmaxu2(y.x & 0x7fff7fffu, y.y & 0x7fff7fffu),
                                             __vmaxu2(y.z & 0x7fff7fffu, y.w & 0x7fff7fffu)));
          st_shared_v4((place[e] ^ (64u * (i & 1))) + (i >> 1) * C::kQChunk, y.x, y.y, y.z, y.w);
        }
      }
      float up[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t most = max(top[e] & 0xffffu, top[e] >> 16);
        most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
        const uint32_t bits =
            __float_as_uint(a.f16 ? Elem<true>::unpack(most).x : Elem<false>::unpack(most).x);
        const int ex = static_cast<int>(bits >> 23);
        // 2^(14 - exponent); 1 for zero, infinity and NaN
        const int sh = ex == 255 || bits == 0 ? 0 : min(126, 127 + 14 - ex);
        up[e] = __uint_as_float(static_cast<uint32_t>(127 + sh) << 23);
        // a row that is not finite has scores that are all NaN
        f[e] = ex == 255 ? __uint_as_float(0x7fffffffu)
                         : a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - sh) << 23);
      }
#pragma unroll 1
      for (int i = 0; i < D / 32; ++i) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t at = (place[e] ^ (64u * (i & 1))) + (i >> 1) * C::kQChunk;
          uint32_t w[4];
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                       : "r"(at)
                       : "memory");
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const float2 v = a.f16 ? Elem<true>::unpack(w[z]) : Elem<false>::unpack(w[z]);
            w[z] = Elem<true>::pack(v.x * up[e], v.y * up[e]);
          }
          st_shared_v4(at, w[0], w[1], w[2], w[3]);
        }
      }
      m[0] = m[1] = SWA_NEG_INF;
      l[0] = l[1] = 0.f;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::kQFull));
    };

    // The item's partial result after its chunk g at `slot`.
    auto finish = [&](int g, int slot) -> bool {
      const float sum0 = row_sum(l[0]), sum1 = row_sum(l[1]);
      if (!warp_wait(bar(C::kPVDone + (g & 1)), (g >> 1) & 1, &abort_flag, c.err)) return false;
      tc_fence_after();
      const int j = static_cast<int>(a.div_hkv.div(static_cast<uint32_t>(item)));
      const TileWalk walk(s_range[j], a.reach, KT);
      const bool ends = slot == walk.at(walk.count - 1) * KT;
      const int at = begins && ends ? 2 * a.parts + item : partial_slot(part, begins);
      const size_t to = static_cast<size_t>(at) * a.stored + r0;
      const bool real[2] = {s_seen[r0].y != INT_MAX, s_seen[r0 + 8].y != INT_MAX};
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 64) {
        uint32_t rr[32];
        tmem_ld16x256_x8(tmem + lane_base + C::kColO + c0, rr);
        tmem_wait_ld(rr);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (real[e]) {
            float* out = a.po + (to + 8 * e) * D + c0 + 2 * kq;
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<float2*>(out + 8 * i) =
                  make_float2(__uint_as_float(rr[4 * i + 2 * e]) * vref,
                              __uint_as_float(rr[4 * i + 2 * e + 1]) * vref);
          }
        }
      }
      warp_arrive(bar(C::kOEmpty));
      if (kq == 0) {
        if (real[0]) *reinterpret_cast<float2*>(a.ml + to * 2) = make_float2(m[0], sum0);
        if (real[1]) *reinterpret_cast<float2*>(a.ml + (to + 8) * 2) = make_float2(m[1], sum1);
      }
      return true;
    };

    int last_slot = 0;
    if (count > 0) {  // the part's first item, known without the look-up
      const int j = sequence_at(s_first, a.tiles, c.Hkv, begin);
      const int64_t nc = s_first[j + 1] - s_first[j], rem = begin - s_first[j] * c.Hkv;
      const int head = static_cast<int>(quotient(rem, nc));
      item = j * c.Hkv + head;
      begins = rem == head * nc;
      start(j, head);
    }
    named_barrier_sync(2, C::kThreads);
    for (int i0 = 0; i0 < count; i0 += C::kBlock) {
      if (i0 > 0) look_up(i0);
      for (int g = i0; ok && g < min(count, i0 + C::kBlock); ++g) {
        const ChunkRec& rec = s_rec[g - i0];
        const int slot = rec.slot;
        const bool starts = rec.item != item || g == 0;
        if (rec.item != item) {
          if (!(ok = finish(g - 1, last_slot))) break;
          item = rec.item;
          const int j = static_cast<int>(a.div_hkv.div(static_cast<uint32_t>(item)));
          begins = slot == TileWalk(s_range[j], a.reach, KT).at(0) * KT;
          start(j, item - j * c.Hkv);
        }
        last_slot = slot;
        float fac[2] = {1.f, 1.f};  // of o and the sums so far
        if (starts || g == i0) {
          const float was = vref;
          vref = reference(rec, vref, starts);
          if (!starts) fac[0] = fac[1] = was / vref;
        }
        if (!(ok = warp_wait(bar(C::kSFull + (g & 1)), (g >> 1) & 1, &abort_flag, c.err))) break;
        // That these scores are there says too that P V of chunk g - 2, issued before them, has read the P buffer.
        tc_fence_after();
        const uint32_t s_addr = tmem + lane_base + C::kColS + KT * (g & 1);
        // 64 columns of this thread's rows: x[4 i], x[4 i + 1] of R0 and x[4 i + 2], x[4 i + 3] of R1.  They
        // are read from TMEM for each pass.
        auto scores = [&](float (&x)[kHalves][32]) {
          uint32_t rr[kHalves][32];
#pragma unroll
          for (int half = 0; half < kHalves; ++half) tmem_ld16x256_x8(s_addr + 64u * half, rr[half]);
          tmem_wait_ld_all();
#pragma unroll
          for (int half = 0; half < kHalves; ++half) {
            reg_fence(rr[half]);
#pragma unroll
            for (int i = 0; i < 32; ++i) x[half][i] = __uint_as_float(rr[half][i]);
          }
        };
        if (rec.edge) {  // what a row does not see becomes -inf, in TMEM: the passes need no mask of their own
          const int2 seen[2] = {s_seen[r0], s_seen[r0 + 8]};
#pragma unroll 1
          for (int half = 0; half < kHalves; ++half) {
            uint32_t rr[32];
            tmem_ld16x256_x8(s_addr + 64u * half, rr);
            tmem_wait_ld(rr);
#pragma unroll
            for (int o = 0; o < 2; ++o) {  // groups of 32 columns
              const int s0 = slot + 64 * half + 32 * o + 2 * kq, csink = a.reach.sinks - s0;
              const bool there = rec.plane[2 * half + o] >= 0;
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int clo = seen[e].x - s0, chi = there ? seen[e].y - s0 : -1;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                  for (int z = 0; z < 2; ++z) {
                    uint32_t& y = rr[16 * o + 4 * i + 2 * e + z];
                    const int at = 8 * i + z;
                    y = (at >= clo || at < csink) && at <= chi ? y : __float_as_uint(SWA_NEG_INF);
                  }
              }
            }
            tmem_st16x256_x8(s_addr + 64u * half, rr);
          }
          tmem_wait_st();
        }
        // a masked score times zero would be NaN
        auto factor_of = [&](int e, int o) {
          const float y = f[e] * rec.ks[o];
          return y < 1e-37f ? 1e-37f : y;
        };
        // One pass against the reference maxima; redone exactly on an item's first chunk or when a thread's
        // part of a row's sum exceeds 2^12.
        float sum[2];
        bool exact = !__all_sync(0xffffffffu, m[0] != SWA_NEG_INF && m[1] != SWA_NEG_INF);
        for (;;) {
          if (exact) {
            float mx[2] = {SWA_NEG_INF, SWA_NEG_INF};
#pragma unroll 1
            for (int half = 0; half < kHalves; ++half) {
              float x[32];
              {
                uint32_t rr[32];
                tmem_ld16x256_x8(s_addr + 64u * half, rr);
                tmem_wait_ld(rr);
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(rr[i]);
              }
#pragma unroll
              for (int o = 0; o < 2; ++o)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  float top = fmaxf(x[16 * o + 2 * e], x[16 * o + 2 * e + 1]);
#pragma unroll
                  for (int i = 1; i < 4; ++i)
                    top = fmaxf(top, fmaxf(x[16 * o + 4 * i + 2 * e], x[16 * o + 4 * i + 2 * e + 1]));
                  mx[e] = fmaxf(mx[e], top * factor_of(e, 2 * half + o));
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float now = fmaxf(m[e], row_max(mx[e]));
              if (now > m[e] + kRescaleThreshold) {
                const float down = ex2(m[e] - now);  // 0 when m is -inf
                fac[e] *= down;
                l[e] *= down;
                m[e] = now;
              }
            }
          }
          const float at0 = m[0] == SWA_NEG_INF ? 0.f : m[0], at1 = m[1] == SWA_NEG_INF ? 0.f : m[1];
          float2 s0 = make_float2(0.f, 0.f), s1 = s0;
          float y[kHalves][32];
          scores(y);
#pragma unroll
          for (int half = 0; half < kHalves; ++half) {
            const float (&x)[32] = y[half];
            uint32_t pk[16];  // pk[2 i] of R0, pk[2 i + 1] of R1: packed column 4 i + kq
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float g0 = factor_of(0, 2 * half + i / 4), g1 = factor_of(1, 2 * half + i / 4);
              const float2 t0 = __ffma2_rn(make_float2(x[4 * i], x[4 * i + 1]), make_float2(g0, g0),
                                           make_float2(-at0, -at0));
              const float2 t1 = __ffma2_rn(make_float2(x[4 * i + 2], x[4 * i + 3]), make_float2(g1, g1),
                                           make_float2(-at1, -at1));
              const float2 e0 = make_float2(ex2(t0.x), ex2(t0.y)), e1 = make_float2(ex2(t1.x), ex2(t1.y));
              s0 = __fadd2_rn(s0, e0);
              s1 = __fadd2_rn(s1, e1);
              pk[2 * i] = Elem<true>::pack(e0.x, e0.y);
              pk[2 * i + 1] = Elem<true>::pack(e1.x, e1.y);
            }
            tmem_st16x128_x8(tmem + lane_base + C::kColP + KT / 2 * (g & 1) + 32u * half, pk);
          }
          sum[0] = s0.x + s0.y;
          sum[1] = s1.x + s1.y;
          if (exact) break;
          if (!__any_sync(0xffffffffu, !(sum[0] <= kFastSumLimit) || !(sum[1] <= kFastSumLimit))) break;
          exact = true;
        }
        l[0] += sum[0];
        l[1] += sum[1];
        if (!starts && __any_sync(0xffffffffu, fac[0] != 1.f || fac[1] != 1.f)) {
          if (!(ok = warp_wait(bar(C::kPVDone + ((g - 1) & 1)), ((g - 1) >> 1) & 1, &abort_flag, c.err)))
            break;
          tc_fence_after();
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 64) {
            const uint32_t oc = tmem + lane_base + C::kColO + c0;
            uint32_t rr[32];
            tmem_ld16x256_x8(oc, rr);
            tmem_wait_ld(rr);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              rr[i] = __float_as_uint(__uint_as_float(rr[i]) * ((i & 2) ? fac[1] : fac[0]));
            tmem_st16x256_x8(oc, rr);
          }
        }
        tmem_wait_st();
        warp_arrive(bar(C::kPFull + (g & 1)));
      }
    }
    if (ok && count > 0) finish(count - 1, last_slot);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  // This kernel may begin while the walk over the sequences' own slots ends; who waits for this one waits
  // for both.
  if (threadIdx.x == 0) wait_predecessor();
}

template <int D>
cudaError_t launch_prefix_d(const CacheView& c, const PrefixDev& a, cudaStream_t stream) {
  using C = PrefixCfg<D>;
  cudaError_t e = allow_smem<swa_cache_prefix_kernel<D>>(C::kSmemBytes);
  if (e != cudaSuccess) return e;
  return launch_early(swa_cache_prefix_kernel<D>, static_cast<unsigned>(a.parts), C::kThreads, C::kSmemBytes,
                      stream, c, a);
}

}  // namespace

PrefixPlan prefix_plan(int B, int Hkv, int R, int D, int base) {
  PrefixPlan p;
  const long long rows = static_cast<long long>(B) * R;
  p.tiles = static_cast<int>((rows + kPrefixRows - 1) / kPrefixRows);
  p.stored = static_cast<int>(rows < kPrefixRows ? rows : kPrefixRows);
  const int64_t items = static_cast<int64_t>(p.tiles) * Hkv, ck = prefix_chunk(D);
  const int64_t chunks = items * ((base + ck - 1) / ck), sms = sm_count();
  // As many parts as SMs, or the least multiple with a part for every item.
  const int64_t most = sms * ((items + sms - 1) / sms);
  p.parts = static_cast<int>(chunks < most ? chunks : most);
  const size_t slots = (2 * static_cast<size_t>(p.parts) + items) * p.stored;
  auto round = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  size_t off = round((kPrefixTiles + 1) * sizeof(int64_t));
  p.off_ml = off;
  off += round(slots * 2 * sizeof(float));
  p.off_po = off;
  off += round(slots * D * sizeof(float));
  p.bytes = off;
  return p;
}

cudaError_t launch_cache_prefix(const CacheView& c, const PrefixDev& a, cudaStream_t stream) {
  if (c.D == 64) return launch_prefix_d<64>(c, a, stream);
  if (c.D == 128) return launch_prefix_d<128>(c, a, stream);
  return launch_prefix_d<256>(c, a, stream);
}

}  // namespace swa
