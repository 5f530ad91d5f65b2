// swa_cache_attn.cu — attention of a few tokens per sequence over the paged e4m3 cache, and the
// accumulation of the weight each cached token received.
//
// Per (sequence, kv head) the R = G T query rows that share a kv head see the same keys:
//   x = scale <q, k>,  o = sum p v,  p = exp(x - lse),  lse = ln sum exp(x).
// Every key and value byte is needed once, 2 D bytes for 4 D R flops, so the memory bounds it and
// the tensor cores (mma.sync, 16 rows a tile) only have to keep up.  What is built around that:
//   * The list of all chunks (32 keys, 16 at D = 256: 8 KB of keys and values at D >= 128) of all
//     items is cut into equal parts, one per team (swa_cache_split.h), so ragged lengths and few
//     heads fill the SMs alike.  One CTA of 8 warps per SM; a team is MT warps with 16 query rows
//     each, in long walks of many rows 32 (MT = 1, 2, 4), which share its ring in shared memory.
//   * Chunks arrive by TMA, swizzled; 192 KB of ring keep 128 KB in flight per SM.  A lane looks up
//     the pages and scales of one of the next 32 chunks, so the walk never waits for a table.
//   * Codes become fp16 exactly (cvt.f16x2.e4m3x2).  S = Q K^T takes keys by ldmatrix, whose 8 x 16
//     byte matrices give each lane 4 consecutive codes; the order of the contraction is permuted
//     the same way in Q.  P V takes two values of neighbouring keys from two rows by byte permutes,
//     which is the transposition that the operand needs; lane group g reads the 16 columns from
//     16 g on, so a row of o ends up 32 columns to a lane.
//   * A block's key scale multiplies its scores; its value scale, divided by the walk's reference
//     scale, multiplies p.  The running maximum and the reference change only when they have to
//     (a score 4 above, in powers of two; a scale outside [ref, 64 ref]), so o is rarely rescaled.
// A second kernel joins the items that several teams shared and answers rows that see nothing; with
// accumulate the first stores its scores, and a third adds exp(x - lse) to the cached tokens' weights.
// With sinks a sequence's list of chunks has those of its sinks before the window's (ChunkWalk).  With a
// shared prefix the list begins behind it, every item leaves a partial result, and the join takes those of
// the prefix (swa_cache_prefix.cu) with them.
//
// Measured in a CUDA graph, D = 128 unless said: 8 sequences of up to 128K tokens, 16 kv heads: 600 us,
// 6.8 TB/s.  64 ragged sequences to 16K with accumulation: 203 us, the walk about 175 of it (5.8 TB/s;
// the last teams end some 15 us after most), the join 8, the weights 20.  A window of 1024: 11 us for
// one sequence with 16 heads, the latency of two kernels; 18.6 us for 16 sequences with 8 heads.  12
// sequences, 5 tokens, D = 256, window 1024: 31 us; a part is only ten chunks there, and its partial
// results, written and read, add 40 % to the cache's bytes.  With sinks: 64 ragged sequences, 4 tokens, 32 /
// 8 heads, window 4096, 68 sinks, accumulating: 151 us, the walk 104 of it (5.4 TB/s with the scores that it
// writes), the join 9, the weights 39, of 16 rows a slot; 12 sequences, D = 256, window 1024, 4 sinks: 31.4 us,
// 6 of them before the first chunk is there, 6 the join.
#include <climits>
#include <type_traits>

#include "swa_cache_kernels.h"
#include "swa_cache_prefix.h"
#include "swa_cache_split.h"
#include "swa_ptx.cuh"
#include "swa_tmap.h"

namespace swa {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxSeqs = 1024;  // sequences per launch; more run as several launches
static_assert(kMaxSeqs <= kPrefixSeqs, "what the prefix's walk holds of each");

// kTiles: tiles of 16 query rows of a warp.
template <int D, int kTiles = 1>
struct AttnCfg {
  static constexpr int CK = D == 256 ? 16 : 32;          // keys of a chunk
  static constexpr int kCols = D < 128 ? D : 128;        // columns of a TMA box
  static constexpr int kBoxes = D / kCols;
  static constexpr int kBoxBytes = CK * kCols;
  static constexpr int kStageBytes = 2 * CK * D;         // keys, then values
  static constexpr int kStages = 192 * 1024 / kStageBytes;  // of the CTA, shared out to its teams
  // Q fragments of 16 x 256 or 32 x 128 elements are kept in shared memory (64 KB), in place of a third
  // of the stages.
  static constexpr bool kQShared = D * kTiles >= 256;
  static constexpr int kQBytes = kQShared ? kWarps * 16 * kTiles * D * 2 : 0;
  static constexpr int kRing = kStages - kQBytes / kStageBytes;
  static constexpr int kOffFirst = kRing * kStageBytes + kQBytes;
  static constexpr int kOffLen = kOffFirst + (kMaxSeqs + 2) * 8;  // lengths, then new tokens
  static constexpr int kOffBar = kOffLen + 2 * kMaxSeqs * 4;
  static constexpr int kOffSums = kOffBar + 2 * kStages * 8 + 16;  // + abort flag
  static constexpr int kSmemBytes = kOffSums + kWarps * 8;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");
};

struct AttnDev {
  const uint16_t* q;
  uint16_t* o;
  float* lse;
  int R;             // query rows per kv head: G T
  int MT, RT, NRT;   // warps of a team, rows of an item, items per kv head
  int rows;          // rows an item stores: min(RT, R)
  Reach reach;       // window, sinks, and the first slot of the walk
  int parts, f16, page_log2;
  int whole;         // 0, or where items that one team finished leave a partial result all the same
  FastDiv div_t, div_nrt, div_per;  // T, NRT, items of a sequence
  float scale_log2;
  int64_t* first;    // [B + 1] chunks before each sequence
  float* ml;         // [2 parts][rows][2] partial maxima and sums
  float* po;         // [2 parts][rows][D] partial outputs
  float* scores;     // [chunks][rows][CK], or null
};

template <int W>
__device__ __forceinline__ void lds_words(uint32_t a, uint32_t (&r)[W]) {
  if constexpr (W == 4)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
  else
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldmatrix_x4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x + __shfl_xor_sync(0xffffffffu, x, 2);
}
__device__ __forceinline__ uint32_t swizzle_of(int cols, uint32_t row) {
  return cols == 128 ? (row & 7u) : ((row >> 1) & 3u);
}

// What a lane holds about one chunk of its team's next 32.
struct ChunkInfo {
  int plane;  // page * Hkv + head, or -1: nothing to be seen there
  int slot;   // first slot
  int item;
  float ks, vs;
};

// The walk's state for one item.
template <int D, int kTiles>
struct ItemState {
  struct Tile {
    float acc[D / 8][4];  // o in units of vref; n-tile i of half x: columns 128 x + 16 n + i
    float m[2], l[2];     // rows g, g + 8: running maximum (base 2) and this lane's part of the sum
    float f[2];           // score factors of the two rows without the block's scale
    int lo[2], hi[2];     // slots the two rows see, inclusive
  } tile[kTiles];
  float vref;
  int sinks;            // slots below are seen whatever the window's first
  int any_lo, any_hi;   // slots any row sees
  int all_lo, all_hi;   // slots every real row sees
};

template <int D, int kTiles, bool kEdge>
__device__ __forceinline__ void process_chunk(ItemState<D, kTiles>& st, const uint32_t (*qf)[4],
                                              uint32_t sq, uint32_t sk, const ChunkInfo& ci,
                                              float* scores, int rows, int row0) {
  using C = AttnCfg<D, kTiles>;
  constexpr int CK = C::CK, kSteps = D / 16;
  const uint32_t lane = lane_id(), g = lane >> 2, t = lane & 3u;
  float s[kTiles][CK / 8][4];
#pragma unroll
  for (int y = 0; y < kTiles; ++y)
#pragma unroll
    for (int j = 0; j < CK / 8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[y][j][i] = 0.f;
#pragma unroll
  for (int x = 0; x < C::kBoxes; ++x) {
#pragma unroll
    for (int cq = 0; cq < C::kCols / 64; ++cq) {
      uint32_t key[CK / 8][4];  // codes of 8 keys, 4 steps of the contraction
#pragma unroll
      for (int j = 0; j < CK / 8; ++j) {
        const uint32_t row = 8 * j + (lane & 7u);
        const uint32_t unit = (4 * cq + (lane >> 3)) ^ swizzle_of(C::kCols, row);
        ldmatrix_x4(sk + x * C::kBoxBytes + row * C::kCols + (unit << 4), key[j]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int step = x * 8 + cq * 4 + i;
        uint32_t qa[kTiles][4];
#pragma unroll
        for (int y = 0; y < kTiles; ++y) {
          if constexpr (C::kQShared) {
            lds_words<4>(sq + ((y * kSteps + step) * 32 + lane) * 16, qa[y]);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) qa[y][e] = qf[y * kSteps + step][e];
          }
        }
#pragma unroll
        for (int j = 0; j < CK / 8; ++j) {
          uint32_t b0, b1;
          e4m3x4_to_f16(key[j][i], b0, b1);
#pragma unroll
          for (int y = 0; y < kTiles; ++y) mma16816(s[y][j], qa[y], b0, b1);
        }
      }
    }
  }
  // scores in base 2
  float mx[kTiles][2];
  bool moves = !(ci.vs >= st.vref && ci.vs <= 64.f * st.vref);
#pragma unroll
  for (int y = 0; y < kTiles; ++y) {
    auto& tl = st.tile[y];
    const float f0 = tl.f[0] * ci.ks, f1 = tl.f[1] * ci.ks;
    float mx0 = SWA_NEG_INF, mx1 = SWA_NEG_INF;
#pragma unroll
    for (int j = 0; j < CK / 8; ++j) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        s[y][j][i] *= f0;
        s[y][j][2 + i] *= f1;
        if (kEdge) {
          const int slot = ci.slot + 8 * j + 2 * static_cast<int>(t) + i;
          const bool sunk = slot < st.sinks;
          s[y][j][i] = (sunk || slot >= tl.lo[0]) && slot <= tl.hi[0] ? s[y][j][i] : SWA_NEG_INF;
          s[y][j][2 + i] =
              (sunk || slot >= tl.lo[1]) && slot <= tl.hi[1] ? s[y][j][2 + i] : SWA_NEG_INF;
        }
        mx0 = fmaxf(mx0, s[y][j][i]);
        mx1 = fmaxf(mx1, s[y][j][2 + i]);
      }
    }
    if (scores != nullptr) {
#pragma unroll
      for (int j = 0; j < CK / 8; ++j) {
        const int r0 = row0 + 16 * y + static_cast<int>(g);
        if (r0 < rows)
          *reinterpret_cast<float2*>(scores + r0 * CK + 8 * j + 2 * t) =
              make_float2(s[y][j][0], s[y][j][1]);
        if (r0 + 8 < rows)
          *reinterpret_cast<float2*>(scores + (r0 + 8) * CK + 8 * j + 2 * t) =
              make_float2(s[y][j][2], s[y][j][3]);
      }
    }
    mx[y][0] = quad_max(mx0);
    mx[y][1] = quad_max(mx1);
    moves = moves || mx[y][0] > tl.m[0] + 4.f || mx[y][1] > tl.m[1] + 4.f;
  }
  // The maximum and the value reference move only when a probability could reach 2^4, or a scale
  // leaves [vref, 64 vref]: p vs / vref then stays within fp16 and above its subnormals as far as
  // p itself is.
  if (__any_sync(0xffffffffu, moves)) {
    const float nref = ci.vs >= st.vref && ci.vs <= 64.f * st.vref ? st.vref : ci.vs * 0.125f;
    const float u = nref == st.vref ? 1.f : st.vref / nref;
#pragma unroll
    for (int y = 0; y < kTiles; ++y) {
      auto& tl = st.tile[y];
      const float n0 = fmaxf(tl.m[0], mx[y][0]), n1 = fmaxf(tl.m[1], mx[y][1]);
      const float a0 = tl.m[0] == SWA_NEG_INF ? 0.f : ex2(tl.m[0] - n0);
      const float a1 = tl.m[1] == SWA_NEG_INF ? 0.f : ex2(tl.m[1] - n1);
      // A sum that is NaN stays so (0 * NaN); before the first visible key everything is zero.
      tl.l[0] *= a0;
      tl.l[1] *= a1;
      const float w0 = a0 * u, w1 = a1 * u;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        tl.acc[i][0] *= w0;
        tl.acc[i][1] *= w0;
        tl.acc[i][2] *= w1;
        tl.acc[i][3] *= w1;
      }
      tl.m[0] = n0;
      tl.m[1] = n1;
    }
    st.vref = nref;
  }
  const float ratio = ci.vs / st.vref;
  uint32_t pa[kTiles][CK / 16][4];
#pragma unroll
  for (int y = 0; y < kTiles; ++y) {
    auto& tl = st.tile[y];
    const float b0 = tl.m[0] == SWA_NEG_INF ? 0.f : tl.m[0];
    const float b1 = tl.m[1] == SWA_NEG_INF ? 0.f : tl.m[1];
#pragma unroll
    for (int j = 0; j < CK / 8; ++j) {
      float p[4];
      p[0] = ex2(s[y][j][0] - b0);
      p[1] = ex2(s[y][j][1] - b0);
      p[2] = ex2(s[y][j][2] - b1);
      p[3] = ex2(s[y][j][3] - b1);
      tl.l[0] += p[0] + p[1];
      tl.l[1] += p[2] + p[3];
      pa[y][j / 2][2 * (j & 1)] = pack_f16(p[0] * ratio, p[1] * ratio);
      pa[y][j / 2][2 * (j & 1) + 1] = pack_f16(p[2] * ratio, p[3] * ratio);
    }
  }
  // o += P V
  const uint32_t sv = sk + CK * D;
  constexpr int W = C::kCols / 32;  // words a lane reads of a row: 16 or 8 columns
#pragma unroll
  for (int i = 0; i < CK / 16; ++i) {
#pragma unroll
    for (int x = 0; x < C::kBoxes; ++x) {
      uint32_t v[4][W];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t row = 16 * i + 2 * t + (e & 1) + 8 * (e >> 1);
        uint32_t at;
        if constexpr (W == 4)
          at = row * 128u + ((g ^ (row & 7u)) << 4);
        else
          at = row * 64u + (((g >> 1) ^ ((row >> 1) & 3u)) << 4) + ((g & 1u) << 3);
        lds_words<W>(sv + x * C::kBoxBytes + at, v[e]);
        if (kEdge) {
          const int slot = ci.slot + static_cast<int>(row);
          if ((slot < st.any_lo && slot >= st.sinks) || slot > st.any_hi) {
#pragma unroll
            for (int w = 0; w < W; ++w) v[e][w] = 0u;
          }
        }
      }
#pragma unroll
      for (int w = 0; w < W; ++w) {
        uint32_t a0, a1, a2, a3, c0, c1, c2, c3;
        e4m3x4_to_f16(__byte_perm(v[0][w], v[1][w], 0x5140), a0, a1);
        e4m3x4_to_f16(__byte_perm(v[0][w], v[1][w], 0x7362), a2, a3);
        e4m3x4_to_f16(__byte_perm(v[2][w], v[3][w], 0x5140), c0, c1);
        e4m3x4_to_f16(__byte_perm(v[2][w], v[3][w], 0x7362), c2, c3);
        const int tile = x * (D > 128 ? 16 : 0) + 4 * w;
#pragma unroll
        for (int y = 0; y < kTiles; ++y) {
          mma16816(st.tile[y].acc[tile], pa[y][i], a0, c0);
          mma16816(st.tile[y].acc[tile + 1], pa[y][i], a1, c1);
          mma16816(st.tile[y].acc[tile + 2], pa[y][i], a2, c2);
          mma16816(st.tile[y].acc[tile + 3], pa[y][i], a3, c3);
        }
      }
    }
  }
}

template <int D, int kTiles>
__global__ void __launch_bounds__(kThreads, 1)
    swa_cache_attn_kernel(const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v, const CacheView c,
                          const AttnDev a) {
  using C = AttnCfg<D, kTiles>;
  constexpr int CK = C::CK;
  extern __shared__ __align__(1024) uint8_t smem[];
  wait_predecessor();  // from here on whoever follows may take all inputs to be there
  launch_dependents();
  if (!smem_base_ok(smem, c.err)) return;
  int64_t* s_first = reinterpret_cast<int64_t*>(smem + C::kOffFirst);
  int* s_len = reinterpret_cast<int*>(smem + C::kOffLen);
  int* s_new = s_len + kMaxSeqs;  // 0 for a sequence that does not fit its table
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  int& abort_flag = *reinterpret_cast<int*>(bars + 2 * C::kStages);
  const int tid = static_cast<int>(threadIdx.x);
  const int warp = static_cast<int>(warp_id()), lane = static_cast<int>(lane_id());
  const int teams = kWarps / a.MT, team = warp / a.MT, wt = warp % a.MT;
  const int NS = C::kRing / teams;  // stages of a team's ring
  auto full = [&](int s) { return smem_u32(&bars[team * NS + s]); };
  auto empty = [&](int s) { return smem_u32(&bars[C::kStages + team * NS + s]); };
  if (warp == kWarps - 1) {
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
      abort_flag = 0;
    }
    for (int i = lane; i < C::kRing; i += 32) {
      mbar_init(smem_u32(&bars[i]), 1);
      mbar_init(smem_u32(&bars[C::kStages + i]), static_cast<uint32_t>(a.MT));
    }
    fence_barrier_init();
  }
  // Chunks before each sequence: a run of sequences a thread, an inclusive scan over the warps.  Loops stay
  // rolled, here and below: what runs once takes its time by the instructions that have to be fetched.
  {
    int64_t* s_sum = reinterpret_cast<int64_t*>(smem + C::kOffSums);
    const int each = c.B / kThreads + 1, b0 = min(tid * each, c.B + 1), b1 = min(b0 + each, c.B + 1);
    int64_t sum = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      int n = 0, len = 0;
      if (b < c.B) {
        if (!sequence_of(c, b, &len, &n)) n = 0;
        s_len[b] = len;
        s_new[b] = n;
      }
      s_first[b] = sum;
      sum += ChunkWalk(len, n, a.reach, CK).count;
    }
    int64_t scan = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, scan, d);
      if (lane >= d) scan += up;
    }
    if (lane == 31) s_sum[warp] = scan;
    __syncthreads();
    int64_t base = scan - sum;
#pragma unroll 1
    for (int w = 0; w < warp; ++w) base += s_sum[w];
#pragma unroll 1
    for (int b = b0; b < b1; ++b) s_first[b] += base;
    __syncthreads();
    if (blockIdx.x == 0)
      for (int b = tid; b <= c.B; b += kThreads) a.first[b] = s_first[b];
  }
  const int per = c.Hkv * a.NRT;  // items of a sequence
  const int64_t total = s_first[c.B] * per;
  // Neighbouring parts go to different SMs: with few chunks every SM still gets some.
  const int part = team * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x);
  const Parts cut(total, used_parts(total, a.parts, a.rows * D));
  const int64_t begin = part < cut.parts ? cut.start(part) : total;
  const int64_t count = part < cut.parts ? cut.start(part + 1) - begin : 0;

  auto load_info = [&](int64_t i) {  // chunk i of the part
    ChunkInfo ci = {-1, 0, -1, 1.f, 1.f};
    if (i < count) {
      const int64_t x = begin + i;
      const int b = sequence_at(s_first, c.B, per, x);
      const int nc = static_cast<int>(s_first[b + 1] - s_first[b]);
      const int64_t rem = x - s_first[b] * per;
      const int hr = static_cast<int>(quotient(rem, nc));
      ci.item = b * per + hr;
      ci.slot = ChunkWalk(s_len[b], 1, a.reach, CK)
                    .at(static_cast<int>(rem - static_cast<int64_t>(hr) * nc)) * CK;
      const int page = page_of(c, c.table, b, ci.slot >> a.page_log2, c.max_pages);
      if (page >= 0) {
        ci.plane = page * c.Hkv + static_cast<int>(a.div_nrt.div(static_cast<uint32_t>(hr)));
        ci.ks = c.k_scale[ci.plane];
        ci.vs = c.v_scale[ci.plane];
      }
    }
    return ci;
  };
  // Scores are read back by the weights kernel; keys and values that are read once make room for them
  // in the L2 (64 ragged sequences to 16K, accumulating: 203 us, 207 without).
  uint64_t policy;
  if (a.scores != nullptr && a.NRT == 1)
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  else
    asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
  ChunkInfo cur = load_info(lane), nxt = load_info(32 + lane);
  const uint32_t ring = smem_u32(smem) + static_cast<uint32_t>(team * NS) * C::kStageBytes;
  int64_t issued = 0;
  auto issue = [&](int64_t i, int s, bool in_next) {  // whole warp; chunk i into stage s = i % NS
    const int plane = __shfl_sync(0xffffffffu, in_next ? nxt.plane : cur.plane, static_cast<int>(i & 31));
    const int slot = __shfl_sync(0xffffffffu, in_next ? nxt.slot : cur.slot, static_cast<int>(i & 31));
    if (wt == 0 && lane == 0) {
      const uint32_t dst = ring + static_cast<uint32_t>(s) * C::kStageBytes;
      mbar_arrive_expect_tx(full(s), C::kStageBytes);
      // A chunk whose page is out of range loads plane 0 and is masked.
#pragma unroll
      for (int x = 0; x < C::kBoxes; ++x) {
        tma_load_3d(dst + x * C::kBoxBytes, &tm_k, full(s), 128 * x, slot & (c.page - 1),
                    max(plane, 0), policy);
        tma_load_3d(dst + CK * D + x * C::kBoxBytes, &tm_v, full(s), 128 * x,
                    slot & (c.page - 1), max(plane, 0), policy);
      }
    }
    issued = i + 1;
  };
  for (int i = 0; i < NS && i < count; ++i) issue(i, i, i >= 32);

  const uint32_t sq = smem_u32(smem + C::kRing * C::kStageBytes) +
                      static_cast<uint32_t>(warp) * 16 * kTiles * D * 2;
  constexpr int kSteps = D / 16;
  uint32_t qf[C::kQShared ? 1 : kTiles * kSteps][4];
  ItemState<D, kTiles> st = {};
  int item = -1, b = 0, tile0 = 0, item_last = 0;
  size_t base = 0;  // first row of the item, of all rows
  bool begins = false;
  const int g = lane >> 2, t = lane & 3;
  const int r0 = wt * 16 * kTiles + g;  // this thread's rows of the item: r0, r0 + 8, r0 + 16, ..

  // Finishes the item after its chunk at `slot`.
  auto finish = [&](int slot) {
    const bool ends = slot / CK == item_last;
#pragma unroll
    for (int ye = 0; ye < 2 * kTiles; ++ye) {
      const int e = ye & 1, r = r0 + 8 * ye;
      const auto& tl = st.tile[ye >> 1];
      const float l = quad_sum(tl.l[e]);
      if (tile0 + r >= a.R) continue;
      if (begins && ends && a.whole == 0) {
        const float inv = l == 0.f ? 0.f : st.vref / l;
        uint16_t* out = a.o + (base + r) * D;
#pragma unroll
        for (int x = 0; x < (D > 128 ? 2 : 1); ++x) {
          constexpr int kRun = D < 128 ? 8 : 16;  // = columns of a run
#pragma unroll
          for (int run = 0; run < 2; ++run) {
            uint32_t pk[kRun / 2];
#pragma unroll
            for (int i = 0; i < kRun / 2; ++i) {
              const float y0 = tl.acc[x * 16 + 2 * i][2 * e + run] * inv;
              const float y1 = tl.acc[x * 16 + 2 * i + 1][2 * e + run] * inv;
              pk[i] = a.f16 ? Elem<true>::pack(y0, y1) : Elem<false>::pack(y0, y1);
            }
            uint4* dst = reinterpret_cast<uint4*>(out + 128 * x + kRun * (2 * t + run));
#pragma unroll
            for (int i = 0; i < kRun / 8; ++i)
              dst[i] = make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
          }
        }
        if (t == 0) a.lse[base + r] = l == 0.f ? SWA_NEG_INF : (tl.m[e] + log2f(l)) * kLn2;
      } else {
        const int at = begins && ends ? a.whole + item : partial_slot(part, begins);
        const size_t slot_row = static_cast<size_t>(at) * a.rows + r;
        float* out = a.po + slot_row * D;
#pragma unroll
        for (int x = 0; x < (D > 128 ? 2 : 1); ++x) {
          constexpr int kRun = D < 128 ? 8 : 16;
#pragma unroll
          for (int run = 0; run < 2; ++run) {
            float4* dst = reinterpret_cast<float4*>(out + 128 * x + kRun * (2 * t + run));
#pragma unroll
            for (int i = 0; i < kRun / 4; ++i)
              dst[i] = make_float4(tl.acc[x * 16 + 4 * i][2 * e + run] * st.vref,
                                   tl.acc[x * 16 + 4 * i + 1][2 * e + run] * st.vref,
                                   tl.acc[x * 16 + 4 * i + 2][2 * e + run] * st.vref,
                                   tl.acc[x * 16 + 4 * i + 3][2 * e + run] * st.vref);
          }
        }
        if (t == 0) {
          a.ml[slot_row * 2] = tl.m[e];
          a.ml[slot_row * 2 + 1] = l;
        }
      }
    }
  };

  auto start = [&](int new_item, int slot) {
    item = new_item;
    b = static_cast<int>(a.div_per.div(static_cast<uint32_t>(item)));
    const uint32_t hr = static_cast<uint32_t>(item - b * per), h = a.div_nrt.div(hr);
    tile0 = static_cast<int>(hr - h * a.div_nrt.d) * a.RT;
    const int len = s_len[b], n = s_new[b];
    base = (static_cast<size_t>(b) * c.Hkv + h) * a.R + tile0;
    // Both rows of q are on their way before anything waits for them.
    uint2 raw[2 * kTiles][kSteps];
#pragma unroll
    for (int e = 0; e < 2 * kTiles; ++e) {
      const uint32_t r = static_cast<uint32_t>(tile0 + r0 + 8 * e);
      const int tq = static_cast<int>(a.div_t.mod(r));
      const bool real = static_cast<int>(r) < a.R && tq < n;
      const uint2* row = reinterpret_cast<const uint2*>(a.q + (base + r0 + 8 * e) * D) + t;
#pragma unroll
      for (int i = 0; i < kSteps; ++i) raw[e][i] = real ? __ldg(row + 4 * i) : make_uint2(0u, 0u);
      auto& tl = st.tile[e >> 1];
      tl.lo[e & 1] = visible_lo(len + tq, a.reach.window);
      tl.hi[e & 1] = real ? len + tq : -1;
      tl.m[e & 1] = SWA_NEG_INF;
      tl.l[e & 1] = 0.f;
    }
    const ChunkWalk walk(len, n, a.reach, CK);
    item_last = walk.last();
    begins = slot / CK == walk.at(0);
    st.sinks = a.reach.sinks;
    st.any_lo = visible_lo(len, a.reach.window);
    st.any_hi = len + n - 1;
    st.all_lo = visible_lo(len + n - 1, a.reach.window);
    st.all_hi = n < c.T ? -1 : len;  // a row without a query sees nothing
    float up[2 * kTiles];
#pragma unroll
    for (int ye = 0; ye < 2 * kTiles; ++ye) {
      const int y = ye >> 1, e = ye & 1;
      // The row as fp16, its largest element brought to [2^14, 2^15) (a row below 2^-112 less far).  The
      // largest magnitude is that of the bits, two elements a word.
      uint32_t most = 0;
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
        most = __vmaxu2(most, __vmaxu2(raw[ye][i].x & 0x7fff7fffu, raw[ye][i].y & 0x7fff7fffu));
      most = max(most & 0xffffu, most >> 16);
      most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
      most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
      const uint32_t top =
          __float_as_uint(a.f16 ? Elem<true>::unpack(most).x : Elem<false>::unpack(most).x);
      const int ex = static_cast<int>(top >> 23);
      // 2^(14 - exponent); 1 for zero, infinity and NaN
      const int sh = ex == 255 || top == 0 ? 0 : min(126, 127 + 14 - ex);
      up[ye] = __uint_as_float(static_cast<uint32_t>(127 + sh) << 23);
      // Scores of an infinite query are infinite, and exp(x - lse) of them NaN: all NaN from here on, since
      // a row whose scores were all -inf would look like one that sees nothing.
      st.tile[y].f[e] = ex == 255 ? __uint_as_float(0x7fffffffu)
                                  : a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - sh) << 23);
    }
    auto scaled = [&](uint32_t w, float by) {
      const float2 v = a.f16 ? Elem<true>::unpack(w) : Elem<false>::unpack(w);
      return pack_f16(v.x * by, v.y * by);
    };
    if constexpr (C::kQShared) {
      // Into shared memory as they are, and scaled there by a loop: what runs once takes as long as its
      // instructions take to be fetched.
#pragma unroll
      for (int y = 0; y < kTiles; ++y) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
          st_shared_v4(sq + ((y * kSteps + i) * 32 + lane) * 16, raw[2 * y][i].x, raw[2 * y + 1][i].x,
                       raw[2 * y][i].y, raw[2 * y + 1][i].y);
#pragma unroll 1
        for (int i = 0; i < kSteps; ++i) {
          const uint32_t at = sq + ((y * kSteps + i) * 32 + lane) * 16;
          uint32_t w[4];
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                       : "r"(at)
                       : "memory");
          st_shared_v4(at, scaled(w[0], up[2 * y]), scaled(w[1], up[2 * y + 1]), scaled(w[2], up[2 * y]),
                       scaled(w[3], up[2 * y + 1]));
        }
      }
    } else {
#pragma unroll
      for (int y = 0; y < kTiles; ++y)
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            qf[y * kSteps + i][e] = scaled(raw[2 * y + e][i].x, up[2 * y + e]);
            qf[y * kSteps + i][2 + e] = scaled(raw[2 * y + e][i].y, up[2 * y + e]);
          }
    }
    st.vref = 1.f;
#pragma unroll
    for (int y = 0; y < kTiles; ++y)
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) st.tile[y].acc[i][e] = 0.f;
    __syncwarp();
  };

  int last_slot = 0, s = 0;
  uint32_t phase = 0;
  int64_t done = 0;
  bool ok = true;
  for (int64_t i = 0; i < count; ++i) {
    if (i > 0 && (i & 31) == 0) {
      cur = nxt;
      nxt = load_info(i + 32 + lane);
    }
    const int from = static_cast<int>(i & 31);
    ChunkInfo ci;
    ci.plane = __shfl_sync(0xffffffffu, cur.plane, from);
    ci.slot = __shfl_sync(0xffffffffu, cur.slot, from);
    ci.item = __shfl_sync(0xffffffffu, cur.item, from);
    ci.ks = __shfl_sync(0xffffffffu, cur.ks, from);
    ci.vs = __shfl_sync(0xffffffffu, cur.vs, from);
    if (ci.item != item) {
      if (item >= 0) finish(last_slot);
      start(ci.item, ci.slot);
    }
    last_slot = ci.slot;
    if (!(ok = warp_wait(full(s), phase, &abort_flag, c.err))) break;
    const uint32_t sk = ring + static_cast<uint32_t>(s) * C::kStageBytes;
    float* sc = a.scores == nullptr ? nullptr
                                    : a.scores + static_cast<size_t>(begin + i) * a.rows * CK;
    const bool edge = ci.plane < 0 || (ci.slot < st.all_lo && ci.slot + CK > st.sinks) ||
                      ci.slot + CK - 1 > st.all_hi;
    if (edge) {
      ItemState<D, kTiles>& e = st;
      int lo[2 * kTiles];
      const int any = e.any_lo;
#pragma unroll
      for (int y = 0; y < 2 * kTiles; ++y) {
        lo[y] = e.tile[y >> 1].lo[y & 1];
        if (ci.plane < 0) e.tile[y >> 1].lo[y & 1] = INT_MAX;  // nothing of it is seen
      }
      if (ci.plane < 0) {
        e.any_lo = INT_MAX;
        e.sinks = 0;
      }
      process_chunk<D, kTiles, true>(e, qf, sq, sk, ci, sc, a.rows, wt * 16 * kTiles);
#pragma unroll
      for (int y = 0; y < 2 * kTiles; ++y) e.tile[y >> 1].lo[y & 1] = lo[y];
      e.any_lo = any;
      e.sinks = a.reach.sinks;
    } else {
      process_chunk<D, kTiles, false>(st, qf, sq, sk, ci, sc, a.rows, wt * 16 * kTiles);
    }
    __syncwarp();
    done = i + 1;
    if (a.MT > 1 && lane == 0) mbar_arrive(empty(s));
    const int64_t ahead = i + NS;
    if (ahead < count) {
      if (a.MT > 1 && wt == 0 &&
          !(ok = warp_wait(empty(s), phase, &abort_flag, c.err)))
        break;
      issue(ahead, s, (ahead >> 5) != (i >> 5));
    }
    if (++s == NS) {
      s = 0;
      phase ^= 1u;
    }
  }
  if (ok) {
    if (item >= 0) finish(last_slot);
  } else if (wt == 0) {  // a wait ran out: this team's copies in flight land before the CTA ends
    for (int64_t i = done; i < issued; ++i)
      warp_drain_wait(full(static_cast<int>(i % NS)), static_cast<uint32_t>(i / NS) & 1u, c.err);
  }
}

// Where an item's partial results are: parts p0 .. p1 of the list, the item's first chunk x0.  Both
// equal: the item was finished by one team.  No chunks: nobody saw anything.
struct ItemParts {
  int64_t x0, chunks;
  int p0, p1;
};
__device__ __forceinline__ ItemParts item_parts(const AttnDev& a, const Parts& cut, int per, int item) {
  const int b = static_cast<int>(a.div_per.div(static_cast<uint32_t>(item)));
  const int64_t f0 = a.first[b];
  ItemParts ip;
  ip.chunks = a.first[b + 1] - f0;
  ip.x0 = f0 * per + (item - b * per) * ip.chunks;
  ip.p0 = ip.p1 = 0;
  if (ip.chunks > 0) {
    ip.p0 = cut.of(ip.x0);
    ip.p1 = cut.of(ip.x0 + ip.chunks - 1);
  }
  return ip;
}

// Row `r` of an item, of all rows of the call; false when the last tile of a kv head is shorter.
__device__ __forceinline__ bool row_of_item(const AttnDev& a, int item, int r, size_t* row) {
  const uint32_t bh = a.div_nrt.div(static_cast<uint32_t>(item));
  const int in_head = (item - static_cast<int>(bh * a.div_nrt.d)) * a.RT + r;
  *row = static_cast<size_t>(bh) * a.R + in_head;
  return in_head < a.R;
}

template <int N>
__device__ __forceinline__ void store_row(const AttnDev& a, uint16_t* out, const float (&o)[N],
                                          float scale) {
  uint32_t pk[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i)
    pk[i] = a.f16 ? Elem<true>::pack(o[2 * i] * scale, o[2 * i + 1] * scale)
                  : Elem<false>::pack(o[2 * i] * scale, o[2 * i + 1] * scale);
  if constexpr (N == 8)
    *reinterpret_cast<uint4*>(out) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
  else if constexpr (N == 4)
    *reinterpret_cast<uint2*>(out) = make_uint2(pk[0], pk[1]);
  else
    *reinterpret_cast<uint32_t*>(out) = pk[0];
}

// Joins the partial results of items that several teams shared, and answers the rows of sequences
// without a chunk: a warp a row, its lanes the row's columns.
template <int D>
__global__ void __launch_bounds__(256) swa_cache_join_kernel(const CacheView c, const AttnDev a) {
  constexpr int N = D / 32;
  wait_predecessor();
  launch_dependents();
  const int lane = static_cast<int>(lane_id());
  const int per = c.Hkv * a.NRT;
  const int64_t total = a.first[c.B] * per;
  const Parts cut(total, used_parts(total, a.parts, a.rows * D));
  const uint32_t tasks = static_cast<uint32_t>(c.B) * per * a.rows;
  for (uint32_t task = blockIdx.x * 8 + warp_id(); task < tasks; task += gridDim.x * 8) {
    const int item = static_cast<int>(task / static_cast<uint32_t>(a.rows));
    const int r = static_cast<int>(task - static_cast<uint32_t>(item) * a.rows);
    size_t row;
    if (!row_of_item(a, item, r, &row)) continue;
    const ItemParts ip = item_parts(a, cut, per, item);
    if (ip.chunks > 0 && ip.p0 == ip.p1) continue;
    float o[N] = {}, l = 0.f, top = SWA_NEG_INF;
    if (ip.chunks > 0) {
      auto partial = [&](int p) {
        return static_cast<size_t>(partial_slot(p, cut.start(p) <= ip.x0)) * a.rows + r;
      };
      for (int p = ip.p0 + lane; p <= ip.p1; p += 32) top = fmaxf(top, a.ml[partial(p) * 2]);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      const float base = top == SWA_NEG_INF ? 0.f : top;
      for (int p = ip.p0; p <= ip.p1; p += 32) {
        const int n = min(32, ip.p1 - p + 1);
        float w = 0.f;
        if (lane < n) {
          const float2 ml = *reinterpret_cast<const float2*>(a.ml + partial(p + lane) * 2);
          w = ex2(ml.x - base);
          l += w * ml.y;
        }
#pragma unroll 4
        for (int j = 0; j < n; ++j) {
          const float wj = __shfl_sync(0xffffffffu, w, j);
          const float* y = a.po + partial(p + j) * D + lane * N;
          float v[N];
          if constexpr (N == 2) {
            const float2 u = *reinterpret_cast<const float2*>(y);
            v[0] = u.x, v[1] = u.y;
          } else {
#pragma unroll
            for (int i = 0; i < N; i += 4) {
              const float4 u = *reinterpret_cast<const float4*>(y + i);
              v[i] = u.x, v[i + 1] = u.y, v[i + 2] = u.z, v[i + 3] = u.w;
            }
          }
#pragma unroll
          for (int i = 0; i < N; ++i) o[i] += wj * v[i];
        }
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    }
    store_row<N>(a, a.o + row * D + lane * N, o, l == 0.f ? 0.f : 1.f / l);
    if (lane == 0) a.lse[row] = l == 0.f ? SWA_NEG_INF : (top + log2f(l)) * kLn2;
  }
}

// The same with a warp for 16 columns of a row: 8 groups of 4 lanes take the partials in turn.
template <int D>
__global__ void __launch_bounds__(256) swa_cache_join_part_kernel(const CacheView c, const AttnDev a) {
  constexpr uint32_t kRuns = D / 16;
  wait_predecessor();
  launch_dependents();
  const int lane = static_cast<int>(lane_id()), group = lane / 4, sub = lane % 4;
  const int per = c.Hkv * a.NRT;
  const int64_t total = a.first[c.B] * per;
  const Parts cut(total, used_parts(total, a.parts, a.rows * D));
  const uint32_t tasks = static_cast<uint32_t>(c.B) * per * a.rows * kRuns;
  for (uint32_t task = blockIdx.x * 8 + warp_id(); task < tasks; task += gridDim.x * 8) {
    const int run = static_cast<int>(task % kRuns);
    const int item = static_cast<int>(task / kRuns / static_cast<uint32_t>(a.rows));
    const int r = static_cast<int>(task / kRuns - static_cast<uint32_t>(item) * a.rows);
    size_t row;
    if (!row_of_item(a, item, r, &row)) continue;
    const ItemParts ip = item_parts(a, cut, per, item);
    if (ip.chunks > 0 && ip.p0 == ip.p1) continue;
    float top = SWA_NEG_INF, l = 0.f;
    float o[4] = {};
    if (ip.chunks > 0) {
      auto partial = [&](int p) {
        return static_cast<size_t>(partial_slot(p, cut.start(p) <= ip.x0)) * a.rows + r;
      };
      // The first partial of each group is on its way while the maximum is found.
      const bool any = ip.p0 + group <= ip.p1;
      float2 ml0 = make_float2(0.f, 0.f);
      float4 y0 = make_float4(0.f, 0.f, 0.f, 0.f);
      if (any) {
        const size_t pr = partial(ip.p0 + group);
        ml0 = *reinterpret_cast<const float2*>(a.ml + pr * 2);
        y0 = *reinterpret_cast<const float4*>(a.po + pr * D + run * 16 + sub * 4);
      }
      for (int p = ip.p0 + lane; p <= ip.p1; p += 32) top = fmaxf(top, a.ml[partial(p) * 2]);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      const float base = top == SWA_NEG_INF ? 0.f : top;
      auto add = [&](float2 ml, float4 y) {
        const float w = ex2(ml.x - base);
        l += w * ml.y;
        o[0] += w * y.x;
        o[1] += w * y.y;
        o[2] += w * y.z;
        o[3] += w * y.w;
      };
      if (any) add(ml0, y0);
#pragma unroll 4
      for (int p = ip.p0 + group + 8; p <= ip.p1; p += 8) {
        const size_t pr = partial(p);
        add(*reinterpret_cast<const float2*>(a.ml + pr * 2),
            *reinterpret_cast<const float4*>(a.po + pr * D + run * 16 + sub * 4));
      }
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) {
        l += __shfl_xor_sync(0xffffffffu, l, d);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] += __shfl_xor_sync(0xffffffffu, o[i], d);
      }
    }
    if (group == 0) {
      store_row<4>(a, a.o + row * D + run * 16 + sub * 4, o, l == 0.f ? 0.f : 1.f / l);
      if (lane == 0 && run == 0) a.lse[row] = l == 0.f ? SWA_NEG_INF : (top + log2f(l)) * kLn2;
    }
  }
}

// The same with a block for 16 columns of a row, for calls with so few rows that each has very many
// partials: 64 groups of 4 lanes take the partials in turn and meet in shared memory in a fixed order.
template <int D>
__global__ void __launch_bounds__(256) swa_cache_join_few_kernel(const CacheView c, const AttnDev a) {
  constexpr int kGroups = 64, kRuns = D / 16;
  __shared__ float s_red[8], s_l[kGroups];
  __shared__ float4 s_o[256];
  wait_predecessor();
  launch_dependents();
  const int tid = static_cast<int>(threadIdx.x), group = tid / 4, sub = tid % 4;
  const int per = c.Hkv * a.NRT;
  const int64_t total = a.first[c.B] * per;
  const Parts cut(total, used_parts(total, a.parts, a.rows * D));
  const uint32_t tasks = static_cast<uint32_t>(c.B) * per * a.rows * kRuns;
  for (uint32_t task = blockIdx.x; task < tasks; task += gridDim.x) {
    const int run = static_cast<int>(task % kRuns);
    const int item = static_cast<int>(task / kRuns / static_cast<uint32_t>(a.rows));
    const int r = static_cast<int>(task / kRuns - static_cast<uint32_t>(item) * a.rows);
    size_t row;
    if (!row_of_item(a, item, r, &row)) continue;
    const ItemParts ip = item_parts(a, cut, per, item);
    if (ip.chunks > 0 && ip.p0 == ip.p1) continue;
    float top = SWA_NEG_INF, l = 0.f;
    float o[4] = {};
    if (ip.chunks > 0) {
      auto partial = [&](int p) {
        return static_cast<size_t>(partial_slot(p, cut.start(p) <= ip.x0)) * a.rows + r;
      };
      // The first partial of each group is on its way while the maximum is found.
      const bool any = ip.p0 + group <= ip.p1;
      float2 ml0 = make_float2(0.f, 0.f);
      float4 y0 = make_float4(0.f, 0.f, 0.f, 0.f);
      if (any) {
        const size_t pr = partial(ip.p0 + group);
        ml0 = *reinterpret_cast<const float2*>(a.ml + pr * 2);
        y0 = *reinterpret_cast<const float4*>(a.po + pr * D + run * 16 + sub * 4);
      }
      for (int p = ip.p0 + tid; p <= ip.p1; p += 256) top = fmaxf(top, a.ml[partial(p) * 2]);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      if ((tid & 31) == 0) s_red[tid >> 5] = top;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < 8; ++w) top = fmaxf(top, s_red[w]);
      const float base = top == SWA_NEG_INF ? 0.f : top;
      auto add = [&](float2 ml, float4 y) {
        const float w = ex2(ml.x - base);
        l += w * ml.y;
        o[0] += w * y.x;
        o[1] += w * y.y;
        o[2] += w * y.z;
        o[3] += w * y.w;
      };
      if (any) add(ml0, y0);
#pragma unroll 4
      for (int p = ip.p0 + group + kGroups; p <= ip.p1; p += kGroups) {
        const size_t pr = partial(p);
        add(*reinterpret_cast<const float2*>(a.ml + pr * 2),
            *reinterpret_cast<const float4*>(a.po + pr * D + run * 16 + sub * 4));
      }
      if (sub == 0) s_l[group] = l;
      s_o[tid] = make_float4(o[0], o[1], o[2], o[3]);
      __syncthreads();
      if (group == 0) {
        l = o[0] = o[1] = o[2] = o[3] = 0.f;
#pragma unroll 8
        for (int i = 0; i < kGroups; ++i) {
          l += s_l[i];
          const float4 y = s_o[i * 4 + sub];
          o[0] += y.x;
          o[1] += y.y;
          o[2] += y.z;
          o[3] += y.w;
        }
      }
      __syncthreads();  // before the next task's sums
    }
    if (group == 0) {
      store_row<4>(a, a.o + row * D + run * 16 + sub * 4, o, l == 0.f ? 0.f : 1.f / l);
      if (tid == 0 && run == 0) a.lse[row] = l == 0.f ? SWA_NEG_INF : (top + log2f(l)) * kLn2;
    }
  }
}

// With a shared prefix: joins what the parts of the prefix's items and the parts of a sequence's own slots
// left for a row.  A warp for kCols columns of a row: a lane looks up a partial's place, then groups of
// lanes, 4 or 8 columns each, take the partials in turn.
template <int D, int kCols>
__global__ void __launch_bounds__(256)
    swa_cache_join_shared_kernel(const CacheView c, const AttnDev a, const PrefixDev p) {
  constexpr uint32_t kRuns = D / kCols;
  constexpr int kVec = kCols < 64 ? 4 : 8, kSub = kCols / kVec, kGroups = 32 / kSub;
  wait_predecessor();
  launch_dependents();
  const int lane = static_cast<int>(lane_id()), group = lane / kSub, sub = lane % kSub;
  const int per = c.Hkv * a.NRT;
  const int64_t total = a.first[c.B] * per, ptotal = p.first[p.tiles] * c.Hkv;
  const Parts cut(total, used_parts(total, a.parts, a.rows * D));
  const Parts pcut(ptotal, prefix_parts(ptotal, p.parts, p.stored, D));
  const int64_t tasks = static_cast<int64_t>(c.B) * c.Hkv * a.R * kRuns;
  for (int64_t task = blockIdx.x * 8 + warp_id(); task < tasks; task += gridDim.x * 8) {
    const int run = static_cast<int>(task % kRuns);
    const uint32_t row = static_cast<uint32_t>(task / kRuns), bh = p.div_r.div(row),
                   b = p.div_hkv.div(bh);
    const int r = static_cast<int>(row - bh * p.div_r.d), h = static_cast<int>(bh - b * p.div_hkv.d);
    float top = SWA_NEG_INF, l = 0.f;
    float o[kVec] = {};
    int len, n;
    if (sequence_of(c, static_cast<int>(b), &len, &n) &&
        static_cast<int>(a.div_t.mod(static_cast<uint32_t>(r))) < n) {
      // the sequence's own slots
      const int rt = r / a.RT, item = static_cast<int>(bh) * a.NRT + rt;
      const ItemParts ip = item_parts(a, cut, per, item);
      const int own = ip.chunks > 0 ? ip.p1 - ip.p0 + 1 : 0;
      // the prefix
      const int rho = static_cast<int>(b) * a.R + r, j = rho / kPrefixRows;
      const int64_t f0 = p.first[j], chunks = p.first[j + 1] - f0;
      const int64_t x0 = f0 * c.Hkv + h * chunks;
      const int q0 = chunks > 0 ? pcut.of(x0) : 0;
      const int q1 = chunks > 0 ? pcut.of(x0 + chunks - 1) : -1;
      const int all = own + q1 - q0 + 1;
      for (int k0 = 0; k0 < all; k0 += 32) {  // partials in runs of 32, lane k the place of k0 + k
        const int k = k0 + lane;
        const float* y = nullptr;
        float2 s = make_float2(SWA_NEG_INF, 0.f);
        if (k < own) {
          const int part = ip.p0 + k;
          const int at = own == 1 ? a.whole + item : partial_slot(part, k == 0);
          const size_t to = static_cast<size_t>(at) * a.rows + (r - rt * a.RT);
          s = *reinterpret_cast<const float2*>(a.ml + to * 2);
          y = a.po + to * D;
        } else if (k < all) {
          const int part = q0 + k - own;
          const int at = q0 == q1 ? 2 * p.parts + j * c.Hkv + h : partial_slot(part, part == q0);
          const size_t to = static_cast<size_t>(at) * p.stored + (rho - j * kPrefixRows);
          s = *reinterpret_cast<const float2*>(p.ml + to * 2);
          y = p.po + to * D;
        }
        if (s.x == SWA_NEG_INF && s.y == 0.f) y = nullptr;  // the row saw nothing there
        float most = s.x;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
        if (most > top) {  // what came before was against a lower maximum
          const float down = ex2(top - most);
          l *= down;
#pragma unroll
          for (int i = 0; i < kVec; ++i) o[i] *= down;
          top = most;
        }
        const float w = y == nullptr ? 0.f : ex2(s.x - (top == SWA_NEG_INF ? 0.f : top));
        const float lw = y == nullptr ? 0.f : w * s.y;
        const int n = min(32, all - k0);
#pragma unroll 4
        for (int i = 0; i < n; i += kGroups) {
          const int from = i + group;
          const float* src = reinterpret_cast<const float*>(
              __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(y), from & 31));
          const float wk = __shfl_sync(0xffffffffu, w, from & 31);
          const float lk = __shfl_sync(0xffffffffu, lw, from & 31);
          if (from < n && src != nullptr) {
            float v[kVec];
#pragma unroll
            for (int x = 0; x < kVec; x += 4) {
              const float4 y4 = *reinterpret_cast<const float4*>(src + run * kCols + sub * kVec + x);
              v[x] = y4.x, v[x + 1] = y4.y, v[x + 2] = y4.z, v[x + 3] = y4.w;
            }
            l += lk;
#pragma unroll
            for (int x = 0; x < kVec; ++x) o[x] += wk * v[x];
          }
        }
        __syncwarp();
      }
#pragma unroll
      for (int d = kSub; d < 32; d <<= 1) {
        l += __shfl_xor_sync(0xffffffffu, l, d);
#pragma unroll
        for (int i = 0; i < kVec; ++i) o[i] += __shfl_xor_sync(0xffffffffu, o[i], d);
      }
    }
    if (group == 0) {
      store_row<kVec>(a, a.o + static_cast<size_t>(row) * D + run * kCols + sub * kVec, o,
                      l == 0.f ? 0.f : 1.f / l);
      if (lane == 0 && run == 0) a.lse[row] = l == 0.f ? SWA_NEG_INF : (top + log2f(l)) * kLn2;
    }
  }
}

// Adds to each cached token's weight the sum over its kv head's rows of 2^(score - lse / ln 2).  The
// lanes of a warp find the places of up to 32 chunks at once; then it takes 128 keys at a time, four a
// lane, and one thread alone touches a weight.
template <int D>
__global__ void __launch_bounds__(256) swa_cache_weights_kernel(const CacheView c, const AttnDev a) {
  using C = AttnCfg<D>;
  constexpr int CK = C::CK, kLanes = CK / 4, kChunks = 32 / kLanes;  // lanes of a chunk; at a time
  __shared__ int64_t s_first[kMaxSeqs + 1];
  wait_predecessor();
  launch_dependents();
  for (int b = static_cast<int>(threadIdx.x); b <= c.B; b += 256) s_first[b] = a.first[b];
  __syncthreads();
  const int lane = static_cast<int>(lane_id());
  const int64_t tasks = s_first[c.B] * c.Hkv;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * 8;
  // chunks of a turn: up to 32, fewer where that leaves warps without any
  int turn = kChunks;
  while (turn < 32 && tasks > warps * turn) turn *= 2;
  for (int64_t y0 = (static_cast<int64_t>(blockIdx.x) * 8 + warp_id()) * turn; y0 < tasks;
       y0 += warps * turn) {
    int64_t chunk = 0, weight = -1;
    int stride = 0, head = 0;
    if (lane < turn && y0 + lane < tasks) {
      const int64_t y = y0 + lane;
      const int b = sequence_at(s_first, c.B, c.Hkv, y);
      const int64_t f0 = s_first[b];
      stride = static_cast<int>(s_first[b + 1] - f0);
      const int64_t rem = y - f0 * c.Hkv;
      const int h = static_cast<int>(quotient(rem, stride));
      const int cc = static_cast<int>(rem - static_cast<int64_t>(h) * stride);
      const int slot = ChunkWalk(c.lens[b], 1, a.reach, CK).at(cc) * CK;
      const int page = page_of(c, c.table, b, slot >> a.page_log2, c.max_pages);
      if (page >= 0)
        weight = (static_cast<int64_t>(page) * c.Hkv + h) * c.page + (slot & (c.page - 1));
      chunk = f0 * c.Hkv * a.NRT + static_cast<int64_t>(h) * a.NRT * stride + cc;
      head = b * c.Hkv + h;
    }
    for (int g = 0; g < turn; g += kChunks) {
      const int from = g + lane / kLanes, key = lane % kLanes * 4;
      const int64_t at = __shfl_sync(0xffffffffu, weight, from);
      const int64_t x = __shfl_sync(0xffffffffu, chunk, from);
      const int nc = __shfl_sync(0xffffffffu, stride, from);
      const int bh = __shfl_sync(0xffffffffu, head, from);
      if (at < 0) continue;
      float4* w = reinterpret_cast<float4*>(c.weight + at + key);
      const float4 old = *w;
      float4 add = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int rt = 0; rt < a.NRT; ++rt) {
        const int rows = min(a.rows, a.R - rt * a.RT);
        const float* sc =
            a.scores + static_cast<size_t>(x + static_cast<int64_t>(rt) * nc) * a.rows * CK + key;
        const float* lse = a.lse + static_cast<size_t>(bh) * a.R + rt * a.RT;
#pragma unroll 4
        for (int r = 0; r < rows; ++r) {
          const float4 s = *reinterpret_cast<const float4*>(sc + r * CK);
          // a row that sees nothing has scores and lse -inf, and adds nothing
          const float z = lse[r] == SWA_NEG_INF ? 0.f : lse[r] * kLog2e;
          // nor does a row to a slot that it does not see, when its lse is NaN (-inf - NaN is NaN)
          add.x += s.x == SWA_NEG_INF ? 0.f : ex2(s.x - z);
          add.y += s.y == SWA_NEG_INF ? 0.f : ex2(s.y - z);
          add.z += s.z == SWA_NEG_INF ? 0.f : ex2(s.z - z);
          add.w += s.w == SWA_NEG_INF ? 0.f : ex2(s.w - z);
        }
      }
      // Slots that nobody saw have scores -inf and keep their weight.
      *w = make_float4(old.x + add.x, old.y + add.y, old.z + add.z, old.w + add.w);
    }
  }
}

struct Plan {
  int R, tiles, MT, RT, NRT, rows, parts, ck;
  int group;  // sequences per launch
  size_t off_ml, off_po, off_scores, bytes;
  size_t off_prefix;  // with a shared prefix: the workspace of its walk
  PrefixPlan prefix;
};

// Scores take whole units of this size, so that small tables have one size for every window (torch's
// allocator cuts large blocks into such units in any case).
constexpr size_t kScoreUnit = 2 << 20;

// The workspace's layout is the same for every window; the scores, at its end, are fewer under a smaller
// one.
Plan plan_of(int B, int Hq, int Hkv, int T, int D, int max_pages, int page, int accumulate, Reach reach) {
  Plan p;
  p.R = Hq / Hkv * T;
  p.ck = D == 256 ? AttnCfg<256>::CK : AttnCfg<128>::CK;
  // A team covers as many rows as share its chunks: 16, 32 or 64.
  p.MT = p.R <= 16 ? 1 : p.R <= 32 ? 2 : 4;
  p.RT = 16 * p.MT;
  p.NRT = (p.R + p.RT - 1) / p.RT;
  p.rows = p.R < p.RT ? p.R : p.RT;
  const int64_t slots = static_cast<int64_t>(max_pages) * page;
  const int64_t chunks = reach.sinks == 0 && reach.base == 0  // of an item
                             ? most_chunks(T, reach.window, slots, p.ck)
                             : most_chunks(T, reach, slots, p.ck);
  p.tiles = 1;
  size_t parts = static_cast<size_t>(sm_count()) * (kWarps / p.MT);
  if (p.R > 16 && D < 256) {
    // Two tiles a warp halve the conversions of a chunk's codes, and twice as many chunks are in work;
    // but twice as many parts have twice the partial results.  So long walks take them, by the most that
    // the table and the window allow (32 / 8 heads, T = 8, D = 128, 64 sequences of 4,000: 146 us and 174
    // with one; under a window of 1024, 16 sequences: 34 and 26).  Lengths are the device's alone, so
    // short contexts under a wide table take them too, to their loss (16 sequences of 1,000: 48 us and 35).
    parts *= 2;
    if (static_cast<int64_t>(B) * Hkv * p.NRT * chunks >= 32 * static_cast<int64_t>(parts)) {
      p.tiles = 2;
      p.MT /= 2;
    }
  }
  p.parts = sm_count() * (kWarps / p.MT);
  auto round = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  size_t off = round((kMaxSeqs + 1) * sizeof(int64_t));
  // partial results: two a part, and with a shared prefix one for every item that one team finishes
  size_t held = 2 * parts;
  p.group = kMaxSeqs;
  if (reach.base > 0) {
    p.group = prefix_group(kMaxSeqs, p.R);
    held += static_cast<size_t>(B < p.group ? B : p.group) * Hkv * p.NRT;
  }
  p.off_ml = off;
  off += round(held * p.rows * 2 * sizeof(float));
  p.off_po = off;
  off += round(held * p.rows * D * sizeof(float));
  p.off_prefix = off;
  if (reach.base > 0) {
    p.prefix = prefix_plan(B < p.group ? B : p.group, Hkv, p.R, D, reach.base);
    off += round(p.prefix.bytes);
  }
  p.off_scores = off;
  if (accumulate) {
    // The scores of all chunks that can be seen, in whole units, and no more than the table has (64
    // sequences, 32 / 8 heads, 131,072 slots, a window of 1024: 10 MB, 1.07 GB for the table).
    const size_t chunk = static_cast<size_t>(B < kMaxSeqs ? B : kMaxSeqs) * Hkv * p.NRT * p.rows * p.ck *
                         sizeof(float);
    const size_t table = chunk * (slots / p.ck);
    const size_t seen = (chunk * chunks + kScoreUnit - 1) / kScoreUnit * kScoreUnit;
    off += seen < table ? seen : table;
  }
  p.bytes = round(off);
  return p;
}

Reach args_reach(const CacheAttnArgs& args) { return {args.window, args.sinks, args.base}; }

template <int D, int kTiles>
cudaError_t launch_d(const CacheView& all, const CacheAttnArgs& args, const Plan& p,
                     cudaStream_t stream) {
  using C = AttnCfg<D, kTiles>;
  CUtensorMap tk, tv;
  const uint64_t planes = static_cast<uint64_t>(all.pages) * all.Hkv;
  if (!make_tmap_u8(&tk, all.k, planes, all.page, D, C::CK) ||
      !make_tmap_u8(&tv, all.v, planes, all.page, D, C::CK))
    return cudaErrorInvalidValue;
  cudaError_t e = allow_smem<swa_cache_attn_kernel<D, kTiles>>(C::kSmemBytes);
  if (e != cudaSuccess) return e;
  uint8_t* ws = static_cast<uint8_t*>(args.workspace);
  AttnDev a;
  a.R = p.R;
  a.MT = p.MT;
  a.RT = p.RT;
  a.NRT = p.NRT;
  a.rows = p.rows;
  a.reach = args_reach(args);
  a.whole = args.base > 0 ? 2 * p.parts : 0;
  a.parts = p.parts;
  a.f16 = args.dtype == SWA_FP16;
  a.scale_log2 = args.scale * kLog2e;
  a.page_log2 = all.page == 32 ? 5 : all.page == 64 ? 6 : 7;
  a.div_t = FastDiv(static_cast<uint32_t>(all.T));
  a.div_nrt = FastDiv(static_cast<uint32_t>(p.NRT));
  a.div_per = FastDiv(static_cast<uint32_t>(all.Hkv) * p.NRT);
  a.first = reinterpret_cast<int64_t*>(ws);
  a.ml = reinterpret_cast<float*>(ws + p.off_ml);
  a.po = reinterpret_cast<float*>(ws + p.off_po);
  a.scores = args.accumulate ? reinterpret_cast<float*>(ws + p.off_scores) : nullptr;
  PrefixDev pd;
  if (args.base > 0) {
    pd.table = all.table;
    pd.R = p.R;
    pd.reach = a.reach;
    pd.f16 = a.f16;
    pd.page_log2 = a.page_log2;
    pd.parts = p.prefix.parts;
    pd.stored = p.prefix.stored;
    pd.div_t = a.div_t;
    pd.div_r = FastDiv(static_cast<uint32_t>(p.R));
    pd.div_hkv = FastDiv(static_cast<uint32_t>(all.Hkv));
    pd.scale_log2 = a.scale_log2;
    uint8_t* pws = ws + p.off_prefix;
    pd.first = reinterpret_cast<int64_t*>(pws);
    pd.ml = reinterpret_cast<float*>(pws + p.prefix.off_ml);
    pd.po = reinterpret_cast<float*>(pws + p.prefix.off_po);
  }
  for (int b0 = 0; b0 < all.B; b0 += p.group) {
    CacheView c = all;
    c.B = all.B - b0 < p.group ? all.B - b0 : p.group;
    c.table += static_cast<size_t>(b0) * all.max_pages;
    c.lens += b0;
    if (c.new_lens) c.new_lens += b0;
    const size_t row0 = static_cast<size_t>(b0) * args.Hq * all.T;
    a.q = static_cast<const uint16_t*>(args.q) + row0 * D;
    a.o = static_cast<uint16_t*>(args.o) + row0 * D;
    a.lse = args.lse + row0;
    e = launch_early(swa_cache_attn_kernel<D, kTiles>, static_cast<unsigned>(p.parts / (kWarps / p.MT)),
                     kThreads, C::kSmemBytes, stream, tk, tv, c, a);
    if (e != cudaSuccess) return e;
    if (args.base > 0) {
      pd.q = a.q;
      pd.rows = c.B * p.R;
      pd.tiles = (pd.rows + kPrefixRows - 1) / kPrefixRows;
      if ((e = launch_cache_prefix(c, pd, stream)) != cudaSuccess) return e;
      // A warp 64 columns of a row where that fills the SMs, else 16.  (us of the call, with 128 / 64 / 32 / 16
      // columns.  D = 128, 32 / 8 heads: 64 sequences, a prefix of 32,768 84.7 / 83.4 / 87.1 / 92.4; 128 of 8 tokens,
      // 2,048 133 / 150 / 191 / 273.  D = 256, 32 / 16: 12 of 5 tokens, 4,096 76.4 / 77.6 / 84.3 / 94.7; 64, 16,384
      // 149 / 152 / 160 / 169.  D = 64, 32 / 8: 32, 8,192 - / 33.7 / 33.0 / 32.5.  2 and 8 sequences: the same.)
      const int64_t rows = static_cast<int64_t>(c.B) * c.Hkv * p.R, limit = 8ll * sm_count();
      constexpr int kWide = 64;
      const bool wide = rows * (D / kWide) >= 4ll * sm_count();
      const int64_t need = (rows * (D / (wide ? kWide : 16)) + 7) / 8;
      auto join = wide ? swa_cache_join_shared_kernel<D, kWide> : swa_cache_join_shared_kernel<D, 16>;
      e = launch_early(join, static_cast<unsigned>(need < limit ? need : limit), 256, 0, stream, c, a, pd);
      if (e != cudaSuccess) return e;
      continue;
    }
    // A warp a row where that fills the SMs; else a warp 16 columns of a row; and a block for them where
    // even those are few.  (us of the whole call, a window of 1024, 32 / 8 heads, D = 128, as a row / a
    // warp / a block: 1 sequence - / 12.6 / 11.2, 4 sequences 20.2 / 14 / 15.1, 16 sequences 21 / 18.6 /
    // 32.8, 32 sequences 23.6 / 24.6 / -; one of 30,000 tokens at D = 256: - / 48 / 37.)
    const int64_t rows = static_cast<int64_t>(c.B) * c.Hkv * p.NRT * p.rows, runs = rows * (D / 16);
    const int64_t most = 8ll * sm_count();
    auto join = swa_cache_join_kernel<D>;
    int64_t blocks = (rows + 7) / 8;
    if (runs <= 4ll * sm_count()) {
      join = swa_cache_join_few_kernel<D>;
      blocks = runs;
    } else if (rows < 6ll * sm_count()) {
      join = swa_cache_join_part_kernel<D>;
      blocks = (runs + 7) / 8;
    }
    e = launch_early(join, static_cast<unsigned>(blocks < most ? blocks : most), 256, 0, stream, c, a);
    if (e != cudaSuccess) return e;
    if (args.accumulate) {
      // At most this many chunks of 4 warps' turns; the kernel walks what there really is.
      const int64_t chunks = (static_cast<int64_t>(all.max_pages) * all.page / C::CK) * c.B * c.Hkv;
      const int64_t blocks = (chunks + 31) / 32;
      const unsigned wgrid = static_cast<unsigned>(blocks < most ? blocks : most);
      if ((e = launch_early(swa_cache_weights_kernel<D>, wgrid, 256, 0, stream, c, a)) != cudaSuccess)
        return e;
    }
  }
  return cudaSuccess;
}

}  // namespace

size_t cache_attn_workspace_bytes(int B, int Hq, int Hkv, int T, int D, int max_pages, int page,
                                  int window, int sinks, int base, int accumulate) {
  return plan_of(B, Hq, Hkv, T, D, max_pages, page, accumulate, {window, sinks, base}).bytes;
}

cudaError_t launch_cache_attn(const CacheView& c, const CacheAttnArgs& a, cudaStream_t stream) {
  const Plan p =
      plan_of(c.B, a.Hq, c.Hkv, c.T, c.D, c.max_pages, c.page, a.accumulate, args_reach(a));
  if (c.D == 64)
    return p.tiles == 2 ? launch_d<64, 2>(c, a, p, stream) : launch_d<64, 1>(c, a, p, stream);
  if (c.D == 128)
    return p.tiles == 2 ? launch_d<128, 2>(c, a, p, stream) : launch_d<128, 1>(c, a, p, stream);
  return launch_d<256, 1>(c, a, p, stream);
}

}  // namespace swa
