// swa_cache_prefix.h — interface between the attention over a shared prefix (swa_cache_prefix.cu) and
// the join of its partial results with those of what follows the prefix (swa_cache_attn.cu).
#pragma once

#include "swa_cache_kernels.h"
#include "swa_cache_split.h"

namespace swa {

constexpr int kPrefixRows = 128;    // query rows of a tile
constexpr int kPrefixTiles = 512;   // tiles of rows per launch
constexpr int kPrefixSeqs = 1024;   // and sequences

// The rows that share a kv head are those of all sequences, R = G T each, one after another, in tiles of
// kPrefixRows.  A tile and a kv head are an item; the prefix slots that any row of the tile sees are cut
// into chunks, and the list of all items' chunks into parts as swa_cache_split.h does (with the tiles in
// the place of the sequences).
struct PrefixDev {
  const uint16_t* q;
  const int* table;     // the call's first: its first entries are all tables'
  int R, tiles, rows;   // rows of a sequence; tiles; rows of all sequences
  Reach reach;          // window, sinks, and the first slot behind the prefix
  int f16, page_log2, parts;
  int stored;           // rows of a partial result: min(rows, kPrefixRows)
  FastDiv div_t, div_r, div_hkv;
  float scale_log2;
  int64_t* first;       // [tiles + 1] chunks before each tile
  float* ml;            // [2 parts + items][stored][2] maxima (base 2) and sums
  float* po;            // [2 parts + items][stored][D]
};

struct PrefixPlan {
  int tiles, parts, stored;
  size_t off_ml, off_po, bytes;
};
// Keys of a chunk: the tensor core's operands and two stages of them fill shared memory.
SWA_HD int prefix_chunk(int D) { return D == 256 ? 64 : 128; }
// Parts that the list is cut into: by used_parts' rule, whose partial results cost half here, since they are
// still in the L2 when they are read.  Against the rule as it is, with fewer and longer parts, this wins as often
// as it loses (us of the call, half / whole; sequences, tokens, kv heads, prefix).  D = 256: 12, 5, 16, 4,096 with a
// window 70.7 / 72.7; 12, 5, 16, 2,048 45.3 / 51.2; 64, 1, 8, 4,096 60.5 / 69.4; 30, 1, 4, 2,048 33.5 / 39.0; but 64,
// 1, 16, 4,096 125 / 108.  D = 128: 64, 1, 8, 2,048 43.1 / 44.8, but 4,096 52.2 / 43.2, and 64, 1, 4, 8,192 39.2 /
// 35.4; 2, 1, 8, 32,768 43.4 / 43.9.  D = 64: 64, 1, 8, 2,048 35.5 / 32.8.  Within 2 % elsewhere (8 to 64 sequences,
// prefixes of 1,024 to 32,768).
SWA_HD int prefix_parts(int64_t total, int parts, int stored, int D) {
  return used_parts(total, parts, stored * D / 2);
}
PrefixPlan prefix_plan(int B, int Hkv, int R, int D, int base);
// Sequences per launch: their rows are at most kPrefixTiles tiles.
inline int prefix_group(int most, int R) {
  const int n = kPrefixTiles * kPrefixRows / R;
  return n < most ? n : most;
}

cudaError_t launch_cache_prefix(const CacheView& c, const PrefixDev& a, cudaStream_t stream);

}  // namespace swa
