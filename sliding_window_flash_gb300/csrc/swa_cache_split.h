// swa_cache_split.h — how the attention over the paged cache divides its work, in functions that the
// host, the kernels and the CPU tests share.
//
// The visible slots of a sequence are cut at multiples of CK slots into chunks.  All chunks of all
// items (sequence, kv head, tile of query rows) form one list, item after item; the list is cut into
// as many equal parts as there are teams of warps, whatever the sequences' lengths.  A team walks its
// part from left to right: items that lie wholly inside it are finished there, and at most two, its
// first and its last, continue in a neighbour and leave a partial result.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define SWA_HD __host__ __device__ __forceinline__
#else
#define SWA_HD inline
#endif

namespace swa {

// Visible slots [lo, hi) of the n > 0 queries at slots len .. len + n - 1 under `window`, all together.
SWA_HD int visible_lo(int len, int window) { return len >= window ? len - window + 1 : 0; }

// First chunk and number of chunks of a sequence (0 chunks without queries).
SWA_HD int first_chunk(int len, int window, int ck) { return visible_lo(len, window) / ck; }
SWA_HD int chunk_count(int len, int n, int window, int ck) {
  return n > 0 ? (len + n - 1) / ck - first_chunk(len, window, ck) + 1 : 0;
}

// Part i of `parts` of a list of `total` chunks starts here; parts are equal within one chunk.
SWA_HD int64_t part_start(int64_t total, int parts, int i) { return total * i / parts; }

// The part that chunk x of the list belongs to.
SWA_HD int part_of(int64_t total, int parts, int64_t x) {
  return static_cast<int>(((x + 1) * parts - 1) / total);
}

// A team's two partial results: 0 continues an item begun in an earlier part, 1 begins one.
SWA_HD int partial_slot(int part, bool begins) { return 2 * part + (begins ? 1 : 0); }

// Sequence that entry x of the list belongs to: the last b with first[b] * per <= x, where first[b]
// counts the chunks of the sequences before b, first[B] all of them, and x < first[B] * per.
SWA_HD int sequence_at(const int64_t* first, int B, int64_t per, int64_t x) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (first[mid] * per <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

}  // namespace swa
