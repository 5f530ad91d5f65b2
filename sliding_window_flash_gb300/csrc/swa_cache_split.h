// swa_cache_split.h — how the attention over the paged cache divides its work, in functions that the
// host, the kernels and the CPU tests share.
//
// The visible slots of a sequence are cut at multiples of CK slots into chunks.  All chunks of all
// items (sequence, kv head, tile of query rows) form one list, item after item; the list is cut into
// as many parts as there are teams of warps, or fewer where their partial results would be more than
// they are worth, equal within one chunk whatever the sequences' lengths.
// A team walks its part from left to right: items that lie wholly inside it are finished there, and at
// most two, its first and its last, continue in a neighbour and leave a partial result.
#pragma once

#include <cmath>
#include <cstdint>

#ifdef __CUDACC__
#define SWA_HD __host__ __device__ __forceinline__
#else
#define SWA_HD inline
#endif

namespace swa {

// First slot that a query at slot `at` sees under `window`.
SWA_HD int visible_lo(int at, int window) { return at >= window ? at - window + 1 : 0; }

// First chunk and number of chunks of a sequence (0 chunks without queries): the n queries sit at
// slots len .. len + n - 1.
SWA_HD int first_chunk(int len, int window, int ck) { return visible_lo(len, window) / ck; }
SWA_HD int chunk_count(int len, int n, int window, int ck) {
  return n > 0 ? (len + n - 1) / ck - first_chunk(len, window, ck) + 1 : 0;
}

// Most chunks that T queries can see under `window` in a table of `slots`: of window + T - 1 consecutive
// slots, wherever they begin.
SWA_HD int64_t most_chunks(int T, int window, int64_t slots, int ck) {
  const int64_t span = static_cast<int64_t>(window) + T - 1;
  return ((span < slots ? span : slots) + ck - 2) / ck + 1;
}

// x / d for 0 <= x, 1 <= d, in 32 bits where they fit (a 64-bit division costs ten times as much).
SWA_HD int64_t quotient(int64_t x, int64_t d) {
  if (((x | d) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(d);
  return x / d;
}

// A list of `total` chunks in `parts` parts: the first `extra` have size + 1 chunks, the others size.
struct Parts {
  int64_t size;
  int parts, extra;
  SWA_HD Parts(int64_t total, int n)
      : size(quotient(total, n)), parts(n), extra(static_cast<int>(total - size * n)) {}
  // First chunk of part i (parts + 1 of them: the last is the total).
  SWA_HD int64_t start(int i) const { return size * i + (i < extra ? i : extra); }
  // The part of chunk x < total.
  SWA_HD int of(int64_t x) const {
    const int64_t longer = (size + 1) * extra;
    return static_cast<int>(x < longer ? quotient(x, size + 1) : extra + quotient(x - longer, size));
  }
};

// How many of `parts` parts a list of `total` chunks is cut into, when a part's partial result has `size`
// floats.  Parts of n chunks take about n us, and 8 size total / n bytes of partial results, written and
// read at 3 TB/s; the sum is least at n^2 = 8 size total / 3 MB.  n is rounded down.  (One kv head, 24
// rows, D = 256, 14,000 tokens: 21 us, 30 with all parts; 64 rows: 33 and 47.)
SWA_HD int used_parts(int64_t total, int parts, int size) {
  int64_t used = total;
  if (total * size >= 4 * 375000ll) {  // n is at least 2
    const int64_t n = static_cast<int64_t>(
        sqrtf(static_cast<float>(total) * (static_cast<float>(size) * (1.f / 375000.f))));
    used = n > 1 ? quotient(total + n - 1, n) : total;
  }
  return used >= parts ? parts : used < 1 ? 1 : static_cast<int>(used);
}

// A part's two partial results: 0 continues an item begun in an earlier part, 1 begins one.
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
