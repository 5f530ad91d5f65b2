// Brute-force check of ChunkWalk and most_chunks with sinks (swa_cache_split.h): the chunks of a sequence
// are those that hold a visible slot from `base` on, each once and in order.
#include <cstdio>
#include <random>
#include <set>

#include "swa_cache_split.h"

using namespace swa;

int main() {
  std::mt19937 rng(11);
  auto pick = [&](int lo, int hi) { return lo + static_cast<int>(rng() % (hi - lo + 1)); };
  for (int round = 0; round < 60000; ++round) {
    const int ck = pick(0, 1) ? 32 : 16, page = 32 << pick(0, 2), width = pick(1, 12), slots = page * width;
    const int T = pick(1, 9), n = pick(0, T), len = pick(0, slots - (n < slots ? n : slots));
    if (len + n > slots) continue;
    const int window = pick(0, 3) ? pick(1, 200) : slots, sinks = pick(0, 3) ? pick(0, 90) : pick(0, slots);
    const int base = pick(0, 1) ? 0 : page * pick(0, width - 1);
    std::set<int> want;
    for (int t = 0; t < n; ++t)
      for (int s = base; s <= len + t; ++s)
        if (len + t - s < window || s < sinks) want.insert(s / ck);
    const Reach r{window, sinks, base};
    const ChunkWalk w(len, n, r, ck);
    bool ok = static_cast<int>(want.size()) == w.count;
    int i = 0;
    for (int c : want) ok = ok && i < w.count && w.at(i++) == c;
    ok = ok && (w.count == 0 || w.last() == *want.rbegin());
    // where n is not known the chunks are the same
    ok = ok && (w.count == 0 || ChunkWalk(len, 1, r, ck).at(w.count - 1) == w.last());
    ok = ok && w.count <= most_chunks(T, r, slots, ck);
    if (base == 0 && sinks == 0)
      ok = ok && w.count == chunk_count(len, n, window, ck) &&
           (w.count == 0 || w.at(0) == first_chunk(len, window, ck));
    if (!ok) {
      std::printf("failed: ck %d len %d n %d window %d sinks %d base %d: %d chunks, want %d\n", ck, len, n,
                  window, sinks, base, w.count, static_cast<int>(want.size()));
      return 1;
    }
  }
  std::puts("ok");
  return 0;
}
