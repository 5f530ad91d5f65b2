// Brute-force check of swa_cache_split.h: every chunk of the list belongs to exactly one part, the
// chunks cover exactly the blocks of the visible slots, each item's parts are the ones part_of names,
// and no two of a team's partial results share a slot.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <set>
#include <vector>

#include "swa_cache_split.h"

using namespace swa;

#define CHECK(x)                                                     \
  do {                                                               \
    if (!(x)) {                                                      \
      std::printf("failed line %d: %s\n", __LINE__, #x);             \
      std::exit(1);                                                  \
    }                                                                \
  } while (0)

int main() {
  std::mt19937 rng(7);
  auto pick = [&](int lo, int hi) { return lo + static_cast<int>(rng() % (hi - lo + 1)); };
  for (int round = 0; round < 3000; ++round) {
    const int B = pick(1, 9), per = pick(1, 5), most = pick(1, 40), ck = pick(0, 1) ? 32 : 16;
    const int window = pick(0, 2) ? pick(1, 300) : 1 << 30;
    std::vector<int64_t> first(B + 1, 0);
    std::vector<int> len(B), n(B);
    for (int b = 0; b < B; ++b) {
      len[b] = pick(0, 3) ? pick(0, 700) : pick(0, 2);
      n[b] = pick(0, 4) ? pick(1, 20) : 0;
      const int c0 = first_chunk(len[b], window, ck), nc = chunk_count(len[b], n[b], window, ck);
      std::set<int> want;
      for (int t = 0; t < n[b]; ++t)
        for (int s = 0; s <= len[b] + t; ++s)
          if (len[b] + t - s < window) want.insert(s / ck);
      CHECK(static_cast<int>(want.size()) == nc);
      if (nc) CHECK(*want.begin() == c0 && *want.rbegin() == c0 + nc - 1);
      first[b + 1] = first[b] + nc;
    }
    const int64_t total = first[B] * per;
    const int size = pick(0, 1) ? pick(1, 4000) : pick(4000, 2000000);
    const int parts = used_parts(total, most, size);
    CHECK(parts >= 1 && parts <= most && parts <= (total > 0 ? total : 1));
    CHECK(used_parts(total, most, 1) == (total >= most ? most : total > 0 ? total : 1));
    CHECK(used_parts(total, most, size + 1000) <= parts);
    if (total == 0) continue;
    std::set<int> slots;
    const Parts cut(total, parts);
    CHECK(cut.start(0) == 0 && cut.start(parts) == total);
    for (int i = 0; i < parts; ++i) {
      const int64_t a = cut.start(i), z = cut.start(i + 1);
      CHECK(z >= a && z - a <= total / parts + 1);
      int64_t last_item = -1, item_from = 0;
      for (int64_t x = a; x <= z; ++x) {
        int64_t item = -1;
        if (x < z) {
          CHECK(cut.of(x) == i);
          const int b = sequence_at(first.data(), B, per, x);
          CHECK(b >= 0 && b < B && first[b] * per <= x && x < first[b + 1] * per);
          const int64_t nc = first[b + 1] - first[b];
          item = b * per + (x - first[b] * per) / nc;
        }
        if (item != last_item) {
          if (last_item >= 0) {  // the segment [item_from, x) of last_item ends
            const int b = static_cast<int>(last_item / per);
            const int64_t nc = first[b + 1] - first[b];
            const int64_t x0 = first[b] * per + (last_item % per) * nc;
            const bool begins = item_from == x0, ends = x == x0 + nc;
            CHECK(begins == (cut.start(i) <= x0));
            const int p0 = cut.of(x0), p1 = cut.of(x0 + nc - 1);
            CHECK((begins && ends) == (p0 == p1) && p0 <= i && i <= p1);
            if (!(begins && ends)) {
              const int s = partial_slot(i, begins);
              CHECK(s >= 0 && s < 2 * parts && slots.insert(s).second);
            }
          }
          last_item = item;
          item_from = x;
        }
      }
    }
    // every part between an item's first and last holds some of it: the join reads only what was written
    for (int64_t item = 0; item < static_cast<int64_t>(B) * per; ++item) {
      const int b = static_cast<int>(item / per);
      const int64_t nc = first[b + 1] - first[b];
      if (nc == 0) continue;
      const int64_t x0 = first[b] * per + (item % per) * nc;
      const int p0 = cut.of(x0), p1 = cut.of(x0 + nc - 1);
      if (p0 != p1)
        for (int p = p0; p <= p1; ++p) {
          CHECK(cut.start(p + 1) > cut.start(p));
          CHECK(slots.count(partial_slot(p, cut.start(p) <= x0)) == 1);
        }
    }
  }
  // past 32 bits
  for (int round = 0; round < 2000; ++round) {
    const int64_t total = (static_cast<int64_t>(rng()) << 8) + rng() % 1000 + 1;
    const int parts = pick(1, 1300);
    const Parts cut(total, parts);
    const int64_t x = static_cast<int64_t>((static_cast<unsigned __int128>(total) * rng()) >> 32);
    const int i = cut.of(x);
    CHECK(i >= 0 && i < parts && cut.start(i) <= x && x < cut.start(i + 1));
    CHECK(quotient(x, parts) == x / parts);
    CHECK(used_parts(total, parts, 16384) == parts);
  }
  std::puts("ok");
  return 0;
}
