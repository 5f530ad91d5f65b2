// Brute-force check of most_chunks (swa_cache_split.h): no sequence that fits its table has more chunks,
// and, up to the table's own number, some sequence has as many.
#include <cstdio>

#include "swa_cache_split.h"

using namespace swa;

int main() {
  for (int ck = 16; ck <= 32; ck += 16)
    for (int slots = 32; slots <= 256; slots += 32)
      for (int T = 1; T <= 64; T += T < 6 ? 1 : 29)
        for (int window = 1; window <= slots; ++window) {
          const int64_t table = slots / ck, bound = most_chunks(T, window, slots, ck);
          const int64_t held = bound < table ? bound : table;
          int64_t most = 0;
          for (int len = 0; len <= slots; ++len)
            for (int n = 0; n <= T && len + n <= slots; ++n) {
              const int64_t c = chunk_count(len, n, window, ck);
              most = c > most ? c : most;
            }
          // a table shorter than T has no sequence of T queries, and may have fewer chunks than the bound
          if (most > held || (T <= slots - window && most != held)) {
            std::printf("failed: ck %d slots %d T %d window %d: %lld, bound %lld\n", ck, slots, T, window,
                        static_cast<long long>(most), static_cast<long long>(held));
            return 1;
          }
        }
  // no overflow at the ends
  if (most_chunks(64, 1 << 30, (1ll << 30) - 32, 16) != ((1ll << 30) - 32 + 14) / 16 + 1) {
    std::puts("failed: ends");
    return 1;
  }
  std::puts("ok");
  return 0;
}
