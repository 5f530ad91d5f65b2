// sinks_check.cpp — CPU check of the walk over key blocks with sinks (swa::KeyWalk, column_visible and
// sink_plan in swa_kernels.h) against brute force over the visibility rule: query i at position
// p = i + off sees key j iff dmin <= p - j and (p - j <= dmax or j < sinks).
// Prints "ok <cases>" and exits 0, or prints the first mismatch and exits 1.
#include <cstdio>
#include <vector>

#include "swa_kernels.h"

namespace {

int fail(const char* what, const swa::Span& sp, int sinks, int q0, int at) {
  std::printf("mismatch %s: Lq=%d Lk=%d dmin=%d dmax=%d sinks=%d q0=%d: %d\n", what, sp.Lq, sp.Lk, sp.dmin,
              sp.dmax, sinks, q0, at);
  return 1;
}

}  // namespace

int main() {
  using swa::kBlockM;
  using swa::kBlockN;
  long long cases = 0;
  const int lks[] = {1, 2, 127, 128, 129, 257, 700}, lqs[] = {1, 130, 1000}, ws[] = {1, 7, 128, 129, 300};
  const int counts[] = {1, 5, 32, 33, 127, 128, 129, 160, 161, 256, 300, 700};
  for (int Lk : lks)
    for (int lq : lqs)
      for (int W : ws)
        for (int sinks : counts)
          for (int causal = 0; causal < 2; ++causal) {
            const int Lq = lq < Lk ? lq : Lk;
            if (sinks > Lk) continue;
            const swa::Span sp{Lq, Lk, Lk - Lq, causal ? 0 : -(W - 1), W - 1};
            auto visible = [&](int i, int j) {
              const int d = i + sp.off - j;
              return d >= sp.dmin && (d <= sp.dmax || j < sinks);
            };
            for (int q0 = 0; q0 < Lq; q0 += kBlockM) {
              ++cases;
              swa::KeyWalk<true> walk;
              walk.set(sp, sinks, q0);
              std::vector<int> times((Lk + kBlockN - 1) / kBlockN);
              for (int j = 0, last = -1; j < walk.nkv; ++j) {
                const int k0 = walk.k0(j);
                if (k0 % kBlockN != 0 || (k0 <= last && !walk.is_narrow(j - 1)) || k0 >= Lk)
                  return fail("order", sp, sinks, q0, j);
                // a narrow block is the last of the far ones, and holds the last sink
                if (walk.is_narrow(j) && (j != 0 || !walk.is_far(0) || sinks <= k0 || sinks > k0 + swa::kNarrowSinks))
                  return fail("narrow", sp, sinks, q0, j);
                last = walk.is_narrow(j) ? -1 : k0;
                ++times[k0 / kBlockN];
                for (int i = q0; i < q0 + kBlockM && i < Lq; ++i) {
                  const int rel = i + sp.off - k0, lo = rel - sp.dmax;
                  const int hi = rel - sp.dmin < Lk - 1 - k0 ? rel - sp.dmin : Lk - 1 - k0;
                  for (int c = 0; c < kBlockN; ++c) {
                    const bool see = k0 + c < Lk && visible(i, k0 + c);
                    if (swa::column_visible<true>(c, lo, hi, sinks - k0) != see)
                      return fail("column", sp, sinks, q0, k0 + c);
                    if (sp.interior(q0, k0) && !see) return fail("interior", sp, sinks, q0, k0 + c);
                    if (walk.is_far(j) && see != (k0 + c < sinks))
                      return fail("far block", sp, sinks, q0, k0 + c);
                  }
                }
              }
              for (int i = q0; i < q0 + kBlockM && i < Lq; ++i)
                for (int j = 0; j < Lk; ++j)
                  if (visible(i, j) && times[j / kBlockN] != 1) return fail("block", sp, sinks, q0, j);
              swa::KeyWalk<false> plain;
              plain.set(sp, sinks, q0);
              if (plain.nkv != sp.last_kblock(q0) - sp.first_kblock(q0) + 1 || plain.is_far(0) ||
                  plain.k0(0) != sp.first_kblock(q0) * kBlockN)
                return fail("window", sp, sinks, q0, 0);
            }
            for (int width = 1; width <= 2; ++width) {
              swa::Problem pb{};
              pb.B = 2, pb.Hq = 6, pb.Hkv = 2, pb.D = 64, pb.span = sp, pb.sinks = sinks;
              const swa::SinkPlan p = swa::sink_plan(pb, width, 152 / width);
              if (p.blocks * width * kBlockN < sinks || p.splits < 1 ||
                  p.splits > 3 * ((Lq + kBlockM - 1) / kBlockM) || p.blocks * p.splits > 152)
                return fail("plan", sp, sinks, width, p.splits);
            }
          }
  std::printf("ok %lld\n", cases);
  return 0;
}
