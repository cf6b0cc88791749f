// Driver of grown_bytes (csrc/lb_pages.h) for the CPU tests: the workspace of a cache
// whose calls' max_length grows from call to call, as a prompt's chunks' does, without
// a reservation.  Every outgrown workspace is kept.  Prints the most allocations and the
// most bytes kept, in hundredths of the final size; returns 1 with a message at the
// first mistake.
#include <cstdio>

#include "../../binary_rank_gemv_littlebitlinear_amd/csrc/lb_pages.h"

using namespace lbi;

#define CHECK(c) \
  if (!(c)) return printf("line %d: %s\n", __LINE__, #c), 1

int main() {
  int most_allocations = 0;
  double most_kept = 0;
  const int cus = 256;
  for (int Dp = 32; Dp <= 256; Dp += 32)
    for (int KV : {1, 2, 8, 32})
      for (int group : {1, 4, 32})
        for (int rows : {1, 2, 16, 100, 512, 2048})
          for (bool starts : {false, true}) {
            if (!starts && rows > 1) continue;
            size_t have = 0, kept = 0;
            int allocations = 0;
            const size_t bound = reserve_bytes(Dp, cus, kMaxTokens, 1, kMaxTokens);
            for (int most = rows; most <= 131072; most += rows < 64 ? 64 : rows) {
              const View A = {group, 1, 0, most};
              const Plan p = plan_of(KV, Dp, cus, starts, rows, 1, A);
              const size_t need = p.few_ws + p.many_ws;
              CHECK(need <= bound);
              if (need <= have) continue;
              const size_t now = grown_bytes(Dp, cus, have, need);
              CHECK(now >= need && now <= bound);
              kept += have;
              have = now;
              ++allocations;
            }
            if (!have) continue;
            // each one twice the one before, up to the bound: those before the last make less
            // than two of it, the doublings of a first one that holds a piece of 16 rows few
            CHECK(kept < 2 * have);
            CHECK(allocations <= 12);
            most_allocations = std::max(most_allocations, allocations);
            most_kept = std::max(most_kept, (double)kept / (double)have);
          }
  printf("%d %d\n", most_allocations, (int)(most_kept * 100));
  return 0;
}
