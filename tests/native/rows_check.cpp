// Driver of csrc/lb_rows.h for the CPU tests: `meet` against marking every
// byte, for all small pairs of strided arrays.  Prints the number of pairs, of
// those that share a byte, and of those without one that are refused all the
// same (different pitches, or at a buffer's ends).
#include <cstdio>
#include <cstring>

#include "../../binary_rank_gemv_littlebitlinear_amd/csrc/lb_rows.h"

int main() {
  static char mem[64];
  long pairs = 0, shared = 0, cautious = 0, blocks = 0, refused_blocks = 0;
  for (int64_t ra = 0; ra <= 3; ++ra)
    for (int64_t rb = 0; rb <= 3; ++rb)
      for (size_t pa = 1; pa <= 6; ++pa)
        for (size_t pb = 1; pb <= 6; ++pb)
          for (size_t wa = 1; wa <= pa; ++wa)
            for (size_t wb = 1; wb <= pb; ++wb)
              for (int ob = 0; ob <= 40; ++ob) {
                const lbi::Rows a = {mem + 20, ra, pa, wa}, b = {mem + ob, rb, pb, wb};
                char used[64];
                memset(used, 0, sizeof used);
                for (int64_t r = 0; r < ra; ++r) memset(used + 20 + r * pa, 1, wa);
                bool truth = false;
                for (int64_t r = 0; r < rb; ++r)
                  for (size_t i = 0; i < wb; ++i) truth |= used[ob + r * pb + i] != 0;
                const bool got = lbi::meet(a, b);
                if (got != lbi::meet(b, a)) return printf("not symmetric\n"), 1;
                if (truth && !got) return printf("a shared byte was missed\n"), 1;
                ++pairs;
                shared += truth;
                cautious += got && !truth;
                // column blocks of one buffer: neither wraps round a row's end
                const int at = (ob - 20 + 60 * (int)pa) % (int)pa;
                if (ra > 1 && rb > 1 && pa == pb && !truth && (size_t)at >= wa && at + wb <= pa) {
                  ++blocks;
                  refused_blocks += got;
                }
              }
  printf("%ld %ld %ld %ld %ld\n", pairs, shared, cautious, blocks, refused_blocks);
  return 0;
}
