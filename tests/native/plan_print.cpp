// Prints the plan of an attention call (csrc/lb_pages.h): rows of a tile of
// k_attend_many, pieces of its items and of k_attend_few's.  Arguments: key heads,
// padded head width, CUs, whether there are starts, rows, sequences, query heads of a
// key head, window, keys.
#include <cstdio>
#include <cstdlib>

#include "../../binary_rank_gemv_littlebitlinear_amd/csrc/lb_pages.h"

int main(int argc, char **argv) {
  if (argc != 10) return 1;
  int a[9];
  for (int i = 0; i < 9; ++i) a[i] = atoi(argv[i + 1]);
  const lbi::View view = {a[6], 1, a[7], a[8]};
  const lbi::Plan p = lbi::plan_of(a[0], a[1], a[2], a[3] != 0, a[4], a[5], view);
  printf("%d %d %d\n", p.many ? p.tr : 0, p.many_pieces, p.few ? p.few_pieces : 0);
  return 0;
}
