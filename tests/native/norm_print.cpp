// Prints the shape in which lb_norm is launched (csrc/lb_norm.h): threads of a row and
// pieces of a thread, for each pair of arguments: rows, width.
#include <cstdio>
#include <cstdlib>

#include "../../binary_rank_gemv_littlebitlinear_amd/csrc/lb_norm.h"

int main(int argc, char **argv) {
  for (int i = 1; i + 1 < argc; i += 2) {
    const lbi::NormShape s = lbi::norm_shape(atoll(argv[i + 1]), atoll(argv[i]));
    printf("%d %d\n", s.threads, s.pieces);
  }
  return 0;
}
