// How lb_norm is launched (host arithmetic only).
#pragma once
#include <cstdint>

namespace lbi {

// Threads of a row x pieces of 8 columns of each: many threads share out the latency of
// few rows, few need less of the machine for many.  4096 wide, 1 row: 512 x 1 3.3 us,
// 256 x 2 3.8, 1024 x 1 4.0 (4096 rows: 31.7, 31.6, 35.8).  8192 wide with a norm on each
// side, 1 row: 1024 x 1 4.6, 512 x 2 4.8, 256 x 4 6.2; 1023 rows: 21.0, 18.0, 18.2; 4096
// rows: 77.1, 76.6, 81.4.  1031 wide: 64 x 3 and 256 x 1 take 8.6 and 7.7 for 1023 rows,
// 15.2 and 19.9 for 4096.
struct NormShape {
  int threads, pieces;
};
inline NormShape norm_shape(int64_t width, int64_t rows) {
  if (width <= 512) return {64, 1};
  if (width <= 1536 && rows >= 2048) return {64, 3};
  if (width <= 2048) return {256, 1};
  if (width <= 4096) return {512, 1};
  if (width <= 8192) return rows >= 256 ? NormShape{512, 2} : NormShape{1024, 1};
  return {1024, width <= 16384 ? 2 : 4};
}

}  // namespace lbi
