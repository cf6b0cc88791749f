// Driver of walk_tiles (csrc/lb_pages.h) for the CPU tests: what the waves of a
// workgroup of k_attend_many read and write in LDS between two barriers, in the
// kernel's own order.  A place that a wave writes must not be one that any wave
// reads before the next barrier, and what is read must be what was put there.
// Prints how many reads were looked at; returns 1 with a message at the first mistake.
#include <cstdio>
#include <map>
#include <set>
#include <utility>

#include "../../binary_rank_gemv_littlebitlinear_amd/csrc/lb_pages.h"

using namespace lbi;

enum Kind { kKeys, kKeyScales, kValues };
using Place = std::pair<Kind, int>;

int main() {
  long reads = 0;
  for (int tiles = 0; tiles <= 40; ++tiles) {
    std::map<Place, int> holds;            // as of the last barrier
    std::map<Place, int> wrote;            // since
    std::set<Place> read;                  // since
    int barriers = 0;
    const char *wrong = nullptr;
    const auto see = [&](Kind kind, int place, int what) {
      const Place p = {kind, place};
      ++reads;
      read.insert(p);
      const auto it = holds.find(p);
      if (wrote.count(p)) wrong = "read where another wave may have written";
      if (it == holds.end() || it->second != what) wrong = "read what is not there";
    };
    const auto write = [&](Kind kind, int place, int what) {
      const Place p = {kind, place};
      if (read.count(p)) wrong = "written where another wave may still read";
      if (wrote.count(p) && wrote[p] >= 0) wrong = "written twice";
      wrote[p] = what;
    };
    const auto put = [&](int tile) {
      for (int i = 0; i < 2; ++i) {
        write(kKeys, keys_place(put_half(tile) + i), put_half(tile) + i);
        write(kKeyScales, keys_scale_place(put_half(tile) + i), put_half(tile) + i);
      }
      write(kValues, values_place(tile), tile);
    };
    walk_tiles(
        tiles,
        [&] {
          put(-1);
          put(0);
        },
        [&](int half) { see(kKeys, keys_place(half), half); },
        [&](int tile, int half) {
          see(kKeys, keys_place(2 * tile + half + 1), 2 * tile + half + 1);
          see(kKeyScales, keys_scale_place(2 * tile + half), 2 * tile + half);
          see(kValues, values_place(tile), tile);
        },
        put,
        [&] {
          ++barriers;
          for (const auto &w : wrote) holds[w.first] = w.second;
          wrote.clear();
          read.clear();
        });
    if (wrong) return printf("%d tiles: %s\n", tiles, wrong), 1;
    if ((tiles > 0) != (barriers > 0)) return printf("%d tiles: %d barriers\n", tiles, barriers), 1;
  }
  printf("%ld\n", reads);
  return 0;
}
