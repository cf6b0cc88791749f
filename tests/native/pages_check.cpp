// Driver of csrc/lb_pages.h for the CPU tests: the work items of random calls,
// laid out as the kernels lay them out, with starts, lengths and pages that are
// good in half of the calls and anything in the others.  Prints how many calls,
// rows and pieces were looked at; returns 1 with a message at the first mistake.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "../../binary_rank_gemv_littlebitlinear_amd/csrc/lb_pages.h"

using namespace lbi;

static uint64_t seed = 88172645463325252ull;
static int rnd(int lo, int hi) {  // both included
  seed ^= seed << 13;
  seed ^= seed >> 7;
  seed ^= seed << 17;
  return lo + (int)(seed % (uint64_t)(hi - lo + 1));
}

#define CHECK(c) \
  if (!(c)) return printf("line %d: %s\n", __LINE__, #c), 1

// As the kernels' search: the last sequence whose items begin at or before `item`.
static int find(const Sequences &S, int64_t item, int mul, int lg, int extra, int64_t *first) {
  int found = -1;
  for (int b = 0; b < S.n; ++b)
    if (first_item(S, b, mul, lg, extra) <= item) found = b, *first = first_item(S, b, mul, lg, extra);
  return found;
}

int main() {
  long rows_seen = 0, pieces_seen = 0;
  int calls = 0;
  for (; calls < 60000; ++calls) {
    const bool good = rnd(0, 1), starts = rnd(0, 3) > 0;
    Sequences S;
    const int lg = rnd(4, 6);
    S.n = rnd(1, 6);
    S.columns = rnd(1, 5);
    S.ldt = S.columns + rnd(0, 2);
    S.pages = rnd(1, 20);
    std::vector<int> start(S.n + 1), length(S.n), table(S.n * S.ldt, 1 << 29);
    const int cap = S.columns << lg;
    for (int b = 0; b < S.n; ++b) {
      length[b] = good ? rnd(0, cap) : rnd(0, 4) ? rnd(-3, 2 * cap) : rnd(0, 1) ? INT32_MAX : INT32_MIN;
      for (int c = 0; c < S.columns; ++c) table[b * S.ldt + c] = rnd(0, 9) ? rnd(0, S.pages - 1) : rnd(0, 1) ? -1 : S.pages;
    }
    start[0] = good ? 0 : rnd(-2, 5);
    for (int b = 0; b < S.n; ++b)
      start[b + 1] = good ? start[b] + rnd(0, rnd(0, 2) ? 3 : 70) : rnd(0, 5) ? start[b] + rnd(0, 40) : rnd(-100, 300);
    S.rows = starts ? (good ? start[S.n] + rnd(0, 2) : rnd(1, 200)) : S.n;
    S.start = starts ? start.data() : nullptr;
    S.lengths = length.data();
    S.table = table.data();
    if (S.rows == 0) continue;

    // appending by pages and reading by units of 16: every row with a position in
    // range is in one item, at its own place
    for (int unit = 0; unit < 2; ++unit) {
      const int l2 = unit ? 4 : lg;
      std::vector<int> count(S.rows, 0);
      const int64_t items = starts ? (S.rows >> l2) + 2 * (int64_t)S.n : S.n;
      for (int64_t item = 0; item < items; ++item) {
        int64_t first = item;
        const int b = starts ? find(S, item, 1, l2, 2, &first) : (int)item;
        if (b < 0) continue;
        const Sequence q = sequence(S, b);
        CHECK(q.row0 >= 0 && q.rows >= 0 && q.row0 + q.rows <= S.rows);
        int p0, p1, block, a, e;
        row_tokens(S, q, lg, &p0, &p1);
        if (unit) p1 = q.length;
        if (!touched(p0, p1, l2, item - first, &block, &a, &e)) continue;
        CHECK(a < e && a >= 0 && e <= 1 << l2);
        const int page = page_of(S, b, unit ? block >> (lg - 4) : block);
        CHECK(page >= -1 && page < S.pages);
        for (int t = a; t < e; ++t) {
          const int pos = (block << l2) + t, row = row_of(q, pos);
          CHECK(row >= q.row0 && row < q.row0 + q.rows);
          CHECK(pos == q.length - q.rows + row - q.row0 && (unit || pos < cap));
          ++count[row];
        }
      }
      if (good || !starts)
        for (int b = 0; b < S.n; ++b) {
          const Sequence q = sequence(S, b);
          for (int i = 0; i < q.rows; ++i) {
            const int64_t pos = (int64_t)q.length - q.rows + i;
            CHECK(count[q.row0 + i] == (pos >= 0 && (unit || pos < cap)));
            ++rows_seen;
          }
        }
    }

    // attention: every row of every head group is in one item, whose pieces hold
    // all its keys and fit grid and workspace
    View A;
    A.group = rnd(0, 3) ? rnd(1, 9) : rnd(10, 40);
    A.causal = rnd(0, 2) > 0;
    A.window = A.causal && rnd(0, 2) == 0 ? rnd(1, cap + 5) : 0;
    A.most = rnd(0, 1) ? cap : rnd(1, cap);
    const int KV = rnd(1, 3), Dp = 32 * rnd(1, 8), cus = rnd(1, 300);
    const Plan p = plan_of(KV, Dp, cus, starts, S.rows, S.n, A);
    // (the smallest pieces of the kernels hold more keys than these tables, so cut them again)
    int few_chunk = p.few_chunk, many_chunk = p.many_chunk, few_pieces = p.few_pieces, many_pieces = p.many_pieces;
    if (rnd(0, 1)) {
      const auto span = [&](int rows) { return A.window ? std::min(A.most, A.window + rows / A.group + 17) : A.most; };
      if (p.few) few_pieces = cut(p.few_items, span(p.frows), 50, 16, &few_chunk);
      if (p.many) many_pieces = cut(p.many_items, span(p.tr), 50, 16, &many_chunk);
    }
    std::vector<int> seen((size_t)S.rows * A.group, 0);
    const auto item = [&](const Sequence &q, int r0, int n, int chunk, int pieces) {
      int lo, hi;
      keys_of_rows(A, q, r0, n, &lo, &hi);
      CHECK(lo >= 0 && lo % 16 == 0 && hi <= A.most && hi <= q.length && lo <= hi);
      CHECK(pieces_of(lo, hi, chunk) <= pieces);
      pieces_seen += pieces_of(lo, hi, chunk);
      for (int r = r0; r < r0 + n; ++r) {
        int first, last;
        keys_of_row(A, q, r, &first, &last);
        CHECK(first >= 0 && last <= A.most);
        CHECK(first >= last || (lo <= first && last <= hi));
        const int64_t pos = (int64_t)q.length - q.rows + r / A.group;
        for (int t = 0; t < std::min(q.length, A.most); t += 7)
          CHECK((t >= first && t < last) == ((!A.causal || t <= pos) && (!A.window || t > pos - A.window)));
        const int64_t at = (int64_t)(q.row0 + r / A.group) * A.group + r % A.group;
        CHECK(at >= 0 && at < (int64_t)seen.size());
        ++seen[at];
      }
      return 0;
    };
    if (p.few) {
      CHECK(p.few_items == (int64_t)S.n * KV * p.tiles && p.frows >= 1 && p.frows <= 16);
      for (int b = 0; b < S.n; ++b)
        for (int tile = 0; tile < p.tiles; ++tile) {
          const Sequence q = sequence(S, b);
          const int64_t rows = (int64_t)q.rows * A.group;
          if (rows > p.few_rows || tile * 16 >= rows) continue;
          const int n = (int)std::min<int64_t>(16, rows - tile * 16);
          CHECK(n <= p.frows);
          if (item(q, tile * 16, n, few_chunk, few_pieces)) return 1;
        }
    }
    if (p.many) {
      const int tlg = p.tr == 256 ? 8 : 7;
      CHECK(p.tr == 1 << tlg && starts);
      for (int slot = 0; slot < p.row_tiles; ++slot) {
        int64_t first;
        const int b = find(S, slot, A.group, tlg, 1, &first);
        if (b < 0) continue;
        const Sequence q = sequence(S, b);
        const int64_t rows = (int64_t)q.rows * A.group, r0 = (slot - first) * p.tr;
        if (rows <= p.few_rows || r0 >= rows) continue;
        if (item(q, (int)r0, (int)std::min<int64_t>(p.tr, rows - r0), many_chunk, many_pieces)) return 1;
      }
    }
    if (good || !starts)
      for (int b = 0; b < S.n; ++b) {
        const Sequence q = sequence(S, b);
        for (int i = 0; i < q.rows * A.group; ++i) CHECK(seen[(size_t)q.row0 * A.group + i] == 1);
      }
  }

  // the workspace: every plan's fits what is reserved for calls at least as large
  for (int i = 0; i < 200000; ++i, ++calls) {
    View A;
    A.group = rnd(1, rnd(0, 1) ? 8 : 128);
    A.causal = 1;
    A.window = rnd(0, 3) ? 0 : rnd(1, 1 << rnd(1, 20));
    A.most = rnd(1, 1 << rnd(1, 20));
    const int KV = rnd(1, 1 << rnd(0, 6)), Dp = 32 * rnd(1, 8), cus = rnd(0, 1) ? 256 : rnd(1, 304);
    const bool starts = rnd(0, 1);
    const int64_t n = rnd(1, 1 << rnd(0, 10)), rows = starts ? rnd(1, 1 << rnd(0, 16)) : n;
    const Plan p = plan_of(KV, Dp, cus, starts, rows, n, A);
    CHECK(p.few_ws + p.many_ws <= reserve_bytes(Dp, cus, rows + rnd(0, 9), A.group, std::min(1 << 30, A.most + rnd(0, 99))));
    CHECK(p.few || p.many);
    CHECK(!p.few || (p.few_chunk >= kFewChunk && p.few_chunk % 16 == 0));
    CHECK(!p.many || (p.many_chunk >= kManyChunk && p.many_chunk % 64 == 0));
    CHECK((p.few_pieces > 1) <= (p.few_items * p.few_pieces <= kFewPieces));
    CHECK((p.many_pieces > 1) <= (p.many_items * p.many_pieces <= kManyPieces));
  }
  printf("%d %ld %ld\n", calls, rows_seen, pieces_seen);
  return 0;
}
