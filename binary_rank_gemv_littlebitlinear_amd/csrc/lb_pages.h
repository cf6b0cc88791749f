// Which rows, pages and keys the work items of the cache calls have: integer
// arithmetic alone, the same on the host (where it is tested) and the device.
// Starts, lengths and pages come from device memory and may hold anything: what
// is computed from them stays inside the call's rows, the table and the cache.
#pragma once
#include <algorithm>
#include <cstddef>
#include <cstdint>

#if defined(__HIPCC__)
#define LB_HD __host__ __device__ __forceinline__
#else
#define LB_HD inline
#endif

namespace lbi {

constexpr int kMaxTokens = 1 << 30;

LB_HD int imin(int a, int b) { return a < b ? a : b; }
LB_HD int imax(int a, int b) { return a > b ? a : b; }

// The sequences of a call, on the device: sequence b's rows are start[b] ..
// start[b + 1] - 1 (row b alone without start), its last tokens of lengths[b].
struct Sequences {
  const int *start, *lengths, *table;
  int64_t ldt;
  int n, rows, columns, pages;
};

struct Sequence {
  int row0, rows, length;  // the length as given, within [0, 2^30]
};

LB_HD Sequence sequence(const Sequences &S, int b) {
  Sequence q;
  q.row0 = S.start ? imin(imax(S.start[b], 0), S.rows) : b;
  q.rows = S.start ? imin(imax(S.start[b + 1], q.row0), S.rows) - q.row0 : 1;
  q.length = imin(imax(S.lengths[b], 0), kMaxTokens);
  return q;
}

// Work items of all sequences in one row: those of sequence b begin here, which
// leaves it floor(rows * mul / 2^lg) + extra of them or more.
LB_HD int64_t first_item(const Sequences &S, int b, int mul, int lg, int extra) {
  return (((int64_t)imin(imax(S.start[b], 0), S.rows) * mul) >> lg) + (int64_t)extra * b;
}

// Tokens before the table's end that the sequence's rows are, by position; rows at
// positions below 0 or past the table are none.
LB_HD void row_tokens(const Sequences &S, const Sequence &q, int lg, int *p0, int *p1) {
  *p0 = imax(0, q.length - q.rows);
  *p1 = imin(q.length, S.columns << lg);
}

// The row of the token at position p.
LB_HD int row_of(const Sequence &q, int p) { return q.row0 + (q.rows - q.length) + p; }

// The index-th block of 2^lg tokens (page or unit) that the tokens p0 .. p1 - 1
// touch: its number, and the first and last + 1 of them in it; false past the last.
LB_HD bool touched(int p0, int p1, int lg, int64_t index, int *block, int *a, int *e) {
  if (p0 >= p1) return false;
  const int64_t at = (p0 >> lg) + index;
  if (at > (p1 - 1) >> lg) return false;
  const int base = (int)at << lg;
  *block = (int)at;
  *a = imax(0, p0 - base);
  *e = imin(1 << lg, p1 - base);
  return true;
}

// The page of a sequence's column, -1 if there is none.
LB_HD int page_of(const Sequences &S, int b, int column) {
  const int page = column < S.columns ? S.table[b * S.ldt + column] : -1;
  return page >= 0 && page < S.pages ? page : -1;
}

// What an attention call looks at.
struct View {
  int group;           // rows of a key head for each token
  int causal, window;  // window 0: none
  int most;            // keys of a sequence, at most what the table holds
};

// Rows are token * group + head.  The keys [first, last) that row r sees.
LB_HD void keys_of_row(const View &A, const Sequence &q, int r, int *first, int *last) {
  const int keys = imin(q.length, A.most), p = q.length - q.rows + r / A.group;
  *last = A.causal ? imax(0, imin(keys, p + 1)) : keys;
  *first = A.window ? imax(0, p - A.window + 1) : 0;
}

// The keys [lo, hi) that rows r0 .. r0 + n - 1 see together, lo a multiple of 16;
// 0, 0 if there are none.
LB_HD void keys_of_rows(const View &A, const Sequence &q, int r0, int n, int *lo, int *hi) {
  int unused;
  keys_of_row(A, q, r0, lo, &unused);
  keys_of_row(A, q, r0 + n - 1, &unused, hi);
  *lo &= ~15;
  if (*lo >= *hi) *lo = *hi = 0;
}

// Where k_attend_many keeps its tiles of 64 keys in LDS: halves of 32 keys (half h of
// tile t is number 2 t + h) in four places and their scales in eight, tiles of values
// and their scales in two.  Tile t of values is put there together with halves 2 t + 1
// and 2 t + 2 of keys, of which the first product is a half ahead of the rest.
LB_HD int keys_place(int half) { return half & 3; }
LB_HD int keys_scale_place(int half) { return half & 7; }
LB_HD int values_place(int tile) { return tile & 1; }
LB_HD int put_half(int tile) { return 2 * tile + 1; }

// The order of a workgroup's work on them.  `begin` puts half 0 and tile 0; `score` makes
// a half's first product; `weigh` has the rest of a half, and the first product of the
// half behind it; `put` puts a tile.  Between two barriers no wave puts what another may
// still read: the one behind score(0) keeps put(1), whose half 4 takes the place of half
// 0, behind the slowest wave's reading of that.
template <typename Begin, typename Score, typename Weigh, typename Put, typename Barrier>
LB_HD void walk_tiles(int tiles, const Begin &begin, const Score &score, const Weigh &weigh, const Put &put,
                      const Barrier &barrier) {
  if (tiles < 1) return;
  begin();
  barrier();
  score(0);
  barrier();
  for (int tile = 0; tile < tiles; ++tile) {
    weigh(tile, 0);
    put(tile + 1);
    weigh(tile, 1);
    barrier();
  }
}

LB_HD int pieces_of(int lo, int hi, int chunk) { return imax(1, (int)(((int64_t)hi - lo + chunk - 1) / chunk)); }

// How an attention call is cut up.  A sequence of up to few_rows rows (tokens x
// group) has tiles of 16 rows in k_attend_few, one with more has tiles of tr rows
// in k_attend_many; the keys of each are cut into pieces.
struct Plan {
  bool few = false, many = false;
  int few_rows = 0, tiles = 0, frows = 0;  // tiles a sequence may have, rows of a tile
  int few_chunk = 0, few_pieces = 1, many_chunk = 0, many_pieces = 1, row_tiles = 0, tr = 0;
  int64_t few_items = 0, many_items = 0;
  size_t few_ws = 0, many_ws = 0;  // bytes of partial sums
};

constexpr int kFewWhole = 1024;   // keys that k_attend_few does not cut
constexpr int kFewChunk = 256;    // keys of its smallest piece
constexpr int kFewLong = 2048;    // and of one that only evens out the work
constexpr int kManyChunk = 512;   // and of k_attend_many
constexpr int kFewPieces = 2048;  // the most of a call of k_attend_few
constexpr int kManyLong = 1024;   // (again, one that evens out the work)
constexpr int kManyPieces = 1024;  // the most of a call of k_attend_many

// Rows of a tile of k_attend_many: 256 where registers allow it (Dp <= 128), the GPU has
// more than two such tiles a CU and they are full of work, else 128 (two workgroups a CU).
// 256 against 128 rows, us, 128 wide:
//   tiles enough      32 heads: a prompt of 4096 (544 items of 256) 177 and 201, two of 4096
//                     352 and 364; of 2048 (288 items) 87 and 78; 64 heads, 2048, 105 and 113
//   rows enough, five tiles a sequence: a last tile is half empty on the average, every
//                     sequence has a place in the grid, and those with few rows run in
//                     workgroups of the same size.  32 heads: 16 prompts of 600 160 and 128,
//                     16 chunks of 300 of 4096 keys 637 and 538, a prompt of 4096 beside 60
//                     tokens 335 and 294; 64 heads on 8, 100 tokens beside 8 chunks of 100
//                     103 and 75; but 16 chunks of 256 of 4096 358 and 379
//   keys enough, 2048, a window 4096: of 256 rows' keys more are hidden from some of them.
//                     32 heads: 8 prompts of 1024 148 and 139, 6 of 1500 192 and 190, 4 of
//                     2048 206 and 212; one of 8192 644 and 675, with a window of 4096 512 and
//                     529, of 2048 364 and 343, of 1024 232 and 215
inline int many_tile(int KV, int Dp, int cus, int64_t rows, int64_t n, const View &A) {
  const int64_t all = rows * A.group;
  const bool full = (all / 256 + n) * KV > 2 * cus && all >= 5 * 256 * n;
  return Dp <= 128 && full && A.most >= 2048 && (A.window == 0 || A.window >= 4096) ? 256 : 128;
}

// Pieces of an item's keys: about `target` for all items together, of `least`
// keys or more; `span` bounds an item's keys.
inline int cut(int64_t items, int64_t span, int64_t target, int64_t least, int *chunk) {
  const int64_t each = std::max<int64_t>(1, target / items);
  const int64_t c = std::max<int64_t>(least, ((span + each - 1) / each + 63) / 64 * 64);
  *chunk = (int)c;
  return (int)std::max<int64_t>(1, (span + c - 1) / c);
}

inline Plan plan_of(int KV, int Dp, int cus, bool starts, int64_t rows, int64_t n, const View &A) {
  Plan p;
  const int group = A.group;
  const int64_t per_row = (int64_t)Dp + 2;
  p.tr = many_tile(KV, Dp, cus, rows, n, A);
  if (!starts) {
    p.few = true;
    p.few_rows = group;
    p.tiles = (group + 15) / 16;
  } else {
    p.tiles = std::max(2, (group + 15) / 16);
    p.few_rows = 16 * p.tiles;
    p.many = rows * group > p.few_rows;
    p.few = n > 1 || !p.many;
    if (!p.few) p.few_rows = 0;
    if (!p.many) p.tiles = (int)((rows * group + 15) / 16);
  }
  p.frows = std::min(16, std::max(1, p.few_rows));
  // the keys of tile_rows rows: from the first's window, cut down to a unit, to the last's position
  const auto span_of = [&](int64_t tile_rows) {
    return A.window ? std::min<int64_t>(A.most, A.window + tile_rows / group + 1 + 16) : (int64_t)A.most;
  };
  if (p.few) {
    p.few_items = n * KV * p.tiles;
    const int64_t span = span_of(p.frows);
    // Few items are cut to have one for each CU.  Then nothing is left that takes much
    // longer than the rest, which pays only for long pieces.  64 heads of 128 on 8:
    // 64 sequences of up to 4096 keys 49 us in pieces of 2048, 53 whole and 51 in pieces
    // of 1024; of up to 16384 169, 200 and 169; 25 of up to 32768 140 and 207; but 30 of
    // up to 4096 31 in pieces of 2048 and 29 whole, one of 131072 62 and 59 in 4096s.
    p.few_pieces = cut(p.few_items, span, std::min(cus, kFewPieces), span <= kFewWhole ? kFewWhole : kFewChunk, &p.few_chunk);
    int chunk;
    const int pieces = cut(p.few_items, span, kFewPieces, p.few_items >= cus ? kFewLong : 2 * kFewLong, &chunk);
    if (pieces > p.few_pieces) {
      p.few_pieces = pieces;
      p.few_chunk = chunk;
    }
    if (p.few_pieces > 1) p.few_ws = (size_t)(p.few_items * p.few_pieces * p.frows * per_row) * 4;
  }
  if (p.many) {
    p.row_tiles = (int)(rows * group / p.tr + n);
    p.many_items = (int64_t)p.row_tiles * KV;
    // The same here, while there is little more than an item for each CU (a CU has room
    // for two) and keys enough to pay for joining.  In pieces of 1024 and whole: a prompt
    // of 4096 with 8 heads of 128 85 us and 131, of 256 200 and 323; 6 chunks of 300 rows
    // of up to 8000 keys, 32 heads on 8, 140 and 244; 500 rows of 9000 keys, 32 heads, 138
    // and 159.  But a prompt of 1500 with 32 heads 75 and 59, the last 1500 rows of 4500
    // keys (400 items) 196 and 167 in pieces of 2250.
    const int64_t span = span_of(p.tr);
    p.many_pieces = cut(p.many_items, span, std::min(cus, kManyPieces), kManyChunk, &p.many_chunk);
    int chunk;
    const int pieces = cut(p.many_items, span, kManyPieces, kManyLong, &chunk);
    if (p.many_items <= cus * 5 / 4 && span >= 4 * kManyLong && pieces > p.many_pieces) {
      p.many_pieces = pieces;
      p.many_chunk = chunk;
    }
    if (p.many_pieces > 1) p.many_ws = (size_t)(p.many_items * p.many_pieces * p.tr * per_row) * 4;
  }
  return p;
}

// Workspace that is enough for every call of up to `rows` rows, any number of
// sequences and `most` keys: an item has more than one piece only while all of
// them together stay below the target.
inline size_t reserve_bytes(int Dp, int cus, int64_t rows, int group, int64_t most) {
  const int64_t per_row = (int64_t)Dp + 2;
  size_t need = 0;
  if (most > kFewWhole) need += (size_t)((most > kFewLong ? kFewPieces : std::min(cus, kFewPieces)) * 16 * per_row) * 4;
  // (calls with 256-row tiles have more items than CUs and are not cut)
  if (most > kManyChunk && rows * group > 32)
    need += (size_t)((int64_t)(most > kManyLong ? kManyPieces : std::min(cus, kManyPieces)) * 128 * per_row) * 4;
  return need;
}

// The size of the workspace that takes the place of one of `have` bytes when a call needs
// more: twice that, up to what any call may need.  Outgrown ones are kept (captured graphs
// use them), so a size that followed each call's need would pile up as lengths grow:
// chunks of 16 tokens of a prompt of 131072 with 32 heads of 128 on one would keep 2.7 GB.
inline size_t grown_bytes(int Dp, int cus, size_t have, size_t need) {
  return std::max(need, std::min(2 * have, reserve_bytes(Dp, cus, kMaxTokens, 1, kMaxTokens)));
}

}  // namespace lbi
