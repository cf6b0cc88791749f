// The paged 8-bit cache: storage, appending (with the position rotation) and
// reading back.  See lb_cache.h for the layout.
//
// lb_cache_append: rows k, v of new tokens at positions p of their sequences.
//
//   k'   = R(p) k       pairs of the first `rot` dims turned by the angles of
//                       p's row of the table, in fp32
//   s'   = max(s, max |k'| / 127)   over the page's new tokens, s = 0 where the
//                       page's first token is among them
//   byte = rint(k' / s') + 128, and rint(byte s / s') for the page's earlier
//                       tokens where s' > s
//
// and the same for v without R; q' = R(p) q, rounded once to fp16.  A page that
// grows token by token therefore has the scale it would have got at once, and
// its numbers are off by half a step for each time the scale grew.  A page with
// a value that is not finite gets the scale NaN: all of it reads as NaN.
//
// A workgroup (a wave of it where most tokens come one at a time) has one head of
// one page, keys or values, and waves behind those turn the queries.  A thread
// keeps 4 tokens x 8 dims, the smallest block that is whole words of the cache for
// keys and values alike, in registers between finding the largest value and
// rounding; a page with more of them than threads has the rest read again (a
// prompt of 4096 took 61 us with all read twice, its reading back included, 47 now).
// Prompts are bound by reading and writing: 4096 tokens of 64 heads on 8, 128 wide,
// 159 MB in 32 to 35 us (4.5 to 5 TB/s, a copy's rate is 5.1).  A token is bound by a
// chain of loads (length, page, scale, rows): 7 us for 1 sequence as for 64.
#include <algorithm>
#include <new>

#include "lb_cache.h"

namespace {

using namespace lbi;

constexpr int64_t kMaxRows = (int64_t)1 << 30;

struct AppendArgs {
  Sequences S;
  const uint16_t *k, *v, *q;
  uint16_t *qo;
  int64_t ldk, ldv, ldq, ldqo;
  const float *rope;  // positions x rot: cosines, then sines
  uint8_t *kc, *vc;
  float *ks, *vs;
  int heads, KV, D, Dp, P, lg, rot, inter;
  int both;        // queries are whole heads of two partner halves, each a multiple of 8 dims
  int64_t items;   // page slots of the launch
  int64_t kvwgs;   // workgroups of keys and values; the others turn queries
  int qparts;      // waves a row of queries has
};

// Dims 8 e .. 8 e + 7 of a head's row x, turned by the cosines and sines at cs
// (rot / 2 of each).
__device__ __forceinline__ void turn8(const uint16_t *x, int e, int D, const float *cs, int rot, int inter,
                                      float (&o)[8]) {
  const int d0 = 8 * e, half = rot >> 1;
  const u32x4_t own = *LB_LOOSE128(x + d0);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[2 * i] = h2f((uint16_t)(own[i] & 0xffffu));
    o[2 * i + 1] = h2f((uint16_t)(own[i] >> 16));
  }
  if (d0 >= rot) return;
  if (inter) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int pair = (d0 >> 1) + i;
      if (pair >= half) break;
      const float c = cs[pair], s = cs[half + pair], a = o[2 * i], b = o[2 * i + 1];
      o[2 * i] = a * c - b * s;
      o[2 * i + 1] = a * s + b * c;
    }
    return;
  }
  if ((half & 7) == 0) {  // the partners are a group of 8 too
    const bool low = d0 < half;
    const u32x4_t other = *LB_LOOSE128(x + (low ? d0 + half : d0 - half));
    const float *cp = cs + (low ? d0 : d0 - half);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float p = h2f((uint16_t)(i & 1 ? other[i >> 1] >> 16 : other[i >> 1] & 0xffffu));
      const float c = cp[i], s = cp[half + i];
      o[i] = low ? o[i] * c - p * s : p * s + o[i] * c;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int d = d0 + i;
    if (d < half)
      o[i] = o[i] * cs[d] - h2f(x[d + half]) * cs[half + d];
    else if (d < rot)
      o[i] = h2f(x[d - half]) * cs[d] + o[i] * cs[d - half];
  }
}

__device__ __forceinline__ uint32_t to_byte(float v, float s) {
  // s = 0: the page holds zeros alone.  A NaN (of a page without a finite
  // scale) becomes 0.
  const float q = s > 0.f ? rintf(v / s) : 0.f;
  return (uint32_t)((int)fminf(fmaxf(q, -127.f), 127.f) + 128);
}
// A number rounded again for a scale that is 1 / f times larger.  In fp64: ratios of
// the scales of 16-bit numbers make exact halves, which fp32 would send either way.
__device__ __forceinline__ uint32_t again(uint32_t byte, double f) {
  return (uint32_t)((int)rint((double)((int)byte - 128) * f) + 128);
}

__device__ __forceinline__ float wave_amax(float v) {
  // keeps NaN, which fmaxf would drop
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const float o = __shfl_xor(v, d);
    v = o > v || o != o ? o : v;
  }
  return v;
}
__device__ __forceinline__ float amax(float m, float v) {
  v = fabsf(v);
  return v > m || v != v ? v : m;
}

// Dims 8 g .. 8 g + 7 of up to four new tokens, tok .. tok + 3 of the page; those
// outside a .. e - 1 are 0.  x: the row of token a; cs: the table's row of its
// position.
template <bool KEYS>
__device__ __forceinline__ void load_item(const AppendArgs &A, const uint16_t *x, const float *cs, int tok, int g, int a,
                                          int e, float (&v)[4][8]) {
  const int64_t ld = KEYS ? A.ldk : A.ldv;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = tok + j - a;
    if (r >= 0 && tok + j < e) {
      turn8(x + r * ld, g, A.D, KEYS ? cs + (int64_t)r * A.rot : nullptr, KEYS ? A.rot : 0, A.inter, v[j]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = 0.f;
    }
  }
}

// Writes those tokens' bytes.  Keys: 8 bytes a token.  Values: 4 bytes a dim, of
// which those of other tokens stay (earlier ones rounded again by f where grown).
template <bool KEYS>
__device__ __forceinline__ void store_item(const AppendArgs &A, uint8_t *out, int tok, int g, int a, int e, float s,
                                           bool grown, double f, const float (&v)[4][8]) {
  const int pairs = A.Dp / 64, c = g >> 3;
  const bool full = c < pairs;
  uint8_t *unit = out + (int64_t)(tok >> 4) * 16 * A.Dp + c * 1024;
  if (KEYS) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (tok + j < a || tok + j >= e) continue;
      u32x2_t w = {0, 0};
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i >> 2] |= to_byte(v[j][i], s) << (8 * (i & 3));
      const int lane = (g & 3) * 16 + (tok & 15) + j;
      *(u32x2_t *)(unit + (full ? lane * 16 + ((g >> 2) & 1) * 8 : lane * 8)) = w;
    }
    return;
  }
  const bool whole = tok >= a && tok + 4 <= e;
  const int i = (g >> 1) & 3;  // of the tiles of 16 dims in a pair
#pragma unroll
  for (int d = 0; d < 8; ++d) {
    const int lane = ((tok >> 2) & 3) * 16 + (g & 1) * 8 + d;
    uint32_t *to = (uint32_t *)(unit + (full ? lane * 16 : lane * 8) + i * 4);
    uint32_t w = 0;
    if (whole) {
#pragma unroll
      for (int j = 0; j < 4; ++j) w |= to_byte(v[j][d], s) << (8 * j);
    } else {
      const uint32_t was = *to;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t byte = (was >> (8 * j)) & 255u;
        w |= (tok + j >= e ? byte : tok + j < a ? (grown ? again(byte, f) : byte) : to_byte(v[j][d], s)) << (8 * j);
      }
    }
    *to = w;
  }
}

// One head of one page, by NT threads: new tokens a .. e - 1 of the page, whose
// first row is `row` (of token a, at position pos).  An item is 4 tokens x 8 dims;
// a thread keeps its first one, and reads later ones again when the scale is known.
template <int NT, bool KEYS>
__device__ void append_block(const AppendArgs &A, int64_t page, int h, int a, int e, int64_t row, int pos, float *part) {
  const int t = threadIdx.x % NT;
  const uint16_t *x = (KEYS ? A.k : A.v) + row * (KEYS ? A.ldk : A.ldv) + (int64_t)h * A.D;
  const float *cs = KEYS && A.rot ? A.rope + (int64_t)pos * A.rot : nullptr;
  float *scale = (KEYS ? A.ks : A.vs) + page * A.KV + h;
  const float before = a > 0 ? *scale : 0.f;
  const int groups = A.D / 8, tok0 = a & ~3, n = ((e - tok0 + 3) >> 2) * groups;
  float v[4][8];
  float m = 0.f, bad = 0.f;  // bad: NaN once a number is not finite
  const auto item = [&](int i, int &tok, int &g) {
    tok = tok0 + (i / groups) * 4;
    g = i % groups;
  };
  for (int i = t + (n - 1 - t) / NT * NT; i >= t; i -= NT) {  // the first last, to be kept
    int tok, g;
    item(i, tok, g);
    load_item<KEYS>(A, x, cs, tok, g, a, e, v);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        m = fmaxf(m, fabsf(v[j][k]));
        bad = fmaf(v[j][k], 0.f, bad);
      }
  }
  if (bad != bad) m = bad;
  m = wave_amax(m);
  if constexpr (NT > 64) {
    if ((t & 63) == 0) part[t >> 6] = m;
    __builtin_amdgcn_s_waitcnt(0);  // every thread has its scale before one writes it
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) m = amax(m, part[i]);
  }
  float s = m / 127.f;
  if (!(s < INFINITY)) s = __uint_as_float(0x7fc00000u);
  if (!(s > before) && s == s) s = before;
  const bool grown = a > 0 && s > before;
  const double f = grown ? (double)before / (double)s : 1.0;
  if (t == 0) *scale = s;

  uint8_t *out = (KEYS ? A.kc : A.vc) + (page * A.KV + h) * (int64_t)A.P * A.Dp;
  for (int i = t; i < n; i += NT) {
    int tok, g;
    item(i, tok, g);
    if (i != t) load_item<KEYS>(A, x, cs, tok, g, a, e, v);
    store_item<KEYS>(A, out, tok, g, a, e, s, grown, f, v);
  }
  if (!grown) return;
  // the page's earlier tokens, except values that share 4 bytes with new ones:
  // pieces of 16 bytes (a pair of 32 dims) and 8 (the odd 32)
  const int pairs = A.Dp / 64, odd = (A.Dp / 32) & 1, per = (pairs + odd) * 64;
  for (int i = t; i < ((a + 15) >> 4) * per; i += NT) {
    const int u = i / per, piece = i % per, c = piece >> 6, lane = piece & 63;
    const int last = KEYS ? u * 16 + (lane & 15) : u * 16 + 4 * (lane >> 4) + 3;
    if (last >= a) continue;
    uint8_t *to = out + (int64_t)u * 16 * A.Dp + (c < pairs ? piece * 16 : pairs * 1024 + lane * 8);
    uint32_t *word = (uint32_t *)to;
    for (int d = 0; d < (c < pairs ? 4 : 2); ++d) {
      const uint32_t was = word[d];
      uint32_t w = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) w |= again((was >> (8 * j)) & 255u, f) << (8 * j);
      word[d] = w;
    }
  }
}

// NT threads a block; a workgroup of 256 has 256 / NT of them.  Block = (page
// slot, head, keys or values).
template <int NT>
__global__ void __launch_bounds__(256) k_cache_append(AppendArgs A) {
  __shared__ float part[256 / 64];
  const Sequences &S = A.S;
  if (blockIdx.x < A.kvwgs) {
    const unsigned block = NT == 64 ? blockIdx.x * 4 + wave_id() : blockIdx.x;
    const unsigned item = block / (unsigned)(2 * A.KV);
    const int which = (int)(block - item * (2 * A.KV)), h = which >> 1;
    if (item >= A.items) return;
    int b = (int)item;
    int64_t first = item;
    if (S.start) b = find_sequence(S, item, 1, A.lg, 2, &first);
    if (b < 0) return;
    const Sequence q = sequence(S, b);
    int p0, p1, col, a, e;
    row_tokens(S, q, A.lg, &p0, &p1);
    if (!touched(p0, p1, A.lg, item - first, &col, &a, &e)) return;
    const int page = page_of(S, b, col);
    if (page < 0) return;
    const int pos = (col << A.lg) + a;
    const int64_t row = row_of(q, pos);
    if (which & 1)
      append_block<NT, false>(A, page, h, a, e, row, pos, part);
    else
      append_block<NT, true>(A, page, h, a, e, row, pos, part);
    return;
  }
  // queries: a wave turns some heads of a row, whole heads at a time, so that a
  // group's partner is read in the same step (q may be turned in place)
  const unsigned wv = (blockIdx.x - (unsigned)A.kvwgs) * 4 + wave_id();
  const unsigned row = wv / (unsigned)A.qparts;
  const int qp = (int)(wv - row * A.qparts), lane = threadIdx.x & 63, groups = A.D / 8, hpi = 64 / groups;
  if (row >= (unsigned)S.rows) return;
  int b = (int)row;
  int64_t first;
  if (S.start) b = find_sequence(S, row, 1, 0, 0, &first);
  if (b < 0) return;
  const Sequence q = sequence(S, b);
  int p0, p1;
  row_tokens(S, q, A.lg, &p0, &p1);
  const int pos = (int)row - q.row0 + (q.length - q.rows);
  if (pos < p0 || pos >= p1) return;
  const float *cs = A.rot ? A.rope + (int64_t)pos * A.rot : nullptr;
  if (A.both) {  // a lane has a group and its partner: half of the loads
    const int half = A.rot / 2, per = groups / 2, hl = lane / per, d = (lane - hl * per) * 8, hpi2 = 64 / per;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int h = (qp * 2 + i) * hpi2 + hl;
      if (hl >= hpi2 || h >= A.heads) continue;
      const uint16_t *x = A.q + row * A.ldq + (int64_t)h * A.D + d;
      const u32x4_t lo = *LB_LOOSE128(x), hi = *LB_LOOSE128(x + half);
      const float *cp = cs + d, *sp = cp + half;
      u32x4_t wl, wh;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float l[2], g[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float p = h2f((uint16_t)(lo[j] >> (16 * k))), q2 = h2f((uint16_t)(hi[j] >> (16 * k)));
          const float c = cp[2 * j + k], sn = sp[2 * j + k];
          l[k] = p * c - q2 * sn;
          g[k] = p * sn + q2 * c;
        }
        wl[j] = f2h(l[0]) | (f2h(l[1]) << 16);
        wh[j] = f2h(g[0]) | (f2h(g[1]) << 16);
      }
      uint16_t *to = A.qo + row * A.ldqo + (int64_t)h * A.D + d;
      *LB_LOOSE128(to) = wl;
      *LB_LOOSE128(to + half) = wh;
    }
    return;
  }
  const int hl = lane / groups, g = lane - hl * groups;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int h = (qp * 4 + i) * hpi + hl;
    const bool mine = hl < hpi && h < A.heads;
    float o[8];
    if (mine) turn8(A.q + row * A.ldq + (int64_t)h * A.D, g, A.D, cs, A.rot, A.inter, o);
    __builtin_amdgcn_wave_barrier();  // all lanes have read before any writes
    if (mine) {
      u32x4_t w;
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = f2h(o[2 * j]) | (f2h(o[2 * j + 1]) << 16);
      *LB_LOOSE128(A.qo + row * A.ldqo + (int64_t)h * A.D + 8 * g) = w;
    }
  }
}

// -------------------------------------------------------------- reading
struct ReadArgs {
  Sequences S;
  const uint8_t *kc, *vc;
  const float *ks, *vs;
  uint16_t *k, *v;
  int64_t ldk, ldv, items;
  int KV, D, Dp, lg;
};

// A wave has one unit of 16 tokens of one head, keys or values.  A lane has 8
// neighbouring dims of a token's key, but of values 4 tokens of single dims: those
// are put in order in LDS, 64 dims of all tokens at a time, and leave as 16 bytes a
// lane too (stored as single numbers: one token 5 us, not 4, a prompt of 4096 9).
// Bound by writing: 4096 tokens of 8 heads of 128, 25 MB, in 8 us; few tokens by the
// chain of loads.
__global__ void __launch_bounds__(256) k_cache_read(ReadArgs A) {
  __shared__ __align__(16) uint16_t order[4][16][72];  // (8 more than it needs keep rows on different banks)
  const Sequences &S = A.S;
  const unsigned block = blockIdx.x * 4 + wave_id();
  const unsigned item = block / (unsigned)(2 * A.KV);
  const int which = (int)(block - item * (2 * A.KV)), h = which >> 1, lane = threadIdx.x & 63;
  if (item >= A.items) return;
  int b = (int)item;
  int64_t first = item;
  if (S.start) b = find_sequence(S, item, 1, 4, 2, &first);
  if (b < 0) return;
  const Sequence q = sequence(S, b);
  int u, a, e;
  if (!touched(max(0, q.length - q.rows), q.length, 4, item - first, &u, &a, &e)) return;
  const int page = page_of(S, b, u >> (A.lg - 4));
  const bool there = page >= 0;  // otherwise the tokens read as zeros
  const int64_t block_of = (int64_t)(there ? page : 0) * A.KV + h;
  const bool values = which & 1;
  const float s = there ? (values ? A.vs : A.ks)[block_of] : 0.f;
  const uint8_t *from = (values ? A.vc : A.kc) + ((block_of << A.lg) + ((u & ((1 << (A.lg - 4)) - 1)) << 4)) * A.Dp;
  const int64_t row0 = row_of(q, u << 4);  // of the unit's first token
  const int pairs = A.Dp / 64, n = pairs + ((A.Dp / 32) & 1), G = lane >> 4, x = lane & 15;
  for (int c = 0; c < n; ++c) {
    u32x4_t w = {0, 0, 0, 0};
    if (c < pairs)
      w = *(const u32x4_t *)(from + c * 1024 + lane * 16);
    else
      *(u32x2_t *)&w = *(const u32x2_t *)(from + c * 1024 + lane * 8);
    const auto value = [&](int i) { return f2h((float)((int)((w[i >> 2] >> (8 * (i & 3))) & 255u) - 128) * s); };
    const int parts = c < pairs ? 2 : 1;
    if (values) {
      uint16_t(*tile)[72] = order[wave_id()];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i >= 2 * parts) break;
#pragma unroll
        for (int j = 0; j < 4; ++j) tile[4 * G + j][16 * i + x] = there ? (uint16_t)value(4 * i + j) : 0;
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      const int lg = parts + 1;  // groups of 8 dims a token: 8 or 4
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (i >= parts) break;
        const int t = (lane + 64 * i) >> lg, d = 8 * (lane & ((1 << lg) - 1));
        if (t >= a && t < e && 64 * c + d < A.D)
          *LB_LOOSE128(A.v + (row0 + t) * A.ldv + (int64_t)h * A.D + 64 * c + d) = *(const u32x4_t *)&tile[t][d];
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();  // before the next dims
    } else {
      if (x < a || x >= e) continue;
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int g = 8 * c + 4 * hh + G;
        if (hh >= parts || g * 8 >= A.D) continue;
        u32x4_t o;
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = there ? value(8 * hh + 2 * j) | (value(8 * hh + 2 * j + 1) << 16) : 0u;
        *LB_LOOSE128(A.k + (row0 + x) * A.ldk + (int64_t)h * A.D + 8 * g) = o;
      }
    }
  }
}

// ------------------------------------------------------------------ host
// Every number 0 and every scale 0: tokens that were never written read as 0.
__global__ void __launch_bounds__(256) k_cache_clear(uint8_t *k, uint8_t *v, int64_t pieces, float *ks, float *vs, int64_t n) {
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
  const u32x4_t zero = {0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u};
  for (int64_t i = at; i < pieces; i += step) ((u32x4_t *)k)[i] = ((u32x4_t *)v)[i] = zero;
  for (int64_t i = at; i < n; i += step) ks[i] = vs[i] = 0.f;
}

Rows strided(const void *p, int64_t rows, int64_t ld, int64_t width) {
  return {p, p ? rows : 0, (size_t)ld * 2, (size_t)width * 2};
}

// Memory of the call's own that must not be among what it writes.
bool meets_sequences(const Sequences &S, const Rows &w) {
  return (S.start && meet({S.start, 1, 0, (size_t)(S.n + 1) * 4}, w)) || meet({S.lengths, 1, 0, (size_t)S.n * 4}, w) ||
         meet({S.table, S.n, (size_t)S.ldt * 4, (size_t)S.columns * 4}, w);
}

}  // namespace

lb_status lbi::check_sequences(const lb_cache *C, const Sequences &S, const char *who) {
  const auto refuse = [who](const std::string &why) { return set_error(LB_EINVAL, std::string(who) + ": " + why); };
  if (S.n && (!S.lengths || !S.table)) return refuse("NULL lengths or table");
  if (!S.start && S.rows != S.n) return refuse("without start there is one row for each sequence");
  if (S.columns < 1 || (int64_t)S.columns * C->P > kMaxRows) return refuse("the table must hold 1 to 2^30 tokens");
  if (S.n > 1 && S.ldt < S.columns) return refuse("the table's row stride is smaller than its row");
  if (S.ldt > (int64_t)1 << 31) return refuse("the table's row stride exceeds 2^31");
  if (((uintptr_t)S.start | (uintptr_t)S.lengths | (uintptr_t)S.table) % 4) return refuse("misaligned pointer");
  return LB_OK;
}

extern "C" lb_status lb_cache_create(int64_t pages, int page_tokens, int kv_heads, int head_dim, lb_cache **out) {
  const auto refuse = [](const char *why) { return set_error(LB_EINVAL, std::string("lb_cache_create: ") + why); };
  if (!out) return refuse("out is NULL");
  if (page_tokens < 16 || page_tokens > 256 || (page_tokens & (page_tokens - 1)))
    return refuse("page_tokens must be a power of two from 16 to 256");
  if (kv_heads < 1 || kv_heads > 1024) return refuse("need 1 to 1024 key heads");
  if (head_dim < 8 || head_dim > 256 || head_dim % 8) return refuse("head_dim must be a multiple of 8 from 8 to 256");
  // units are numbered by 32-bit numbers
  if (pages < 1 || pages > ((int64_t)0x7fffffff) / kv_heads / (page_tokens / 16)) return refuse("too few or too many pages");
  lb_cache *C = nullptr;
  try {
    C = new lb_cache();
  } catch (...) {
    return set_error(LB_ENOMEM, "lb_cache_create: host allocation");
  }
  C->pages = pages;
  C->P = page_tokens;
  C->lg = __builtin_ctz((unsigned)page_tokens);
  C->KV = kv_heads;
  C->D = head_dim;
  C->Dp = (head_dim + 31) / 32 * 32;
  hipError_t e = hipGetDevice(&C->device);
  if (e == hipSuccess) e = hipDeviceGetAttribute(&C->cus, hipDeviceAttributeMultiprocessorCount, C->device);
  if (e != hipSuccess) {
    delete C;
    return set_error(LB_EHIP, std::string("lb_cache_create: ") + hipGetErrorString(e));
  }
  const size_t blocks = (size_t)pages * kv_heads, bytes = blocks * page_tokens * C->Dp;
  void **to[] = {(void **)&C->k, (void **)&C->v, (void **)&C->ks, (void **)&C->vs};
  for (int i = 0; i < 4 && e == hipSuccess; ++i) e = hipMalloc(to[i], i < 2 ? bytes : blocks * 4);
  if (e != hipSuccess) {
    lb_cache_destroy(C);
    return set_error(LB_ENOMEM, std::string("lb_cache_create: hipMalloc: ") + hipGetErrorString(e));
  }
  k_cache_clear<<<dim3((unsigned)std::min<size_t>((bytes / 16 + 255) / 256, 8192)), dim3(256), 0, nullptr>>>(
      C->k, C->v, (int64_t)(bytes / 16), C->ks, C->vs, (int64_t)blocks);
  e = hipGetLastError();
  if (e == hipSuccess) e = hipDeviceSynchronize();
  if (e != hipSuccess) {
    lb_cache_destroy(C);
    return set_error(LB_EHIP, std::string("lb_cache_create: ") + hipGetErrorString(e));
  }
  *out = C;
  return LB_OK;
}

extern "C" lb_status lb_cache_destroy(lb_cache *C) {
  if (!C) return LB_OK;
  DeviceGuard dg(C->device);
  for (void *p : {(void *)C->k, (void *)C->v, (void *)C->ks, (void *)C->vs, C->ws})
    if (p) (void)hipFree(p);
  for (void *p : C->retired) (void)hipFree(p);
  delete C;
  return LB_OK;
}

extern "C" lb_status lb_cache_shape(const lb_cache *C, int64_t *pages, int *page_tokens, int *kv_heads, int *head_dim,
                                    int *device) {
  if (!C) return set_error(LB_EINVAL, "lb_cache_shape: NULL cache");
  if (pages) *pages = C->pages;
  if (page_tokens) *page_tokens = C->P;
  if (kv_heads) *kv_heads = C->KV;
  if (head_dim) *head_dim = C->D;
  if (device) *device = C->device;
  return LB_OK;
}

extern "C" lb_status lb_cache_append(lb_cache *C, const void *k, int64_t ldk, const void *v, int64_t ldv, const void *q,
                                     int64_t ldq, void *q_out, int64_t ldqo, int heads, const float *rope,
                                     int64_t positions, int rot, int interleaved, const int32_t *start,
                                     const int32_t *lengths, const int32_t *table, int64_t ldt, int columns,
                                     int sequences, int64_t rows, void *stream) {
  const auto refuse = [](const char *why) { return set_error(LB_EINVAL, std::string("lb_cache_append: ") + why); };
  if (!C) return refuse("NULL cache");
  if (rows < 0 || rows > kMaxRows || sequences < 0 || sequences > kMaxRows)
    return refuse("rows and sequences must be in [0, 2^30]");
  if (rows == 0) return LB_OK;
  const Sequences S = {start, lengths, table, ldt, sequences, (int)rows, columns, (int)C->pages};
  const lb_status st = check_sequences(C, S, "lb_cache_append");
  if (st != LB_OK) return st;
  if (!k || !v) return refuse("NULL k or v");
  if (!q != !q_out) return refuse("q and q_out go together");
  if (q && (heads < 1 || heads > 65536)) return refuse("need 1 to 65536 heads of q");
  if (rot < 0 || rot > C->D || rot % 2) return refuse("rot must be even and at most head_dim");
  if (rot && !rope) return refuse("NULL rope");
  if (rot && positions < (int64_t)columns * C->P) return refuse("rope needs a row for every token that the table can hold");
  const int64_t kw = (int64_t)C->KV * C->D, qw = (int64_t)heads * C->D, most = (int64_t)1 << 31;
  if (ldk < kw || ldv < kw || (q && (ldq < qw || ldqo < qw))) return refuse("a row stride is smaller than the row");
  if (ldk > most || ldv > most || (q && (ldq > most || ldqo > most))) return refuse("a row stride exceeds 2^31");
  if (((uintptr_t)k | (uintptr_t)v | (uintptr_t)q | (uintptr_t)q_out) % 2 || (uintptr_t)rope % 4)
    return refuse("misaligned pointer");
  if (q) {
    const Rows w = strided(q_out, rows, ldqo, qw);
    if (!(q == q_out && ldq == ldqo) && meet(strided(q, rows, ldq, qw), w))
      return refuse("q and q_out overlap (they may be the same rows)");
    if (meet(strided(k, rows, ldk, kw), w) || meet(strided(v, rows, ldv, kw), w)) return refuse("k or v and q_out overlap");
    if ((rot && meet({rope, 1, 0, (size_t)positions * rot * 4}, w)) || meets_sequences(S, w))
      return refuse("an input and q_out overlap");
  }
  if (sequences == 0) return LB_OK;
  AppendArgs A = {};
  A.S = S;
  A.k = (const uint16_t *)k;
  A.v = (const uint16_t *)v;
  A.q = (const uint16_t *)q;
  A.qo = (uint16_t *)q_out;
  A.ldk = ldk; A.ldv = ldv; A.ldq = ldq; A.ldqo = ldqo;
  A.rope = rope;
  A.kc = C->k; A.vc = C->v; A.ks = C->ks; A.vs = C->vs;
  A.heads = heads; A.KV = C->KV; A.D = C->D; A.Dp = C->Dp; A.P = C->P; A.lg = C->lg;
  A.rot = rot;
  A.inter = interleaved != 0;
  // sequence b begins a new page at most every P rows, and touches one more at each end
  A.items = start ? (rows >> C->lg) + 2 * (int64_t)sequences : sequences;
  const bool single = rows <= 2 * (int64_t)sequences;
  const int64_t blocks = A.items * 2 * C->KV;
  A.kvwgs = single ? (blocks + 3) / 4 : blocks;
  A.both = rot == C->D && rot % 16 == 0 && !interleaved;
  const int per_wave = A.both ? 2 * (64 / (C->D / 16)) : 4 * (64 / (C->D / 8));  // heads
  A.qparts = q ? (heads + per_wave - 1) / per_wave : 0;
  const int64_t qwgs = (rows * A.qparts + 3) / 4;
  if (A.kvwgs + qwgs > 0x7fffffff / 256 || blocks > 0x7fffffff)
    return set_error(LB_EUNSUPPORTED, "lb_cache_append: too many rows and heads for one call");
  DeviceGuard dg(C->device);
  const dim3 grid((unsigned)(A.kvwgs + qwgs));
  if (single)
    k_cache_append<64><<<grid, dim3(256), 0, (hipStream_t)stream>>>(A);
  else
    k_cache_append<256><<<grid, dim3(256), 0, (hipStream_t)stream>>>(A);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return set_error(LB_EHIP, std::string("lb_cache_append: ") + hipGetErrorString(e));
  return LB_OK;
}

extern "C" lb_status lb_cache_read(const lb_cache *C, void *k, int64_t ldk, void *v, int64_t ldv, const int32_t *start,
                                   const int32_t *lengths, const int32_t *table, int64_t ldt, int columns,
                                   int sequences, int64_t rows, void *stream) {
  const auto refuse = [](const char *why) { return set_error(LB_EINVAL, std::string("lb_cache_read: ") + why); };
  if (!C) return refuse("NULL cache");
  if (rows < 0 || rows > kMaxRows || sequences < 0 || sequences > kMaxRows)
    return refuse("rows and sequences must be in [0, 2^30]");
  if (rows == 0) return LB_OK;
  const Sequences S = {start, lengths, table, ldt, sequences, (int)rows, columns, (int)C->pages};
  const lb_status st = check_sequences(C, S, "lb_cache_read");
  if (st != LB_OK) return st;
  if (!k || !v) return refuse("NULL k or v");
  const int64_t kw = (int64_t)C->KV * C->D, most = (int64_t)1 << 31;
  if (ldk < kw || ldv < kw) return refuse("a row stride is smaller than the row");
  if (ldk > most || ldv > most) return refuse("a row stride exceeds 2^31");
  if (((uintptr_t)k | (uintptr_t)v) % 2) return refuse("misaligned pointer");
  const Rows kr = strided(k, rows, ldk, kw), vr = strided(v, rows, ldv, kw);
  if (meet(kr, vr)) return refuse("k and v overlap");
  if (meets_sequences(S, kr) || meets_sequences(S, vr)) return refuse("an input and k or v overlap");
  if (sequences == 0) return LB_OK;
  ReadArgs A = {};
  A.S = S;
  A.kc = C->k; A.vc = C->v; A.ks = C->ks; A.vs = C->vs;
  A.k = (uint16_t *)k;
  A.v = (uint16_t *)v;
  A.ldk = ldk; A.ldv = ldv;
  A.items = start ? (rows >> 4) + 2 * (int64_t)sequences : sequences;
  A.KV = C->KV; A.D = C->D; A.Dp = C->Dp; A.lg = C->lg;
  const int64_t blocks = A.items * 2 * C->KV;
  if (blocks > (int64_t)0x7fffffff / 64) return set_error(LB_EUNSUPPORTED, "lb_cache_read: too many rows and heads for one call");
  DeviceGuard dg(C->device);
  k_cache_read<<<dim3((unsigned)((blocks + 3) / 4)), dim3(256), 0, (hipStream_t)stream>>>(A);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return set_error(LB_EHIP, std::string("lb_cache_read: ") + hipGetErrorString(e));
  return LB_OK;
}
