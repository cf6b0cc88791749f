// Attention over the paged 8-bit cache (lb_cache.h): lb_cache_attend.
//
// For a row (token i of a sequence, query head h, key head h / group) at
// position p = length - rows + i, over the keys t it sees (t < length; t <= p
// when causal; t > p - window with a window):
//
//   z_t = scale * s_k(t) * (q . K_t)        K, V: the bytes - 128, exact in fp16
//   out = sum_t e^(z_t - m) s_v(t) V_t / sum_t e^(z_t - m)
//
// in one pass over the keys with a running reference m and sum l: when the
// largest z so far exceeds m by more than kSlack (in powers of two), m is set to
// it and what has been summed is scaled down; in between the weights may
// exceed 1, which costs nothing and saves most of the scaling.
//
// Precision.  q . K is exact products in fp32 sums.  The weight times s_v has
// to be an fp16 operand: s_v / r, r the largest finite s_v so far (a change of
// r scales the sums too), keeps it within 2^(kUp + kSlack), and 2^kUp lifts it
// over fp16's small numbers.  The kernel for few rows, bound by reading the
// keys, keeps it as two fp16 numbers (22 bits), which leaves the scores' fp32
// roundings as the larger ones.  The one for many rows, bound by matrix and vector
// instructions, keeps one (off by up to 2^-11, the half step of out as well).  l is
// summed in fp32 from the weights before any rounding.
// Keys that a row does not see get weight 0 by selection, so that what lies
// there (numbers of earlier owners, scales that are NaN) does not reach it.  A
// finite s_v that its wave meets there may become r, 2^-37 of which is the finest
// step of a weight times s_v (5e-7 for a page of 65504, 8 of fp16's smallest steps).
//
// Both kernels work on S^T = K Q^T and O^T = V^T P^T: a lane has one row of q
// (column of S^T), its maximum and sum are the lane's own up to one or two
// exchanges, and the weights come out of the first product in the order in
// which the second wants them.
//
// A row's keys may be split over workgroups (pieces of `chunk` keys): each
// leaves its m, l and sums in the workspace, and k_attend_join adds them up.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "lb_cache.h"

namespace {

using namespace lbi;

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float float2_t __attribute__((ext_vector_type(2)));
typedef float float4_t __attribute__((ext_vector_type(4)));
typedef float float16_t __attribute__((ext_vector_type(16)));
typedef float4_t __attribute__((aligned(8))) float4a_t;

constexpr int64_t kMaxRows = (int64_t)1 << 30;
constexpr float kUp = 12.f, kSlack = 3.f;
// The reference before there is one, below every score: e^(-inf - kNothing) is 0,
// and so is the share of what has seen nothing in a sum with what has.
constexpr float kNothing = -1e30f;
// Of k_attend_many: the scale of a page that is not there, and the smallest
// reference of the values' scales (all are above 2^-32).
constexpr float kMissing = -1e9f, kLeast = -100.f;
constexpr int kFewWaves = 8;   // of a workgroup of k_attend_few
constexpr int kJoinHere = 64;  // pieces up to which the last workgroup of k_attend_few to arrive joins them
// LDS of k_attend_few: the waves' sums, or the weights of the pieces.
__host__ __device__ constexpr int few_floats(int rows, int Dp, int waves) {
  return waves * rows * (Dp + 4) > 2 * kJoinHere * 16 ? waves * rows * (Dp + 4) : 2 * kJoinHere * 16;
}
constexpr int kJoinShort = 8;  // pieces up to which k_attend_join_short joins them
constexpr int kJoinRows = 32;  // rows that a workgroup of it has

struct AttendArgs {
  Sequences S;
  const uint16_t *q;
  uint16_t *out;
  int64_t ldq, ldo;
  const uint8_t *kc, *vc;
  const float *ks, *vs;
  // partial sums of the pieces, of each kernel: per item and piece rows x Dp sums,
  // then m and l of each row
  float *few_part, *part;
  unsigned *count;  // arrivals at each item of k_attend_few, 0 between launches; NULL: k_attend_join does it
  float qscale;  // scale * log2 e
  int KV, D, lg;
  View view;
  int few;      // rows x heads of a group up to which k_attend_few has a sequence
  int tiles, frows;  // 16-row tiles a sequence may have there, rows of a tile (16 or fewer)
  int few_chunk, few_pieces;  // keys of a piece, pieces in the grid
  int chunk, pieces;          // the same of k_attend_many
  int row_tiles;      // k_attend_many: row tiles in the grid
  int b0;             // k_attend_few: first sequence of the grid
  unsigned blocks;    // k_attend_many: workgroups with many rows; those behind them have few
};

// What an item (a sequence's row tile of one key head) sees.
struct Item {
  Sequence q;
  int h, r0, n;    // key head, first row (token * group + head), rows
  int lo, hi;      // keys, lo a multiple of 16
};

// Four bytes as fp16 numbers: byte - 128, exact (0x6400 + byte is 1024 + byte).
__device__ __forceinline__ void to_half4(uint32_t w, half2_t &a, half2_t &b) {
  const half2_t bias = {(_Float16)-1152.f, (_Float16)-1152.f};
  a = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0x64646464u, w, 0x04010400u)) + bias;
  b = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0x64646464u, w, 0x04030402u)) + bias;
}
__device__ __forceinline__ half8_t to_half8(uint32_t w0, uint32_t w1) {
  half2_t a, b, c, d;
  to_half4(w0, a, b);
  to_half4(w1, c, d);
  return half8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ float lane_xor(float v, int d) { return __shfl_xor(v, d); }
// The values of lanes 16 and 32 away, without a trip through LDS.
__device__ __forceinline__ float other16(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(threadIdx.x & 16 ? r[0] : r[1]);
}
__device__ __forceinline__ float max32(float v) {  // of a lane and that one
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float max16(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float other32(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(threadIdx.x & 32 ? r[0] : r[1]);
}

// Item of k_attend_few: 16-row tile `tile` of sequence b's rows of key head h, or
// false.  Items are numbered (b KV + h) tiles + tile.
__device__ __forceinline__ bool few_item(const AttendArgs &A, int b, int h, int tile, Item &it) {
  it.h = h;
  it.q = sequence(A.S, b);
  const int64_t rows = (int64_t)it.q.rows * A.view.group;
  if (rows > A.few) return false;
  it.r0 = tile * 16;
  if (it.r0 >= rows) return false;
  it.n = min(16, (int)rows - it.r0);
  keys_of_rows(A.view, it.q, it.r0, it.n, &it.lo, &it.hi);
  return true;
}

// Item of k_attend_many: row tile `slot` of all sequences' tiles of TR rows, head h.
template <int TR>
__device__ __forceinline__ bool many_item(const AttendArgs &A, int slot, int h, Item &it, int *b_out) {
  constexpr int lg = TR == 256 ? 8 : 7;
  static_assert(TR == 1 << lg, "a power of two");
  int64_t first;
  const int b = find_sequence(A.S, slot, A.view.group, lg, 1, &first);
  if (b < 0) return false;
  it.q = sequence(A.S, b);
  const int64_t rows = (int64_t)it.q.rows * A.view.group, r0 = (slot - first) * TR;
  if (rows <= A.few || r0 >= rows) return false;
  it.h = h;
  it.r0 = (int)r0;
  it.n = (int)min((int64_t)TR, rows - r0);
  keys_of_rows(A.view, it.q, it.r0, it.n, &it.lo, &it.hi);
  *b_out = b;
  return true;
}

// The address of row r of a head's group, in q or out.
__device__ __forceinline__ int64_t row_at(const AttendArgs &A, const Item &it, int r, int64_t ld) {
  const int tok = r / A.view.group, j = r - tok * A.view.group;
  return (int64_t)(it.q.row0 + tok) * ld + (int64_t)(it.h * A.view.group + j) * A.D;
}

// Infinities become NaN: the row's softmax is NaN either way, but scores of -inf alone
// would look like those of a row that sees nothing.
__device__ __forceinline__ half8_t load_q(const AttendArgs &A, int64_t at, int d) {
  u32x4_t w = {0, 0, 0, 0};
  if (d < A.D) w = *LB_LOOSE128(A.q + at + d);
  const half8_t q = __builtin_bit_cast(half8_t, w);
  return q + q * (_Float16)0.f;
}

// Four of a row's outputs, from its sum and weights.
__device__ __forceinline__ void write4(const AttendArgs &A, const Item &it, int row, int d, float4_t o, float L) {
  if (d >= A.D) return;
  const float inv = L > 0.f || L != L ? 1.f / L : 0.f;
  u32x2_t h;
  h[0] = f2h(o[0] * inv) | (f2h(o[1] * inv) << 16);
  h[1] = f2h(o[2] * inv) | (f2h(o[3] * inv) << 16);
  typedef u32x2_t __attribute__((aligned(2), address_space(1))) loose64;
  *(loose64 *)(uintptr_t)(A.out + row_at(A, it, it.r0 + row, A.ldo) + d) = h;
}

// Numbers for and from workgroups elsewhere on the GPU: past this CU's and XCD's caches.
__device__ __forceinline__ void store2(float *p, float a, float b) {
  __hip_atomic_store((unsigned long long *)p, __builtin_bit_cast(unsigned long long, float2_t{a, b}), __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float2_t load2(const float *p) {
  return __builtin_bit_cast(float2_t, __hip_atomic_load((unsigned long long *)p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
}
__device__ __forceinline__ void store4(float *p, float4_t v) {
  store2(p, v[0], v[1]);
  store2(p + 2, v[2], v[3]);
}
__device__ __forceinline__ float4_t load4(const float *p) {
  const float2_t a = load2(p), b = load2(p + 2);
  return float4_t{a[0], a[1], b[0], b[1]};
}

// ------------------------------------------------------------- few rows
// 16 rows a workgroup, whose waves share out the keys of a piece and read them
// from memory straight into operands; the waves' sums are joined in LDS.  A step of
// a wave is 32 keys: their scores, weights and values while the next 32 are on
// their way.  Bound by reading where there are keys enough (131072 keys of 8 heads
// of 128, 64 query heads: 268 MB in 55 us, 4.9 TB/s), by latency where there are few
// (512 keys of 32 heads 7.6 us), and between them by vector instructions, of which
// the bytes' conversion to fp16 is nearly half: 64 sequences of 256 to 4096 keys take
// 48 us, 191 MB at 4.0 TB/s.  Eight waves in 128 registers, two workgroups a CU (four
// waves with more registers took 64 us for 131072 keys and 107 for 128 sequences, these
// 63 and 96 at that time).
// Row tile `tile` of key head h of sequence b, one piece of its keys, by W waves.
template <int NC, int W>
__device__ __forceinline__ void few_rows(const AttendArgs &A, int b, int h, int tile, int piece, float *sh) {
  constexpr int Dp = NC * 32, kPairs = NC / 2, kOdd = NC & 1, kUnit = Dp * 16, NT = Dp / 16;
  // sh: [waves][rows][Dp + 4], then m and l [waves][16] each
  const int lane = threadIdx.x & 63, w = wave_id(), n = lane & 15, G = lane >> 4;
  const int upp = 1 << (A.lg - 4);
  // Wave w has pairs of units w, w + W, ... of the piece.  Up to 32 pairs a
  // time: lane i looks up the page of one unit.  The first look-up waits for the
  // lengths only where a window moves the piece (its column is clamped to the table).
  const auto unit_at = [&](int c0, int batch) { return (c0 >> 4) + 2 * (w + W * (batch * 32 + (lane >> 1))) + (lane & 1); };
  const auto look_up = [&](int u) { return A.S.table[b * A.S.ldt + min(u >> (A.lg - 4), A.S.columns - 1)]; };
  int page = A.view.window ? -1 : look_up(unit_at(piece * A.few_chunk, 0));
  Item it;
  if (!few_item(A, b, h, tile, it)) return;
  const int pieces = pieces_of(it.lo, it.hi, A.few_chunk);
  if (piece >= pieces) return;
  const int64_t slot = ((int64_t)b * A.KV + h) * A.tiles + tile;
  const int c0 = it.lo + piece * A.few_chunk, c1 = min(it.hi, c0 + A.few_chunk);
  if (A.view.window) page = look_up(unit_at(c0, 0));
  const int all_pairs = (c1 - c0 + 31) >> 5, pairs = max(0, (all_pairs - w + W - 1) / W);  // the wave's
  const int myrow = it.r0 + min(n, it.n - 1);
  int first, last;
  keys_of_row(A.view, it.q, myrow, &first, &last);
  last = min(last, c1);
  int all_first, all_last;  // the keys that all rows see
  {
    int unused;
    keys_of_row(A.view, it.q, it.r0, &unused, &all_last);
    keys_of_row(A.view, it.q, it.r0 + it.n - 1, &all_first, &unused);
    all_first = __builtin_amdgcn_readfirstlane(all_first);
    all_last = __builtin_amdgcn_readfirstlane(min(all_last, c1));
  }

  half8_t q[NC];
  {
    const int64_t at = row_at(A, it, myrow, A.ldq);
#pragma unroll
    for (int s = 0; s < NC; ++s) q[s] = load_q(A, at, 32 * s + 8 * G);
  }
  float4_t O[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) O[i] = float4_t{0.f, 0.f, 0.f, 0.f};
  float m = kNothing, l = 0.f, r = 1e-30f;

  struct Frag {
    u32x4_t pair[kPairs > 0 ? kPairs : 1];
    u32x2_t odd;
  };
  const auto load = [&](const uint8_t *base, int unit, Frag &f) {
    const uint8_t *p = base + (int64_t)unit * kUnit;
#pragma unroll
    for (int c = 0; c < kPairs; ++c)
      f.pair[c] = *(const u32x4_t __attribute__((address_space(1))) *)(uintptr_t)(p + c * 1024 + lane * 16);
    if constexpr (kOdd)
      f.odd = *(const u32x2_t __attribute__((address_space(1))) *)(uintptr_t)(p + kPairs * 1024 + lane * 8);
  };

  for (int batch = 0; batch * 32 < pairs; ++batch) {
    // lane i: where its unit lies, and its scales
    const int u = unit_at(c0, batch);
    if (batch) page = look_up(u);
    const bool there = u * 16 < c1 && page >= 0 && page < A.S.pages;
    const int blk = (there ? page : 0) * A.KV + it.h;
    const int mine = blk * upp + (u & (upp - 1));
    const float ks = there ? A.ks[blk] * A.qscale : 0.f, vs = there ? A.vs[blk] : 0.f;
    const unsigned long long ok = __ballot(there);
    const int steps = min(32, pairs - batch * 32);
    Frag K[2], V[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) load(A.kc, __builtin_amdgcn_readlane(mine, i), K[i]);
#pragma unroll
    for (int i = 0; i < 2; ++i) load(A.vc, __builtin_amdgcn_readlane(mine, i), V[i]);
    float big = vs < INFINITY ? vs : 0.f;
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) big = fmaxf(big, lane_xor(big, d));
    if (big > r) {
      const float f = r / big;
#pragma unroll
      for (int i = 0; i < NT; ++i) O[i] *= f;
      r = big;
    }
    const float ratio = vs / r;
    for (int st = 0; st < steps; ++st) {
      // the next step's units, this one's again behind the last
      const int n0 = __builtin_amdgcn_readlane(mine, min(2 * st + 2, 2 * steps - 2));
      const int n1 = __builtin_amdgcn_readlane(mine, min(2 * st + 3, 2 * steps - 1));
      const int t0 = c0 + 32 * (w + W * (batch * 32 + st));
      const unsigned both = (unsigned)(ok >> (2 * st)) & 3u;
      const bool usual = both == 3u && t0 >= all_first && t0 + 32 <= all_last;
      float4_t z[2];
      float factor[2], top = -INFINITY;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < kPairs; ++c) {
          acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(to_half8(K[i].pair[c][0], K[i].pair[c][1]), q[2 * c], acc, 0, 0, 0);
          acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(to_half8(K[i].pair[c][2], K[i].pair[c][3]), q[2 * c + 1], acc, 0, 0, 0);
        }
        if constexpr (kOdd)
          acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(to_half8(K[i].odd[0], K[i].odd[1]), q[NC - 1], acc, 0, 0, 0);
        load(A.kc, i ? n1 : n0, K[i]);
        factor[i] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(ks), 2 * st + i));
        z[i] = acc;
      }
      if (usual) {  // the scale (not negative) goes into the exponent's multiply-add
#pragma unroll
        for (int i = 0; i < 2; ++i)
          top = fmaxf(top, fmaxf(fmaxf(z[i][0], z[i][1]), fmaxf(z[i][2], z[i][3])) * factor[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int t = t0 + 16 * i + 4 * G + j;
            const bool in = ((both >> i) & 1u) && t >= first && t < last;
            z[i][j] = in ? z[i][j] * factor[i] : -INFINITY;
            top = fmaxf(top, z[i][j]);
          }
          factor[i] = 1.f;
        }
      }
      top = max32(max16(top));
      const bool up = top > m + kSlack;
      if (__any(up)) {
        const float f = up ? exp2f(m - top) : 1.f;
        l *= f;
#pragma unroll
        for (int i = 0; i < NT; ++i) O[i] *= f;
        if (up) m = top;
      }
      const float ref = m - kUp;
      half8_t ph, pl;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float f = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(ratio), 2 * st + i));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float p = __builtin_amdgcn_exp2f(fmaf(z[i][j], factor[i], -ref));
          l += p;
          const float pv = usual || z[i][j] != -INFINITY ? p * f : 0.f;
          const _Float16 hi = (_Float16)pv;
          ph[4 * i + j] = hi;
          pl[4 * i + j] = (_Float16)(pv - (float)hi);
        }
      }
#pragma unroll
      for (int c = 0; c < kPairs; ++c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const half8_t a = to_half8(V[0].pair[c][i], V[1].pair[c][i]);
          O[4 * c + i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, ph, O[4 * c + i], 0, 0, 0);
          O[4 * c + i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, pl, O[4 * c + i], 0, 0, 0);
        }
      }
      if constexpr (kOdd) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const half8_t a = to_half8(V[0].odd[i], V[1].odd[i]);
          O[4 * kPairs + i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, ph, O[4 * kPairs + i], 0, 0, 0);
          O[4 * kPairs + i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, pl, O[4 * kPairs + i], 0, 0, 0);
        }
      }
      load(A.vc, n0, V[0]);
      load(A.vc, n1, V[1]);
    }
  }
  l += other16(l);
  l += other32(l);

  // the waves' sums, in units of 1
  constexpr int kPitch = Dp + 4;
  const int rows = A.frows;
  float *sm = sh + few_floats(rows, Dp, W), *sl = sm + 16 * W;
  if (n < it.n) {
#pragma unroll
    for (int i = 0; i < NT; ++i) *(float4_t *)(sh + (w * rows + n) * kPitch + 16 * i + 4 * G) = O[i] * r;
  }
  if (G == 0) {
    sm[w * 16 + n] = m;
    sl[w * 16 + n] = l;
  }
  __syncthreads();
  float *part = A.few_part + (slot * A.few_pieces + piece) * rows * (Dp + 2);
  for (int i = threadIdx.x; i < it.n * (Dp / 4); i += W * 64) {
    const int row = i / (Dp / 4), d = (i - row * (Dp / 4)) * 4;
    float M = sm[row];
#pragma unroll
    for (int v = 1; v < W; ++v) M = fmaxf(M, sm[v * 16 + row]);
    float4_t o = {0.f, 0.f, 0.f, 0.f};
    float L = 0.f;
#pragma unroll
    for (int v = 0; v < W; ++v) {
      const float f = __builtin_amdgcn_exp2f(sm[v * 16 + row] - M);
      o += *(const float4_t *)(sh + (v * rows + row) * kPitch + d) * f;
      L += sl[v * 16 + row] * f;
    }
    if (pieces == 1)
      write4(A, it, row, d, o, L);
    else if (A.count) {
      store4(part + row * Dp + d, o);
      if (d == 0) store2(part + rows * Dp + 2 * row, M, L);
    } else {
      *(float4a_t *)(part + row * Dp + d) = o;
      if (d == 0) *(float2_t *)(part + rows * Dp + 2 * row) = float2_t{M, L};
    }
  }
  if (pieces == 1 || !A.count) return;

  // The item's last workgroup to arrive joins its pieces (with a launch for that 64
  // sequences took 65 us, not 59).  Partial sums go past the caches, every wave's before
  // the workgroup counts itself, and are read the same way.  That order is the hardware's
  // (a store past the caches has arrived when its wait ends), not the memory model's,
  // whose release would write the whole L2 back.
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  int *flag = (int *)(sl + 16 * W);
  if (threadIdx.x == 0) {
    const unsigned before = __hip_atomic_fetch_add(A.count + slot, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *flag = before == (unsigned)pieces - 1;
    if (*flag) __hip_atomic_store(A.count + slot, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  if (!*flag) return;
  const int64_t size = (int64_t)rows * (Dp + 2);
  const float *all = A.few_part + slot * A.few_pieces * size;
  float *wm = sh, *wl = sh + kJoinHere * 16;  // [piece][16]; the sums of the waves are no longer needed
  for (int i = threadIdx.x; i < pieces * 16; i += W * 64) {
    const int row = i & 15;
    float2_t ml = {kNothing, 0.f};
    if (row < it.n) ml = load2(all + (i >> 4) * size + rows * Dp + 2 * row);
    wm[i] = ml[0];
    wl[i] = ml[1];
  }
  __syncthreads();
  {
    constexpr int kLanes = W * 4;  // of a row
    const int row = threadIdx.x / kLanes, p0 = threadIdx.x % kLanes;
    float M = kNothing, L = 0.f;
    for (int p = p0; p < pieces; p += kLanes) M = fmaxf(M, wm[p * 16 + row]);
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1) M = fmaxf(M, lane_xor(M, d));
    for (int p = p0; p < pieces; p += kLanes) {
      const float f = __builtin_amdgcn_exp2f(wm[p * 16 + row] - M);
      wm[p * 16 + row] = f;
      L += wl[p * 16 + row] * f;
    }
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1) L += lane_xor(L, d);
    if (p0 == 0) wl[row] = L;  // (piece 0's, read by this row's threads alone, before)
  }
  __syncthreads();
  for (int i = threadIdx.x; i < it.n * (Dp / 4); i += W * 64) {
    const int row = i / (Dp / 4), d = (i - row * (Dp / 4)) * 4;
    const float *from = all + row * Dp + d;
    float4_t o = {0.f, 0.f, 0.f, 0.f};
    int p = 0;
    for (; p + 7 < pieces; p += 8) {
      float4_t v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = load4(from + (p + j) * size);
#pragma unroll
      for (int j = 0; j < 8; ++j) o += v[j] * wm[(p + j) * 16 + row];
    }
    for (; p < pieces; ++p) o += load4(from + p * size) * wm[p * 16 + row];
    write4(A, it, row, d, o, wl[row]);
  }
}

template <int NC>
__global__ void __launch_bounds__(kFewWaves * 64, NC <= 4 ? 4 : 2) k_attend_few(AttendArgs A) {
  extern __shared__ char smem[];
  const unsigned h = A.tiles == 1 ? blockIdx.x : blockIdx.x / (unsigned)A.tiles;
  few_rows<NC, kFewWaves>(A, A.b0 + (int)blockIdx.y, (int)h, (int)(blockIdx.x - h * A.tiles), (int)blockIdx.z, (float *)smem);
}

// Nothing but an order: v is computed before what comes after.  (No
// instruction reads it here, so a matrix instruction's result needs no wait.)
// ACC: it lies in an accumulation register, and stays there.
template <bool ACC = false, typename T>
__device__ __forceinline__ void here(const T &v) {
#if defined(__HIP_DEVICE_COMPILE__)
  if constexpr (ACC)
    asm volatile("" ::"a"(v));
  else
    asm volatile("" ::"v"(v));
#endif
}

// ------------------------------------------------------------ many rows
// 32 rows a wave, NW waves a workgroup; tiles of 64 keys and values go through
// LDS as fp16 operands (converted once for all waves), the bytes of a later tile
// on their way meanwhile.  A step weighs and adds up half a tile, h (exponentials,
// then the second product), while the matrix cores have the first product of half
// h + 1.  Between two barriers (tile t) the waves read keys of halves 2 t + 1 and
// 2 t + 2 and values of halves 2 t and 2 t + 1, and write keys of the two halves
// behind and values of tile t + 1: there is room for four halves of keys and two
// tiles of values, so nothing is written that a slower wave may still read.  Half 0,
// which is read before all of that, has a barrier of its own (walk_tiles).
//
// Bound by vector instructions beside the matrix instructions.  A prompt of 4096 of
// 32 heads of 128 takes 180 us (137 GFLOP, 763 TFLOP/s; all keys for all rows 326 us,
// 833; a large library product reaches 1200).  Steps on the way there: 249 us with a
// tile's scores, weights and sums one after the other, 195 with the next tile's scores
// made meanwhile, 182 in halves with exponentials between the matrix instructions and
// operands read four of those ahead.  16 heads: 160 wide 203 us, 192 234, 256 271.
template <int NC, int NW>
__device__ __forceinline__ void many_rows(const AttendArgs &A, char *smem) {
  constexpr int Dp = NC * 32, kPairs = NC / 2, kOdd = NC & 1, kUnit = Dp * 16, NT = NC, TR = NW * 32;
  constexpr int kHalf = Dp * 128;  // bytes of a tile's keys, or values
  // smem: [4] halves of keys, [2] tiles of values, then scales: of keys [8][2] (read
  // a step after the keys themselves), of values [2][4]
  float *scales = (float *)(smem + 4 * kHalf);
  const int lane = threadIdx.x & 63, w = wave_id(), n = lane & 31, G = lane >> 5;
  // heads vary fastest, so that one head's tiles mostly meet on one XCD; the
  // last row tiles, which see the most keys, go first
  const unsigned hs = blockIdx.x / (unsigned)A.KV;
  const int h = (int)(blockIdx.x - hs * A.KV);
  const unsigned ts = hs / (unsigned)A.pieces;
  const int piece = (int)(hs - ts * A.pieces), slot = A.row_tiles - 1 - (int)ts;
  Item it;
  int b = 0;
  if (!many_item<TR>(A, slot, h, it, &b)) return;
  const int pieces = pieces_of(it.lo, it.hi, A.chunk);
  if (piece >= pieces) return;
  const int c0 = it.lo + piece * A.chunk, c1 = min(it.hi, c0 + A.chunk);
  const int tiles = (c1 - c0 + 63) >> 6;
  const int myrow = it.r0 + min(w * 32 + n, it.n - 1);
  int first, last;
  keys_of_row(A.view, it.q, myrow, &first, &last);
  last = min(last, c1);
  // over the wave: the keys that some row sees, and those that all see
  int some_last, all_first, all_last, some_first;
  {
    const int ra = it.r0 + min(w * 32, it.n - 1), rb = it.r0 + min(w * 32 + 31, it.n - 1);
    keys_of_row(A.view, it.q, ra, &some_first, &all_last);
    keys_of_row(A.view, it.q, rb, &all_first, &some_last);
    some_first = __builtin_amdgcn_readfirstlane(some_first);
    all_first = __builtin_amdgcn_readfirstlane(all_first);
    all_last = __builtin_amdgcn_readfirstlane(min(all_last, c1));
    some_last = __builtin_amdgcn_readfirstlane(min(some_last, c1));
  }
  half8_t q[Dp / 16];
  {
    const int64_t at = row_at(A, it, myrow, A.ldq);
#pragma unroll
    for (int s = 0; s < Dp / 16; ++s) q[s] = load_q(A, at, 16 * s + 8 * G);
  }
  float16_t O[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) O[i][j] = 0.f;
  float m = kNothing, l = 0.f, lr = kLeast;

  // staging: NW = 8: waves 0..3 have the tile's units of keys, 4..7 of values;
  // NW = 4: wave w has unit w of both
  constexpr int kKinds = NW == 8 ? 1 : 2;
  const int su = w & 3;
  struct Frag {
    u32x4_t pair[kPairs > 0 ? kPairs : 1];
    u32x2_t odd;
    float scale;
  };
  Frag f[kKinds];
  const auto is_values = [&](int i) { return NW == 8 ? w >= 4 : i == 1; };
  // Requests tile `tile` of values and halves 2 tile + 1, 2 tile + 2 of keys; their pages
  // were looked up a step before (a look-up and its wait in the same step took a
  // tenth of the step).
  const int *table = A.S.table + b * A.S.ldt;
  const int upp = 1 << (A.lg - 4);
  const auto look_up = [&](int tile, int (&page)[kKinds]) {
#pragma unroll
    for (int i = 0; i < kKinds; ++i) {
      const int tok = c0 + tile * 64 + (is_values(i) ? 0 : 32) + su * 16;
      page[i] = -1;
      if (tok >= c0 && tok < c1) page[i] = table[tok >> A.lg];  // c1 is inside the table
    }
  };
  const auto fetch = [&](int tile, const int (&page)[kKinds]) {
#pragma unroll
    for (int i = 0; i < kKinds; ++i) {
      const bool values = is_values(i);
      const int tok = c0 + tile * 64 + (values ? 0 : 32) + su * 16;
      const bool there = page[i] >= 0 && page[i] < A.S.pages;
      const int blk = (there ? page[i] : 0) * A.KV + it.h;
      const int unit = blk * upp + ((tok >> 4) & (upp - 1));
      const uint8_t *p = (values ? A.vc : A.kc) + (int64_t)unit * kUnit;
#pragma unroll
      for (int c = 0; c < kPairs; ++c)
        f[i].pair[c] = *(const u32x4_t __attribute__((address_space(1))) *)(uintptr_t)(p + c * 1024 + lane * 16);
      if constexpr (kOdd)
        f[i].odd = *(const u32x2_t __attribute__((address_space(1))) *)(uintptr_t)(p + kPairs * 1024 + lane * 8);
      f[i].scale = (values ? A.vs : A.ks)[blk];
      if (!there) f[i].scale = kMissing;
    }
  };
  const auto put = [&](int tile) {
    const int x = lane & 15, g = lane >> 4;
#pragma unroll
    for (int i = 0; i < kKinds; ++i) {
      const bool values = is_values(i);
      const int part = put_half(tile) + (su >> 1);  // of keys
      char *to = smem + (values ? (2 + values_place(tile)) * kHalf : keys_place(part) * (kHalf / 2));
      if (lane == 0) {
        // Keys: the factor of a score, tiny instead of 0 (of a page of zeros, whose
        // scores are 0) so that it keeps a masked -inf.  Values: log2 of the scale.
        float v = f[i].scale;
        if (v != kMissing) v = values ? __log2f(v) : v * A.qscale == 0.f ? 1e-30f : v * A.qscale;
        scales[values ? 16 + values_place(tile) * 4 + su : keys_scale_place(part) * 2 + (su & 1)] = v;
      }
      if (!values) {
        // [dim / 8][key 32][8]
        to += ((su & 1) * 16 + x) * 16;
#pragma unroll
        for (int c = 0; c < kPairs; ++c) {
          *(half8_t *)(to + (8 * c + g) * 512) = to_half8(f[i].pair[c][0], f[i].pair[c][1]);
          *(half8_t *)(to + (8 * c + 4 + g) * 512) = to_half8(f[i].pair[c][2], f[i].pair[c][3]);
        }
        if constexpr (kOdd)
          *(half8_t *)(to + (8 * kPairs + g) * 512) = to_half8(f[i].odd[0], f[i].odd[1]);
      } else {
        // [unit 4][half 2][dim][keys 4 half + 0..3, 8 + 4 half + 0..3]
        const auto half4 = [&](uint32_t word, int d) {
          half2_t a, bb;
          to_half4(word, a, bb);
          u32x2_t o = {__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, bb)};
          *(u32x2_t *)(to + ((su * 2 + (g & 1)) * Dp + d) * 16 + (g >> 1) * 8) = o;
        };
#pragma unroll
        for (int c = 0; c < kPairs; ++c)
#pragma unroll
          for (int j = 0; j < 4; ++j) half4(f[i].pair[c][j], 64 * c + 16 * j + x);
        if constexpr (kOdd) {
#pragma unroll
          for (int j = 0; j < 2; ++j) half4(f[i].odd[j], 64 * kPairs + 16 * j + x);
        }
      }
    }
  };
  const float16_t none = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  // Operands of a step: those of the next half's first product (keys, 16 dims
  // each), then those of this half's second (values, 16 keys and 32 dims each).
  // They are read from LDS kAhead matrix instructions before their use.
  constexpr int kSteps = Dp / 16, kAhead = NC > 1 ? 4 : 2;
  const auto operand = [&](const char *kb, const char *vb, int i) {
    if (i < kSteps) return *(const half8_t *)(kb + i * 1024);
    i -= kSteps;
    return *(const half8_t *)(vb + (i / NT * 2 * Dp + i % NT * 32) * 16);
  };
  const auto keys_at = [&](int part) { return smem + keys_place(part) * (kHalf / 2) + lane * 16; };
  // The first product of half a tile (32 keys) alone.
  const auto score = [&](int part) {
    const char *kb = keys_at(part);
    float16_t z = none;
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
      z = __builtin_amdgcn_mfma_f32_32x32x16_f16(*(const half8_t *)(kb + s * 1024), q[s], z, 0, 0, 0);
    return z;
  };

  // Weighs the scores z of half a tile and adds up its values; returns the next
  // half's scores.
  const auto step = [&](int tile, int half, float16_t z) {
    const int t0 = c0 + tile * 64 + half * 32, part = 2 * tile + half;
    if (t0 >= some_last || t0 + 32 <= some_first) return score(part + 1);
    const char *kb = keys_at(part + 1), *vb = smem + (2 + values_place(tile)) * kHalf + ((half * 4 + G) * Dp + n) * 16;
    half8_t ring[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) ring[i] = operand(kb, vb, i);
    const float2_t ks = *(const float2_t *)(scales + keys_scale_place(part) * 2);
    const float2_t vs = *(const float2_t *)(scales + 16 + values_place(tile) * 4 + half * 2);
    // Units that are missing or have no finite scale are rare: the rest of the step
    // gets stand-ins for their scales.
    float2_t factor = ks, share = vs;
    const bool usual = t0 >= all_first && t0 + 32 <= all_last && !__any(!(ks[0] > 0.f && ks[1] > 0.f && vs[0] > kMissing && vs[1] > kMissing));
    bool odd = false;
    if (!usual) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        odd = odd || ks[u] != ks[u] || vs[u] != vs[u];
        if (!(ks[u] > 0.f)) factor[u] = 1.f;
        if (!(vs[u] > kMissing)) share[u] = lr;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int t = t0 + 16 * u + 8 * (j >> 2) + 4 * G + (j & 3);
          const bool in = ks[u] != kMissing && t >= first && t < last;
          z[8 * u + j] = in ? z[8 * u + j] : -INFINITY;
        }
      }
      odd = __any(odd);
    }
    float top[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      top[u] = z[8 * u];
#pragma unroll
      for (int j = 1; j < 8; ++j) top[u] = fmaxf(top[u], z[8 * u + j]);
    }
    const float best = max32(fmaxf(top[0] * factor[0], top[1] * factor[1]));
    const float big = fmaxf(lr, fmaxf(share[0], share[1]));
    const bool up = best > m + kSlack;
    if (__any(up || big > lr)) {
      float g = up ? __builtin_amdgcn_exp2f(m - best) : 1.f;
      l *= g;
      if (up) m = best;
      g *= __builtin_amdgcn_exp2f(lr - big);
      lr = big;
#pragma unroll
      for (int i = 0; i < NT; ++i) O[i] *= g;
    }
    // weight times scale: the scale's share in the exponent, and out again for l
    float add[2], sums[2][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      share[u] = fmaxf(share[u] - lr, -60.f);
      add[u] = share[u] - (m - kUp);
    }
    half8_t p8[2];
    float16_t zn = none;
    // The order is fixed: exponentials after each matrix instruction, in whose time
    // they run.  Left alone, the compiler puts all of the one before all of the other.
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      zn = __builtin_amdgcn_mfma_f32_32x32x16_f16(ring[s % kAhead], q[s], zn, 0, 0, 0);
      here<(NC > 4)>(zn);  // (with more than 256 registers the sums are in the others)
      if (s + kAhead < 2 * kSteps) ring[s % kAhead] = operand(kb, vb, s + kAhead);
#pragma unroll
      for (int e = 2 * (s * 8 / kSteps); e < 2 * ((s + 1) * 8 / kSteps); e += 2) {
        const int u = e >> 3, j = e & 7;
        const float pa = __builtin_amdgcn_exp2f(fmaf(z[e], factor[u], add[u]));
        const float pb = __builtin_amdgcn_exp2f(fmaf(z[e + 1], factor[u], add[u]));
        sums[u][0] = j ? sums[u][0] + pa : pa;
        sums[u][1] = j ? sums[u][1] + pb : pb;
        p8[u][j] = (_Float16)pa;
        p8[u][j + 1] = (_Float16)pb;
        here(half2_t{p8[u][j], p8[u][j + 1]});
      }
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) l = fmaf(sums[u][0] + sums[u][1], __builtin_amdgcn_exp2f(-share[u]), l);
    if (odd) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
        if (ks[u] != ks[u] || vs[u] != vs[u])
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (z[8 * u + j] != -INFINITY) p8[u][j] = (_Float16)NAN;
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      O[i % NT] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ring[(kSteps + i) % kAhead], p8[i / NT], O[i % NT], 0, 0, 0);
      if (i + kAhead < kSteps) ring[(kSteps + i) % kAhead] = operand(kb, vb, kSteps + i + kAhead);
      __builtin_amdgcn_sched_barrier(0);
    }
    return zn;
  };

  float16_t z = none;
  int page[kKinds];
  walk_tiles(
      tiles,
      [&] {
        int p0[kKinds];
        look_up(-1, p0);
        look_up(0, page);
        fetch(-1, p0);  // keys of half 0 (and values of none)
        put(-1);
        fetch(0, page);
        look_up(1, page);
        put(0);
        fetch(1, page);
        look_up(2, page);
      },
      [&](int part) { z = score(part); }, [&](int tile, int half) { z = step(tile, half, z); },
      [&](int tile) {
        // here rather than before the barrier, so that one wave's conversions run
        // beside another's matrix instructions
        put(tile);
        fetch(tile + 1, page);
        look_up(tile + 2, page);
      },
      [] { __syncthreads(); });
  l += other32(l);
  if (w * 32 + n >= it.n) return;
  const float r = __builtin_amdgcn_exp2f(lr);
  if (pieces == 1) {
    const float inv = (l > 0.f || l != l ? 1.f / l : 0.f) * r;
    uint16_t *to = A.out + row_at(A, it, myrow, A.ldo);
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int d = i * 32 + 8 * j + 4 * G;
        if (d >= A.D) continue;
        u32x2_t o;
        o[0] = f2h(O[i][4 * j] * inv) | (f2h(O[i][4 * j + 1] * inv) << 16);
        o[1] = f2h(O[i][4 * j + 2] * inv) | (f2h(O[i][4 * j + 3] * inv) << 16);
        typedef u32x2_t __attribute__((aligned(2), address_space(1))) loose64;
        *(loose64 *)(uintptr_t)(to + d) = o;
      }
    return;
  }
  float *part = A.part + (((int64_t)slot * A.KV + h) * A.pieces + piece) * TR * (Dp + 2);
  const int row = w * 32 + n;
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float4_t o = {O[i][4 * j], O[i][4 * j + 1], O[i][4 * j + 2], O[i][4 * j + 3]};
      *(float4a_t *)(part + row * Dp + i * 32 + 8 * j + 4 * G) = o * r;
    }
  if (G == 0) {
    part[TR * Dp + 2 * row] = m;
    part[TR * Dp + 2 * row + 1] = l;
  }
}

// Both kinds of sequences of a call: those with few rows run on what the others
// leave idle (15 single tokens beside 8 chunks of 251 of 24 heads of 80: 51 us, 64 in
// two launches).
template <int NC, int NW>
__global__ void __launch_bounds__(NW * 64, NC <= 4 ? 2 : 1) k_attend_many(AttendArgs A) {
  extern __shared__ char smem[];
  if (blockIdx.x < A.blocks) return many_rows<NC, NW>(A, smem);
  const unsigned i = blockIdx.x - A.blocks, ht = (unsigned)(A.KV * A.tiles), bp = i / ht, x = i - bp * ht;
  const unsigned piece = bp / (unsigned)A.S.n, h = x / (unsigned)A.tiles;
  few_rows<NC, NW>(A, (int)(bp - piece * A.S.n), (int)h, (int)(x - h * A.tiles), (int)piece, (float *)smem);
}

// --------------------------------------------------------------- joining
// The pieces of a row, by a workgroup: their weights first, then each group of
// Dp / 4 threads adds up every so-manieth piece, and the groups meet in LDS.
// TR = 16: of k_attend_few.  (One wave a row that went through the pieces in
// turn took 127 us for 256 pieces of 64 rows of 128.)
template <int TR>
__global__ void __launch_bounds__(256) k_attend_join(AttendArgs A, int Dp) {
  __shared__ float weight[TR == 16 ? kFewPieces : kManyPieces];
  __shared__ float4_t sums[256];
  __shared__ float wave[2][4];
  const int rows = TR == 16 ? A.frows : TR;  // of an item's partial sums
  const int t = threadIdx.x;
  const unsigned item = blockIdx.x / (unsigned)rows;
  const int row = (int)(blockIdx.x - item * rows);
  Item it;
  if constexpr (TR == 16) {
    const unsigned bh = item / (unsigned)A.tiles, b = bh / (unsigned)A.KV;
    if (!few_item(A, (int)b, (int)(bh - b * A.KV), (int)(item - bh * A.tiles), it)) return;
  } else {
    const unsigned slot = item / (unsigned)A.KV;
    int b;
    if (!many_item<TR>(A, (int)slot, (int)(item - slot * A.KV), it, &b)) return;
  }
  const int pieces = pieces_of(it.lo, it.hi, TR == 16 ? A.few_chunk : A.chunk);
  if (pieces == 1 || row >= it.n) return;
  const int64_t size = (int64_t)rows * (Dp + 2);
  const float *part = TR == 16 ? A.few_part + (int64_t)item * A.few_pieces * size : A.part + (int64_t)item * A.pieces * size;
  const float *ml = part + rows * Dp + 2 * row;
  float M = kNothing;
  for (int p = t; p < pieces; p += 256) {
    const float v = ml[p * size];
    weight[p] = v;
    M = fmaxf(M, v);
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) M = fmaxf(M, lane_xor(M, d));
  if ((t & 63) == 0) wave[0][t >> 6] = M;
  __syncthreads();
  M = fmaxf(fmaxf(wave[0][0], wave[0][1]), fmaxf(wave[0][2], wave[0][3]));
  float L = 0.f;
  for (int p = t; p < pieces; p += 256) {
    const float f = __builtin_amdgcn_exp2f(weight[p] - M);
    weight[p] = f;
    L += ml[p * size + 1] * f;
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) L += lane_xor(L, d);
  if ((t & 63) == 0) wave[1][t >> 6] = L;
  __syncthreads();
  L = wave[1][0] + wave[1][1] + wave[1][2] + wave[1][3];
  const int per = Dp / 4, groups = 256 / per, g = t / per, d = (t - g * per) * 4;
  float4_t o = {0.f, 0.f, 0.f, 0.f};
  if (g < groups) {
    const float *from = part + row * Dp + d;
    int p = g;
    for (; p + 3 * groups < pieces; p += 4 * groups) {
      float4_t v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = *(const float4a_t *)(from + (p + i * groups) * size);
#pragma unroll
      for (int i = 0; i < 4; ++i) o += v[i] * weight[p + i * groups];
    }
    for (; p < pieces; p += groups) o += *(const float4a_t *)(from + p * size) * weight[p];
  }
  sums[t] = o;
  __syncthreads();
  if (g > 0) return;
  for (int i = 1; i < groups; ++i) o += sums[t + i * per];
  write4(A, it, row, d, o, L);
}

// The same of up to kJoinShort pieces of k_attend_many's items: a lane has four dims
// of a row and all of its pieces.  (A wave a row took 18 us for 4096 rows of 8 heads of
// 128 with up to 4 pieces, this 10; with 12 pieces of 64 rows it takes 3 us more than a
// workgroup a row, with 32 of them 13 more.)
template <int TR>
__global__ void __launch_bounds__(256) k_attend_join_short(AttendArgs A, int Dp) {
  static_assert(TR % kJoinRows == 0, "whole workgroups");
  const unsigned item = blockIdx.x / (TR / kJoinRows), slot = item / (unsigned)A.KV;
  const int r0 = (int)(blockIdx.x % (TR / kJoinRows)) * kJoinRows;
  Item it;
  int b;
  if (!many_item<TR>(A, (int)slot, (int)(item - slot * A.KV), it, &b)) return;
  const int pieces = pieces_of(it.lo, it.hi, A.chunk), end = min(it.n, r0 + kJoinRows);
  const int lanes = Dp <= 128 ? 32 : 64, d = (threadIdx.x % lanes) * 4;
  if (pieces == 1 || d >= Dp) return;
  const int64_t size = (int64_t)TR * (Dp + 2);
  const float *part = A.part + (int64_t)item * A.pieces * size;
  for (int row = r0 + threadIdx.x / lanes; row < end; row += 256 / lanes) {
    float2_t ml[kJoinShort];
    float4_t v[kJoinShort];
    float M = kNothing;
#pragma unroll
    for (int p = 0; p < kJoinShort; ++p) {
      ml[p] = float2_t{kNothing, 0.f};
      v[p] = float4_t{0.f, 0.f, 0.f, 0.f};
      if (p >= pieces) continue;
      const float *from = part + p * size;
      ml[p] = *(const float2_t *)(from + TR * Dp + 2 * row);
      v[p] = *(const float4a_t *)(from + row * Dp + d);
    }
#pragma unroll
    for (int p = 0; p < kJoinShort; ++p) M = fmaxf(M, ml[p][0]);
    float L = 0.f;
    float4_t o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int p = 0; p < kJoinShort; ++p) {
      const float w = __builtin_amdgcn_exp2f(ml[p][0] - M);
      o += v[p] * w;
      L += ml[p][1] * w;
    }
    write4(A, it, row, d, o, L);
  }
}

// ------------------------------------------------------------------ host
// The workspace begins with the counts of arrivals, which every launch leaves 0.
constexpr size_t kCountBytes = (size_t)kFewPieces * 4;
__global__ void k_attend_clear(unsigned *count) {
  for (int i = threadIdx.x; i < kFewPieces; i += blockDim.x) count[i] = 0;
}

lb_status grow(lb_cache *C, size_t need, const char *who, bool in_call, hipStream_t st) {
  if (need == 0 || need <= C->ws_bytes) return LB_OK;
  const std::string pre = std::string(who) + ": ";
  if (in_call) {
    hipStreamCaptureStatus cs = hipStreamCaptureStatusNone;
    const hipError_t e = hipStreamIsCapturing(st, &cs);
    if (e != hipSuccess) return set_error(LB_EHIP, pre + hipGetErrorString(e));
    if (cs != hipStreamCaptureStatusNone)
      return set_error(LB_ENOTREADY, pre + "more workspace than reserved while the stream is being captured; call "
                                           "lb_cache_reserve first");
  }
  void *t = nullptr;
  const size_t bytes = grown_bytes(C->Dp, C->cus, C->ws_bytes, need);
  hipError_t e = hipMalloc(&t, kCountBytes + bytes);
  if (e != hipSuccess) return set_error(LB_ENOMEM, pre + "hipMalloc: " + hipGetErrorString(e));
  k_attend_clear<<<dim3(1), dim3(1024), 0, st>>>((unsigned *)t);
  e = hipGetLastError();
  // (a reservation's later calls may be on any stream)
  if (e == hipSuccess && !in_call) e = hipStreamSynchronize(st);
  if (e != hipSuccess) {
    (void)hipFree(t);
    return set_error(LB_EHIP, pre + hipGetErrorString(e));
  }
  if (C->ws) {
    try {
      C->retired.push_back(C->ws);
    } catch (...) {
      (void)hipFree(t);
      return set_error(LB_ENOMEM, pre + "host allocation");
    }
  }
  C->ws = t;
  C->ws_bytes = bytes;
  return LB_OK;
}

template <typename F>
hipError_t allow_lds(F f, int bytes) {
  return bytes > 65536 ? hipFuncSetAttribute((const void *)f, hipFuncAttributeMaxDynamicSharedMemorySize, bytes) : hipSuccess;
}

template <int NC>
hipError_t launch_few(const AttendArgs &A, const Plan &p, hipStream_t st) {
  const int lds = (few_floats(p.frows, NC * 32, kFewWaves) + 32 * kFewWaves + 4) * 4;
  hipError_t e = allow_lds(k_attend_few<NC>, lds);
  // The heads of a page lie side by side, and so do the workgroups that read them
  // (sequences first: 64 sequences took 58 us, not 55; 64 of up to 16384 220, not 200).
  // Windows of sequences keep the grid within its bounds.
  for (int64_t b0 = 0; b0 < A.S.n && e == hipSuccess; b0 += 65535) {
    AttendArgs W = A;
    W.b0 = (int)b0;
    k_attend_few<NC><<<dim3((unsigned)(A.KV * A.tiles), (unsigned)std::min<int64_t>(65535, A.S.n - b0), (unsigned)p.few_pieces),
                       dim3(kFewWaves * 64), lds, st>>>(W);
    e = hipGetLastError();
  }
  return e;
}

template <int NC, int NW>
hipError_t launch_many(AttendArgs A, const Plan &p, hipStream_t st) {
  constexpr int many = 4 * NC * 32 * 128 + 96;
  const int lds = p.few ? std::max(many, (few_floats(p.frows, NC * 32, NW) + 32 * NW + 4) * 4) : many;
  hipError_t e = allow_lds(k_attend_many<NC, NW>, lds);
  if (e != hipSuccess) return e;
  A.blocks = (unsigned)(p.many_items * p.many_pieces);
  k_attend_many<NC, NW><<<dim3((unsigned)(A.blocks + p.few_items * p.few_pieces)), dim3(NW * 64), lds, st>>>(A);
  e = hipGetLastError();
  if constexpr (NW == 4) {  // (256-row tiles are not cut)
    if (e != hipSuccess || p.many_pieces == 1) return e;
    if (p.many_pieces <= kJoinShort)
      k_attend_join_short<128><<<dim3((unsigned)(p.many_items * (128 / kJoinRows))), dim3(256), 0, st>>>(A, NC * 32);
    else
      k_attend_join<128><<<dim3((unsigned)(p.many_items * 128)), dim3(256), 0, st>>>(A, NC * 32);
    e = hipGetLastError();
  }
  return e;
}

template <int NC>
hipError_t launch(const AttendArgs &A, const Plan &p, hipStream_t st) {
  hipError_t e;
  if (!p.many) {
    e = launch_few<NC>(A, p, st);
  } else if constexpr (NC <= 4) {
    e = p.tr == 256 ? launch_many<NC, 8>(A, p, st) : launch_many<NC, 4>(A, p, st);
  } else {
    e = launch_many<NC, 4>(A, p, st);
  }
  if (e != hipSuccess || !p.few || p.few_pieces == 1 || A.count) return e;
  k_attend_join<16><<<dim3((unsigned)(p.few_items * p.frows)), dim3(256), 0, st>>>(A, NC * 32);
  return hipGetLastError();
}

// The chunk of 32 dims as a constant.
template <typename F>
hipError_t with_dims(int Dp, F f) {
  switch (Dp / 32) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    case 3: return f(std::integral_constant<int, 3>());
    case 4: return f(std::integral_constant<int, 4>());
    case 5: return f(std::integral_constant<int, 5>());
    case 6: return f(std::integral_constant<int, 6>());
    case 7: return f(std::integral_constant<int, 7>());
    default: return f(std::integral_constant<int, 8>());
  }
}

}  // namespace

extern "C" lb_status lb_cache_reserve(lb_cache *C, int64_t rows, int heads, int64_t sequences, int64_t max_length) {
  const auto refuse = [](const char *why) { return set_error(LB_EINVAL, std::string("lb_cache_reserve: ") + why); };
  if (!C) return refuse("NULL cache");
  if (rows < 0 || rows > kMaxRows || sequences < 0 || sequences > kMaxRows || max_length < 0 || max_length > kMaxRows)
    return refuse("rows, sequences and max_length must be in [0, 2^30]");
  if (heads < 1 || heads > 65536 || heads % C->KV) return refuse("heads must be a multiple of the cache's key heads");
  if (rows == 0 || sequences == 0) return LB_OK;
  const size_t need = reserve_bytes(C->Dp, C->cus, rows, heads / C->KV, max_length);
  DeviceGuard dg(C->device);
  return grow(C, need, "lb_cache_reserve", false, nullptr);
}

extern "C" lb_status lb_cache_attend(lb_cache *C, const void *q, int64_t ldq, int heads, void *out, int64_t ldo,
                                     const int32_t *start, const int32_t *lengths, const int32_t *table, int64_t ldt,
                                     int columns, int sequences, int64_t rows, int64_t max_length, float scale,
                                     int causal, int window, void *stream) {
  const auto refuse = [](const char *why) { return set_error(LB_EINVAL, std::string("lb_cache_attend: ") + why); };
  if (!C) return refuse("NULL cache");
  if (rows < 0 || rows > kMaxRows || sequences < 0 || sequences > kMaxRows)
    return refuse("rows and sequences must be in [0, 2^30]");
  if (heads < 1 || heads > 65536 || heads % C->KV) return refuse("heads must be a multiple of the cache's key heads");
  // (scores then stay far above kNothing)
  if (!(scale >= 0.f) || scale > 1e6f) return refuse("scale must be in [0, 1e6]");
  if (window < 0 || (window && !causal)) return refuse("a window is not negative and needs causal");
  if (max_length < 0 || max_length > kMaxRows) return refuse("max_length must be in [0, 2^30]");
  if (rows == 0) return LB_OK;
  const Sequences S = {start, lengths, table, ldt, sequences, (int)rows, columns, (int)C->pages};
  lb_status st = check_sequences(C, S, "lb_cache_attend");
  if (st != LB_OK) return st;
  if (!q || !out) return refuse("NULL q or out");
  const int64_t qw = (int64_t)heads * C->D, most_ld = (int64_t)1 << 31;
  if (ldq < qw || ldo < qw) return refuse("a row stride is smaller than the row");
  if (ldq > most_ld || ldo > most_ld) return refuse("a row stride exceeds 2^31");
  if (((uintptr_t)q | (uintptr_t)out) % 2) return refuse("misaligned pointer");
  const Rows o = {out, rows, (size_t)ldo * 2, (size_t)qw * 2};
  if (meet({q, rows, (size_t)ldq * 2, (size_t)qw * 2}, o)) return refuse("q and out overlap");
  if ((start && meet({start, 1, 0, (size_t)(sequences + 1) * 4}, o)) || meet({lengths, 1, 0, (size_t)sequences * 4}, o) ||
      meet({table, sequences, (size_t)ldt * 4, (size_t)columns * 4}, o))
    return refuse("an input and out overlap");
  if (sequences == 0) return LB_OK;
  int64_t most = (int64_t)columns * C->P;
  if (max_length) most = std::min(most, max_length);
  if (window >= kMaxTokens) window = 0;  // hides nothing, and a position less it passes 32 bits
  View view = {heads / C->KV, causal != 0, window, (int)most};
  if (rows * (int64_t)view.group > 0x7fffffff)
    return set_error(LB_EUNSUPPORTED, "lb_cache_attend: too many rows and heads for one call");
  const Plan p = plan_of(C->KV, C->Dp, C->cus, start != nullptr, rows, sequences, view);
  if ((p.few_items * p.few_pieces + p.many_items * p.many_pieces) > 0x7fffffff / 512 || p.many_items * p.tr > 0x7fffffff)
    return set_error(LB_EUNSUPPORTED, "lb_cache_attend: too many rows and heads for one call");
  DeviceGuard dg(C->device);
  hipStream_t stm = (hipStream_t)stream;
  st = grow(C, p.few_ws + p.many_ws, "lb_cache_attend", true, stm);
  if (st != LB_OK) return st;
  AttendArgs A = {};
  A.S = S;
  A.q = (const uint16_t *)q;
  A.out = (uint16_t *)out;
  A.ldq = ldq; A.ldo = ldo;
  A.kc = C->k; A.vc = C->v; A.ks = C->ks; A.vs = C->vs;
  A.few_part = (float *)((char *)C->ws + kCountBytes);
  A.qscale = scale * 1.44269504088896340736f;
  A.KV = C->KV; A.D = C->D; A.lg = C->lg;
  A.view = view;
  A.few = p.few_rows;
  A.tiles = p.tiles;
  A.frows = p.frows;
  A.row_tiles = p.row_tiles;
  A.few_chunk = p.few_chunk;
  A.few_pieces = p.few_pieces;
  A.chunk = p.many_chunk;
  A.pieces = p.many_pieces;
  A.part = A.few_part + p.few_ws / 4;
  if (p.few_pieces > 1 && p.few_pieces <= kJoinHere) A.count = (unsigned *)C->ws;
  const hipError_t e = with_dims(C->Dp, [&](auto nc) { return launch<decltype(nc)::value>(A, p, stm); });
  if (e != hipSuccess) return set_error(LB_EHIP, std::string("lb_cache_attend: ") + hipGetErrorString(e));
  return LB_OK;
}
