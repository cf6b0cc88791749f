// A bank of LittleBit layers of one shape: the fused-epilogue forward of
// one of them (lb_bank_forward) and the products of many over rows sorted
// by expert (lb_bank_grouped).
//
// For every row x, with the layer of [LB news] Sec. 2
//
//   L(x) = sum_p h_p * ( S_U,p ( l_p * ( S_V,p^T ( g_p * x ) ) ) ),
//
// a call computes y = act(L(x) + bias) + residual, or with a gate layer G of
// the same shape y = act(G(x) + gate_bias) * (L(x) + bias) + residual, in
// two launches on the fp16 matrix cores:
//
//   first product   t = x . (g_p S_V,p), w = l_p t for every segment
//                   (layer side, path) of s latent columns;
//   second product  sum_p w_p . (h_p S_U,p)^T, then the epilogue.
//
// Rounding: the operands +-g and +-h are exact in fp16 (a stored scale with
// its sign bit flipped), x is fp16, the accumulators are fp32.  w is kept as
// two fp16 numbers, hi = fp16(w) and lo = fp16(2^11 (w - hi)): the pair
// carries 22 bits of w for every |w| < 65504 down to 2^-14 (an absolute
// 2^-36 below), so y is rounded once, at the end, whatever the batch size.
// Both are multiplied by the same +-h; the lo sums are kept apart and joined
// to the hi sums times 2^-11 in fp32.  (2^-11 h as an operand would lose a
// bit for every halving of |h| below 2^-3, where it is no longer normal;
// k_bank_second_wide without gates uses one, and scales h first.)  With w as
// one fp16 number the error of an fp16 y is 1.4 times that of its own
// rounding (1.75 times when gated).
//
// Rows are cut into slots of n rows (16, 32 or 64, see run) of one expert.
// Without offsets slot i is rows [i n, (i + 1) n); with offsets every wave
// finds its slot from the experts' row counts, so the host never waits for
// them: the grid is sized for the most slots that `rows` rows can make,
// rows / n + min(experts, rows), and workgroups past the last slot leave.
//
// Latent workspace T, per 32-row part of a slot (ps), segment and block of 16
// columns: [hi, lo][column half 2][32 rows][8 fp16], so that an operand load
// of a wave is 1 KB contiguous:
//   T[(((ps nseg + seg) 2 Wk + k16) 2 + plane) 512 + (c8 32 + row) 8 + c].
// Columns past s are zero.
//
// Instruction (32- and 64-row slots): v_mfma_f32_32x32x16_f16.  Operand lanes: A[i][k] in lane
// i + 32 (k / 8), element k % 8; B[k][j] in lane j + 32 (k / 8), element
// k % 8; D[i][j] in lane j + 32 ((i / 4) % 2), register 4 (i / 8) + i % 4.
#include <hip/hip_fp16.h>

#include <algorithm>
#include <new>
#include <string>
#include <type_traits>
#include <vector>

#include "lb_internal.h"

namespace {

using namespace lbi;

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float float4_t __attribute__((ext_vector_type(4)));
typedef float float16_t __attribute__((ext_vector_type(16)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

// Pointers read from memory say themselves that they are global: through
// generic ones every load would count as an LDS access too and be waited for
// by the next LDS read.
typedef const uint32_t __attribute__((address_space(1))) *gu32;
typedef const uint16_t __attribute__((address_space(1))) *gu16;
typedef const u32x4 __attribute__((address_space(1))) *gu128;

// One layer of the bank: its matrix-core sign copies and scales.
struct LayerDesc {
  gu32 sv, su;
  gu16 g, l, h;
};

struct BankArgs {
  const LayerDesc *desc;  // [side][expert], side 0 = the layers, 1 = the gates
  LayerDesc one[2];       // those of expert e0, when offsets is null: no load to wait for
  const uint16_t *x;
  const int *index;    // x row of every grouped row, or null
  const int *offsets;  // E + 1 row offsets, or null (every row belongs to expert e0)
  uint16_t *T;
  void *y;
  const void *res;
  const uint16_t *bias[2];  // per side, E x b
  const void *zero;         // >= 16 zero bytes, read in place of what is out of range
  int64_t ldx, ldy, ldr;
  int rows, x_rows, E, e0;
  int a, a16, b, b16, s, L, P, G, R1, Wk;
  int lg, slot0;  // rows per slot are 2^lg; first slot of this launch
  int span;       // neighbouring tiles that go to one XCD (many-row kernels)
  int act, f32, xvec;
};

#define LB_G(T, p) ((T)(uintptr_t)(p))

// 16 and 4 bytes at an element's alignment: global memory takes them as one
// access (with eight 2-byte ones 1023 rows of 1031 -> 2743 took 23.7 us, not
// 17.3).
typedef u32x4 __attribute__((aligned(2), address_space(1))) loose128;
typedef uint32_t __attribute__((aligned(2), address_space(1))) loose32;

__device__ __forceinline__ float h2f(uint16_t v) { return __half2float(__ushort_as_half(v)); }
__device__ __forceinline__ uint16_t f2h(float v) { return __half_as_ushort(__float2half_rn(v)); }
__device__ __forceinline__ half8_t as_h8(u32x4 v) { return __builtin_bit_cast(half8_t, v); }
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// 8 operand values v with the signs of wl (matrix-core bit order, shifted to
// the lane's group of 8): one shift and one three-input bit operation per
// pair of values.
__device__ __forceinline__ half8_t flip(u32x4 v, uint32_t wl) {
  v.x ^= wl & 0x80008000u;
  v.y ^= (wl << 1) & 0x80008000u;
  v.z ^= (wl << 2) & 0x80008000u;
  v.w ^= (wl << 3) & 0x80008000u;
  return as_h8(v);
}

__device__ __forceinline__ u32x4 splat(uint32_t v) {
  u32x4 o = {v, v, v, v};
  return o;
}

// Slot `slot` of the call: its expert, first row and row count.
// Uniform over the wave; false past the last slot.  Offsets are clamped to
// [0, rows], so no row outside the call is touched whatever they hold.
__device__ __forceinline__ bool find_slot(const BankArgs &A, int slot, int &e, int &row0, int &n) {
  if (!A.offsets) {
    const int64_t r = (int64_t)slot << A.lg;
    if (r >= A.rows) return false;
    e = A.e0;
    row0 = (int)r;
    n = min(1 << A.lg, A.rows - row0);
    return true;
  }
  const int lane = threadIdx.x & 63;
  int base = 0;
  for (int eb = 0; eb < A.E; eb += 64) {
    const int ee = eb + lane;
    int lo = 0, c = 0;
    if (ee < A.E) {
      lo = min(max(A.offsets[ee], 0), A.rows);
      c = max(min(max(A.offsets[ee + 1], 0), A.rows) - lo, 0);
    }
    const int t = (c + (1 << A.lg) - 1) >> A.lg;
    int inc = t;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(inc, d);
      if (lane >= d) inc += v;
    }
    const int k = slot - (base + inc - t);  // the slot's place among this expert's
    const unsigned long long hit = __ballot(k >= 0 && k < t);
    if (hit) {
      const int src = __ffsll(hit) - 1;
      const int ks = __shfl(k, src);
      e = __builtin_amdgcn_readfirstlane(eb + src);
      row0 = __builtin_amdgcn_readfirstlane(__shfl(lo, src) + (ks << A.lg));
      n = __builtin_amdgcn_readfirstlane(min(1 << A.lg, __shfl(c, src) - (ks << A.lg)));
      return true;
    }
    base += __shfl(inc, 63);
  }
  return false;
}

__device__ __forceinline__ LayerDesc layer_of(const BankArgs &A, int side, int e) {
  return A.offsets ? A.desc[side * A.E + e] : A.one[side];
}

// 8 fp16 of an x row from element i on (any 2-byte alignment unless XV);
// zeros past a.
template <bool XV>
__device__ __forceinline__ u32x4 load8(const uint16_t *p) {
  if constexpr (XV)
    return *LB_G(gu128, p);
  else
    return *LB_G(const loose128 *, p);
}
template <bool XV>
__device__ __forceinline__ u32x4 load_x(const BankArgs &A, const uint16_t *row, int i) {
  if (i + 8 <= A.a) return load8<XV>(row + i);
  uint32_t v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = i + e < A.a ? *LB_G(gu16, row + i + e) : (uint16_t)0;
  u32x4 o;
  o.x = v[0] | (v[1] << 16);
  o.y = v[2] | (v[3] << 16);
  o.z = v[4] | (v[5] << 16);
  o.w = v[6] | (v[7] << 16);
  return o;
}

// The tile of a workgroup: workgroup i runs on XCD i % 8, and each XCD takes
// runs of `span` neighbouring tiles, which share their operands in its L2.
__device__ __forceinline__ int xcd_tile(int span) {
  const int xcd = blockIdx.x & 7, i = blockIdx.x >> 3, run = i / span;
  return (run * 8 + xcd) * span + (i - run * span);
}

// The x row that row r of the slot reads: its own or its index's, and
// whether there is one.  Rows past the slot's end and bad indexes read a row
// that is there; the first are dropped with y's rows, the second zeroed in T.
__device__ __forceinline__ int64_t x_row(const BankArgs &A, int row0, int n, int r, bool &ok) {
  int64_t v = row0 + min(r, n - 1);
  ok = true;
  if (A.index) {
    v = A.index[v];
    ok = v >= 0 && v < A.x_rows;
    if (!ok) v = 0;
  }
  return v;
}

// w as hi and lo halves at o and o + 512 of a T block.
__device__ __forceinline__ void put_w(uint16_t *t, int o, float v) {
  const uint16_t hi = f2h(v);
  const float hf = h2f(hi);
  t[o] = hi;
  t[o + 512] = isinf(hf) ? (uint16_t)0 : f2h((v - hf) * 2048.f);
}

// Copies straight into LDS: lane i's 16 (4) bytes land at dst + 16 i (4 i).
__device__ __forceinline__ void dma16(const void *src, void *dst) {
  __builtin_amdgcn_global_load_lds(src, dst, 16, 0, 0);
}
__device__ __forceinline__ void dma4(const void *src, void *dst) {
  __builtin_amdgcn_global_load_lds(src, dst, 4, 0, 0);
}
// Waits until at most N of the wave's loads are in flight.
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Waits for the wave's LDS reads.
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// ------------------------------------------------------- first product
// Few rows (slots of 16): a workgroup of NW waves computes 16 rows x 16 latent
// columns over the whole input dimension, wave w on the blocks of 32 inputs
// 2 w, 2 w + 1, 2 w + 2 NW, ... (pairs: whole 128-byte lines of x; single blocks
// took 7.2 us, not 4.3, for 16 rows of 1024); the waves' sums are added in wave
// order through LDS.  Bound by latency and by what one CU can issue, hence the
// small tile (a 32 x 32 one took 6.5 us for one row of a 4096-wide layer, two
// thirds of it on the four waves a SIMD that wanted to expand signs at once),
// operands of kF1U blocks requested together, and g (the same for all columns)
// straight into the wave's LDS.  One row of 4096: 5.1 us, 16 rows 7.8; 11008:
// 7.4 and 14.5.  4 waves take 5.8 and 8.2, 11.2 and 15.0; 16 waves 6.1 and 11.2,
// 8.8 and 18.8.  Up to 2048 inputs, all blocks of which 4 waves request at once,
// 4 do: 64 layers of 1024 inputs, 60 gated rows (some 800 workgroups) 5.9 us
// against 8.0 with 8, and one slot as fast (1024 inputs 3.8 against 3.7, 16 rows
// of 2048 5.7 against 5.4).
// v_mfma_f32_16x16x32_f16: A[i][k] in lane i + 16 (k / 8), B[k][j] in lane
// j + 16 (k / 8), D[i][j] in lane j + 16 (i / 4), register i % 4.
constexpr int kF1U = 16;

template <int NW, bool XV>
__global__ void __launch_bounds__(NW * 64)
k_bank_first16(BankArgs A) {
  __shared__ __align__(16) float red[NW * 256];
  const int tile = blockIdx.x, slot = blockIdx.y, W2 = 2 * A.Wk;
  int seg = 0;
#pragma unroll
  for (int i = 1; i < 4; ++i) seg += tile >= i * W2;
  const int k16 = tile - seg * W2, side = A.P == 2 ? seg >> 1 : seg, p = A.P == 2 ? seg & 1 : 0;
  int e, row0, n;
  if (!find_slot(A, A.slot0 + slot, e, row0, n)) return;
  const LayerDesc D = layer_of(A, side, e);

  const int w = wave_id(), lane = threadIdx.x & 63, lr = lane & 15, o = lane >> 4;
  const int k = k16 * 16 + lr;
  uint16_t *T = A.T + ((size_t)slot * A.G * A.P * W2 + tile) * 1024;
  if (k16 * 16 >= A.s) {  // padding
    if (threadIdx.x < 64) {
      const int at = (threadIdx.x >> 4) * 256 + (threadIdx.x & 15) * 8;
      *reinterpret_cast<u32x4 *>(T + at) = splat(0u);
    }
    return;
  }
  const unsigned col = min(k, A.s - 1);  // columns past s repeat the last and are zeroed below
  bool ok;
  const uint16_t *xr = A.x + x_row(A, row0, n, lr, ok) * A.ldx;
  const unsigned there = (unsigned)__ballot(ok);  // lanes 0..15: the rows
  const gu16 g = D.g + (size_t)p * A.a16;
  const gu32 bw = D.sv + (size_t)p * A.s;
  const float lk = h2f(D.l[(size_t)p * ((A.s + 7) / 8 * 8) + col]);

  float4_t acc = {0.f, 0.f, 0.f, 0.f};
  const int full = A.a >> 5;                                            // whole blocks
  unsigned char *gl = reinterpret_cast<unsigned char *>(red + w * 256);  // the wave's own part of red
  const u32x4 *gs = reinterpret_cast<const u32x4 *>(gl);
  auto block = [](int c0, int u) { return c0 + (u >> 1) * 2 * NW + (u & 1); };
  for (int c0 = 2 * w; c0 < full; c0 += NW * kF1U) {
    uint32_t wd[kF1U];
    u32x4 xv[kF1U];
    dma16((const void *)(g + min(block(c0, lane >> 2), full - 1) * 32 + (lane & 3) * 8), gl);
#pragma unroll
    for (int u = 0; u < kF1U; ++u) {
      if (u % 4 == 0 && block(c0, u) >= full) break;
      const int c = min(block(c0, u), full - 1);  // past the end: read, not used
      wd[u] = (bw + (size_t)c * A.L)[col];
      xv[u] = load8<XV>(xr + c * 32 + o * 8);
    }
    wait_loads<0>();
#pragma unroll
    for (int u = 0; u < kF1U; ++u) {
      if (block(c0, u) >= full) break;
      acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(as_h8(xv[u]), flip(gs[4 * u + o], wd[u] << (4 * o)), acc, 0, 0, 0);
    }
    wait_lds();  // g has been read before the next round's is copied over it
  }
  if (full < A.R1 && w == NW - 1) {  // the last block is not whole
    const int i = full * 32 + o * 8;
    const u32x4 gv = *(i < A.a16 ? (gu128)(g + i) : LB_G(gu128, A.zero));
    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(as_h8(load_x<XV>(A, xr, i)),
                                                 flip(gv, (bw + (size_t)full * A.L)[col] << (4 * o)), acc, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) red[(w * 4 + i) * 64 + lane] = acc[i];
  __syncthreads();
  __shared__ __align__(16) uint16_t tl[1024];  // the T block
  if (w < 4) {  // wave w finishes register w
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < NW; ++q) v += red[(q * 4 + w) * 64 + lane];
    const int row = 4 * o + w;
    const bool keep = k < A.s && ((there >> row) & 1u);
    put_w(tl, ((lr >> 3) * 32 + row) * 8 + (lr & 7), keep ? v * lk : 0.f);
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    const int at = (threadIdx.x >> 4) * 256 + (threadIdx.x & 15) * 8;  // [plane, c8][row]
    *reinterpret_cast<u32x4 *>(T + at) = *reinterpret_cast<const u32x4 *>(tl + at);
  }
}

// Workgroup barrier for LDS alone: global loads in flight stay in flight.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Many rows: a workgroup of NW waves computes 32 RT rows x 32 CT columns of one
// segment over the whole input dimension, wave w on the blocks of 32 inputs
// 2 w, 2 w + 1, 2 w + 2 NW, ... (pairs: whole 128-byte lines of x).  A wave
// shares its operands with no other, so it stages them itself, without
// barriers: x rows, the block's g and its columns' sign words are copied into
// a ring of kW1Ring blocks in the wave's own LDS, all but one in flight (piece
// c of row r in slot c ^ (r / 2) % 4, so that the operand reads meet no bank
// twice).  One expanded sign operand serves RT products.  The waves' sums are
// added in wave order through LDS, 32 columns at a time.  The workgroups of
// one slot lie side by side (xcd_tile), so its x rows come from an L2 after
// the first.  A round of workgroups over 4096 inputs takes 9.5, 11.4, 15 and
// 20 us with RT = 1 and CT = 1, 2, 3 and 5 (start and sums included), 22 and
// 33 with RT = 2 and CT = 3 and 5: at 5 a wave's products are 60% of its time,
// the rest is sign flips and LDS reads, and the start and end of the launch.
constexpr int kW1Ring = 4;
template <int RT, int CT>
constexpr int w1_block() { return RT * 2048 + (CT + 1) / 2 * 256 + 64; }  // x, words, g
template <int RT, int CT, int NW>
constexpr int w1_lds() {
  return std::max(NW * kW1Ring * w1_block<RT, CT>(), RT * (NW * 4096 + 4096));
}

template <int RT, int CT, int NW, bool XV>
__global__ void __launch_bounds__(NW * 64, 8 / NW)
k_bank_first_wide(BankArgs A, int slots, int ncs) {
  extern __shared__ __align__(16) unsigned char sm[];
  constexpr int kBlock = w1_block<RT, CT>(), kWords = RT * 2048, kG = kBlock - 64, kPer = 2 * RT + (CT + 1) / 2 + 1;
  const int ncg = A.G * A.P * ncs, at = xcd_tile(A.span);
  const int slot = at / ncg, cg = at - slot * ncg;
  int e, row0, n;
  if (slot >= slots || !find_slot(A, A.slot0 + slot, e, row0, n)) return;
  const int seg = cg / ncs, ct0 = (cg - seg * ncs) * CT;
  const int side = seg / A.P, p = seg - side * A.P;
  const LayerDesc D = layer_of(A, side, e);

  const int w = wave_id(), lane = threadIdx.x & 63, lr = lane & 31, lh = lane >> 5;
  unsigned char *ring = sm + w * kW1Ring * kBlock;
  const gu16 g = D.g + (size_t)p * A.a16;
  const gu32 bw = D.sv + (size_t)p * A.s;  // uniform
  unsigned col[(CT + 1) / 2];              // the columns whose words the lane copies
#pragma unroll
  for (int q = 0; q < (CT + 1) / 2; ++q) col[q] = min(ct0 * 32 + q * 64 + lane, A.s - 1);
  // the lane's rows: 16 u + lane / 4, 16 bytes of each
  const int piece = (lane & 3) ^ ((lane >> 3) & 3);
  const uint16_t *xrow[2 * RT];
  bool ok;
#pragma unroll
  for (int u = 0; u < 2 * RT; ++u) xrow[u] = A.x + x_row(A, row0, n, 16 * u + (lane >> 2), ok) * A.ldx;
  (void)x_row(A, row0, n, lane & (32 * RT - 1), ok);
  const unsigned long long there = __ballot(ok);

  float16_t acc[RT][CT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[rt][ct][i] = 0.f;

  // the wave's block number i is block 2 NW (i / 2) + 2 w + i % 2 of the input
  const int behind = max(0, A.R1 - 2 * w);  // blocks from its first on
  const int mine = (behind + 2 * NW - 1) / (2 * NW) * 2 - (behind % (2 * NW) == 1 ? 1 : 0);
  // the next block to be copied: its number, place, and the addresses, which
  // only advance
  int kb = 2 * w, fs = 0;
#pragma unroll
  for (int u = 0; u < 2 * RT; ++u) xrow[u] += kb * 32 + piece * 8;
  gu32 wrow = bw + (size_t)kb * A.L;
  gu16 grow = g + kb * 32 + (lane & 3) * 8;
  auto issue = [&]() {  // kPer loads
    unsigned char *dst = ring + fs;
    const bool whole = kb * 32 + 32 <= A.a;  // uniform
#pragma unroll
    for (int u = 0; u < 2 * RT; ++u) {
      if constexpr (XV)
        dma16(whole || kb * 32 + piece * 8 < A.a ? (const void *)xrow[u] : A.zero, dst + u * 1024);
      else
        *reinterpret_cast<u32x4 *>(dst + u * 1024 + lane * 16) =
            load_x<false>(A, xrow[u] - (kb * 32 + piece * 8), kb * 32 + piece * 8);
    }
#pragma unroll
    for (int q = 0; q < (CT + 1) / 2; ++q) dma4((const void *)(wrow + col[q]), dst + kWords + q * 256);
    if (lane < 4) dma16(whole || kb * 32 + lane * 8 < A.a16 ? (const void *)grow : A.zero, dst + kG);
    const int step = kb & 1 ? 2 * NW - 1 : 1;
    kb += step;
#pragma unroll
    for (int u = 0; u < 2 * RT; ++u) xrow[u] += step * 32;
    wrow += (size_t)step * A.L;
    grow += step * 32;
    fs = fs + kBlock == kW1Ring * kBlock ? 0 : fs + kBlock;
  };
  // operands: half 0 of a block is read during the products of half 1 of the
  // one before, half 1 during those of half 0
  u32x4 gv[2], xv[2][RT];
  uint32_t wd[CT], wn[CT];
  auto read = [&](int t, const unsigned char *blk) {
    gv[t] = reinterpret_cast<const u32x4 *>(blk + kG)[2 * t + lh];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
      xv[t][rt] = reinterpret_cast<const u32x4 *>(blk)[(rt * 32 + lr) * 4 + ((2 * t + lh) ^ ((lr >> 1) & 3))];
  };
  auto read_words = [&](uint32_t (&to)[CT], const unsigned char *blk) {
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) to[ct] = reinterpret_cast<const uint32_t *>(blk + kWords)[ct * 32 + lr];
  };
  auto multiply = [&](int t) {
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      const half8_t b = flip(gv[t], wd[ct] << (8 * t));
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
        acc[rt][ct] = __builtin_amdgcn_mfma_f32_32x32x16_f16(as_h8(xv[t][rt]), b, acc[rt][ct], 0, 0, 0);
    }
  };
#pragma unroll
  for (int i = 0; i < kW1Ring - 1; ++i)
    if (i < mine) issue();
  if (mine > 0) {
    if (XV && mine >= 3)
      wait_loads<2 * kPer>();
    else
      wait_loads<0>();
    read(0, ring);
    read_words(wd, ring);
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) wd[ct] <<= 4 * lh;
  }
  int rs = 0;  // place of block i
  auto round = [&](bool more, bool next, auto wait) {
    const unsigned char *blk = ring + rs;
    rs = rs + kBlock == kW1Ring * kBlock ? 0 : rs + kBlock;
    read(1, blk);
    if (more) issue();  // into the block read in the round before this
    multiply(0);
    if (next) {
      wait();  // the next block has landed
      read(0, ring + rs);
      read_words(wn, ring + rs);
    }
    multiply(1);
    if (next) {
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) wd[ct] = wn[ct] << (4 * lh);
      // The words were requested last and LDS answers in order: the block read
      // in this round has been read before the next round copies over it.
      asm volatile("" : "+v"(wd[CT - 1])::"memory");
    }
  };
  int i = 0;
  for (; i + 3 < mine; ++i) round(true, true, [] { wait_loads<XV ? 2 * kPer : 0>(); });
  for (; i < mine; ++i) round(false, i + 1 < mine, [] { wait_loads<0>(); });
  // sums over the waves and w = l t, a column tile at a time
  float4_t *red = reinterpret_cast<float4_t *>(sm);                         // [wave][rt][registers / 4][lane]
  uint16_t *tl = reinterpret_cast<uint16_t *>(sm + RT * NW * 4096);  // [rt][2048]
  const int nseg = A.G * A.P;
  __syncthreads();
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    const int tile = ct0 + ct;
    if (tile >= A.Wk) break;  // uniform
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float16_t &c = acc[rt][ct];
        red[((w * RT + rt) * 4 + q) * 64 + lane] = float4_t{c[4 * q], c[4 * q + 1], c[4 * q + 2], c[4 * q + 3]};
      }
    __syncthreads();
    const int k = tile * 32 + lr;
    const float lk = k < A.s ? h2f(D.l[(size_t)p * ((A.s + 7) / 8 * 8) + k]) : 0.f;
#pragma unroll
    for (int u = 0; u < (RT * 4 + NW - 1) / NW; ++u) {
      const int idx = u * NW * 64 + threadIdx.x, rt = idx >> 8, q = (idx >> 6) & 3;
      if (RT * 4 < NW && idx >= RT * 256) break;
      float4_t v = red[idx];
#pragma unroll
      for (int z = 1; z < NW; ++z) v += red[z * RT * 256 + idx];
      const int row = 8 * q + 4 * lh;
      const unsigned here = (unsigned)(there >> (rt * 32 + row)) & 15u;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        put_w(tl, rt * 2048 + (lr >> 4) * 1024 + (((lr >> 3) & 1) * 32 + row + i) * 8 + (lr & 7),
              k < A.s && ((here >> i) & 1u) ? v[i] * lk : 0.f);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < RT * 256; i += NW * 64) {
      const int rt = i >> 8;
      u32x4 *dst = reinterpret_cast<u32x4 *>(A.T + (((size_t)(slot * RT + rt) * nseg + seg) * A.Wk + tile) * 2048);
      dst[i & 255] = reinterpret_cast<const u32x4 *>(tl)[i];
    }
  }
}

// ------------------------------------------------------ second product
// Activations in fp32 on the hardware's exp2 and reciprocal (a step of error
// each): v / (1 + exp(-c)) takes six instructions, where expf and a division
// take some forty, and a wave has 64 of them against 288 matrix products.  The
// rounding of exp's argument u adds a few times |u| 2^-24 of the result, so far
// into a tail the relative error grows (SiLU at -10: up to 2e-6); the absolute
// one does not.
__device__ __forceinline__ float exp2_hw(float v) { return __builtin_amdgcn_exp2f(v); }
__device__ __forceinline__ float rcp_hw(float v) { return __builtin_amdgcn_rcpf(v); }
constexpr float kLog2e = 1.4426950408889634f;

template <int ACT>
__device__ __forceinline__ float activate(float v) {
  if constexpr (ACT == LB_ACT_RELU) {
    return v > 0.f || v != v ? v : 0.f;
  } else if constexpr (ACT == LB_ACT_GELU) {
    // v/2 erfc(-v / sqrt 2).  For z = |v| / sqrt 2, exp(z^2) erfc(z) = t P(t) with
    // t = 1 / (1 + 0.21 |v|) and P a least-maximum fit of degree 8 to 0 <= z <= 10
    // (2^-25.8 of the value), so the tail is as exact as the rest.  (A fit of
    // small absolute error, 1.5e-7, was off by 5e-4 of gelu(-4), a whole half
    // step of fp16.)
    const float t = rcp_hw(fmaf(0.21f, fabsf(v), 1.f));
    float q = fmaf(-0.14310356f, t, 0.56614528f);
    q = fmaf(q, t, -0.65833091f);
    q = fmaf(q, t, 0.69624549f);
    q = fmaf(q, t, -0.18602241f);
    q = fmaf(q, t, 0.24893199f);
    q = fmaf(q, t, 0.1386041f);
    q = fmaf(q, t, 0.17010479f);
    q = fmaf(q, t, 0.16742524f) * t * exp2_hw(-0.5f * kLog2e * (v * v));  // erfc(z)
    return 0.5f * v * (v > 0.f ? 2.f - q : q);
  } else if constexpr (ACT == LB_ACT_GELU_TANH) {
    // (1 + tanh u) / 2 = 1 / (1 + exp(-2 u)): no cancellation for negative u
    return v * rcp_hw(1.f + exp2_hw(-2.f * 0.79788456080286536f * kLog2e * fmaf(0.044715f * v * v, v, v)));
  } else if constexpr (ACT == LB_ACT_SILU) {
    return v * rcp_hw(1.f + exp2_hw(-kLog2e * v));
  } else {
    return v;
  }
}

// Calls f with the activation as a compile-time constant.
template <class F>
__device__ __forceinline__ void with_act(int act, F &&f) {
  switch (act) {
    case LB_ACT_RELU: return f(std::integral_constant<int, LB_ACT_RELU>());
    case LB_ACT_GELU: return f(std::integral_constant<int, LB_ACT_GELU>());
    case LB_ACT_GELU_TANH: return f(std::integral_constant<int, LB_ACT_GELU_TANH>());
    case LB_ACT_SILU: return f(std::integral_constant<int, LB_ACT_SILU>());
    default: return f(std::integral_constant<int, LB_ACT_NONE>());
  }
}

template <int CT>
constexpr int pitch2() { return 32 * CT + 4; }

// The biases of the lane's columns j0 + 32 ct + lane % 32.
template <int CT>
__device__ __forceinline__ void load_bias(const BankArgs &A, int side, int e, int j0, float (&v)[CT]) {
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    const int j = j0 + ct * 32 + (threadIdx.x & 31);
    v[ct] = A.bias[side] && j < A.b ? h2f(A.bias[side][(size_t)e * A.b + j]) : 0.f;
  }
}

// The epilogue of one 32-row tile (rows 32 rt .. of the slot) and 32 CT columns
// from j0 on: up and gate hold the wave's accumulators (gate unused unless
// G = 2), lds 32 x (32 CT + 4) floats of the wave's own.
template <int G, int CT>
__device__ __forceinline__ void finish(const BankArgs &A, int row0, int n, int rt, int j0, const float16_t (&up)[CT],
                                       const float16_t (&gate)[CT], const float (&bu)[CT], const float (&bg)[CT],
                                       float *lds) {
  constexpr int kPitch = pitch2<CT>();
  const int lane = threadIdx.x & 63, lr = lane & 31, lh = lane >> 5;
  with_act(A.act, [&](auto act) {
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float v = up[ct][i] + bu[ct];
        if constexpr (G == 2)
          v = activate<decltype(act)::value>(gate[ct][i] + bg[ct]) * v;
        else
          v = activate<decltype(act)::value>(v);
        lds[(8 * (i >> 2) + 4 * lh + (i & 3)) * kPitch + ct * 32 + lr] = v;
      }
  });
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int u = 0; u < 2 * CT; ++u) {
    const int at = u * 64 + lane, row = at / (4 * CT), c8 = at % (4 * CT);
    const int j = j0 + c8 * 8, rr = rt * 32 + row;
    if (rr >= n || j >= A.b) continue;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = lds[row * kPitch + c8 * 8 + i];
    const int64_t yo = (int64_t)(row0 + rr) * A.ldy + j, ro = (int64_t)(row0 + rr) * A.ldr + j;
    if (j + 8 <= A.b) {
      if (A.f32) {
        float *y = (float *)A.y + yo;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          u32x4 o;
          if (A.res) {
            const u32x4 r = *LB_G(const loose128 *, (const float *)A.res + ro + 4 * h);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[4 * h + i] += __uint_as_float(r[i]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = __float_as_uint(v[4 * h + i]);
          *LB_G(loose128 *, y + 4 * h) = o;
        }
      } else {
        u32x4 o;
        if (A.res) {
          const u32x4 r = *LB_G(const loose128 *, (const uint16_t *)A.res + ro);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[2 * i] += h2f((uint16_t)(r[i] & 0xffffu));
            v[2 * i + 1] += h2f((uint16_t)(r[i] >> 16));
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = f2h(v[2 * i]) | ((uint32_t)f2h(v[2 * i + 1]) << 16);
        *LB_G(loose128 *, (uint16_t *)A.y + yo) = o;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (j + i >= A.b) break;
        if (A.f32)
          ((float *)A.y)[yo + i] = v[i] + (A.res ? ((const float *)A.res)[ro + i] : 0.f);
        else
          ((uint16_t *)A.y)[yo + i] = f2h(v[i] + (A.res ? h2f(((const uint16_t *)A.res)[ro + i]) : 0.f));
      }
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Few rows (slots of 16): a workgroup of NW waves computes 16 rows x 16 CT
// columns of all G sides, the waves interleaved over the (side, path, 32-column
// word) parts of K, U of them requested at once; their sums are added in wave
// order through LDS, where a thread finishes two neighbouring columns.  A wave's
// parts of the layer come before those of the gate, so it holds the hi and lo
// sums of one side only.  Bound by
// latency: 4.0 us for one row of 4096 -> 4096 at s = 86 (all of K requested at
// once), 5.0 us for one gated row 4096 -> 11008 at s = 133; 8.8 us for 8 layers
// of it, a row each (9.2 MB).
template <int G, int CT, int NW, int U>
__global__ void __launch_bounds__(NW * 64)
k_bank_second16(BankArgs A) {
  __shared__ __align__(16) float red[NW * G * CT * 256];  // [wave][side][column tile][register][lane]
  const int slot = blockIdx.y, j0 = blockIdx.x * 16 * CT;
  const int w = wave_id(), lane = threadIdx.x & 63, lr = lane & 15, o = lane >> 4;
  int e, row0, n;
  if (!find_slot(A, A.slot0 + slot, e, row0, n)) return;
  const LayerDesc D0 = layer_of(A, 0, e), D1 = layer_of(A, G - 1, e);

  const int nit = A.P * A.Wk, items = G * nit;
  unsigned jc[CT];
  float4_t acc[CT], low[CT];  // hi and lo sums of the side in hand
  const auto clear = [&]() {
#pragma unroll
    for (int c = 0; c < CT; ++c) acc[c] = low[c] = float4_t{0.f, 0.f, 0.f, 0.f};
  };
  clear();
#pragma unroll
  for (int c = 0; c < CT; ++c) jc[c] = min(j0 + 16 * c + lr, A.b16 - 1);
  int side = 0;
  const auto next_side = [&]() {  // the side's sums to LDS
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        red[(((w * G + side) * CT + ct) * 4 + i) * 64 + lane] = fmaf(low[ct][i], 0x1p-11f, acc[ct][i]);
    clear();
    ++side;
  };
  // the lane's 8 latent columns of a word: block o / 2, half o % 2
  const uint16_t *tp = A.T + (size_t)slot * items * 2048 + (o >> 1) * 1024 + ((o & 1) * 32 + lr) * 8;
  for (int x0 = w; x0 < items; x0 += U * NW) {
    u32x4 t[U][2];  // [plane]
    uint32_t wd[U][CT];
    uint16_t hv[U][CT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int x = min(x0 + u * NW, items - 1);  // past the end: read, not used
      const int q = G == 2 && x >= nit, it = x - q * nit, pp = it >= A.Wk;
#pragma unroll
      for (int f = 0; f < 2; ++f) t[u][f] = *LB_G(gu128, tp + (size_t)x * 2048 + f * 512);
      const gu32 row = (q ? D1.su : D0.su) + (size_t)it * A.b16;
      const gu16 h = (q ? D1.h : D0.h) + (size_t)pp * A.b16;
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        wd[u][c] = row[jc[c]];
        hv[u][c] = h[jc[c]];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int x = x0 + u * NW;
      if (x >= items) break;
      if (G == 2 && side == 0 && x >= nit) next_side();
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        const half8_t b = flip(splat(hv[u][ct] | ((uint32_t)hv[u][ct] << 16)), wd[u][ct] << (4 * o));
        acc[ct] = __builtin_amdgcn_mfma_f32_16x16x32_f16(as_h8(t[u][0]), b, acc[ct], 0, 0, 0);
        low[ct] = __builtin_amdgcn_mfma_f32_16x16x32_f16(as_h8(t[u][1]), b, low[ct], 0, 0, 0);
      }
    }
  }
  while (side < G) next_side();  // a wave may have no part of a side
  __syncthreads();
  for (int id = threadIdx.x; id < n * 8 * CT; id += NW * 64) {
    const int row = id / (8 * CT), c = id % (8 * CT) * 2, j = j0 + c;
    if (j >= A.b) continue;
    const int at = ((c >> 4) * 4 + (row & 3)) * 64 + (c & 15) + 16 * (row >> 2);
    const bool two = j + 1 < A.b;
    float v[2], g[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[i] = g[i] = 0.f;
#pragma unroll
      for (int q = 0; q < NW; ++q) {
        v[i] += red[q * G * CT * 256 + at + i];
        if constexpr (G == 2) g[i] += red[(q * G + 1) * CT * 256 + at + i];
      }
      const int ji = min(j + i, A.b - 1);
      if (A.bias[0]) v[i] += h2f(A.bias[0][(size_t)e * A.b + ji]);
      if (G == 2 && A.bias[1]) g[i] += h2f(A.bias[1][(size_t)e * A.b + ji]);
    }
    with_act(A.act, [&](auto act) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        v[i] = G == 2 ? activate<decltype(act)::value>(g[i]) * v[i] : activate<decltype(act)::value>(v[i]);
    });
    const int64_t yo = (int64_t)(row0 + row) * A.ldy + j, ro = (int64_t)(row0 + row) * A.ldr + j;
    if (A.f32) {
      float *y = (float *)A.y + yo;
      if (A.res) {
        const float *r = (const float *)A.res + ro;
        v[0] += r[0];
        if (two) v[1] += r[1];
      }
      y[0] = v[0];
      if (two) y[1] = v[1];
    } else {
      uint16_t *y = (uint16_t *)A.y + yo;
      if (A.res) {
        const uint16_t *r = (const uint16_t *)A.res + ro;
        v[0] += h2f(r[0]);
        if (two) v[1] += h2f(r[1]);
      }
      if (two)
        *LB_G(loose32 *, y) = f2h(v[0]) | ((uint32_t)f2h(v[1]) << 16);
      else
        y[0] = f2h(v[0]);
    }
  }
}

// Between the two: a workgroup of 8 waves, 32 rows of one slot x 256 columns.
// Four waves take one half of the words of K, four the other: with gates the
// layer's and the gate's, without the first and the last.  So twice the waves
// share what a row tile of 32 offers, and each expands half the signs.  Every
// wave has 64 columns, hi and lo sums apart.  T and words go through two LDS
// buffers, a word of each half at a time, and from there into two sets of
// registers.  At the end the waves of the two halves exchange sums through LDS,
// each for one of their two column tiles, and finish the other.  128 gated rows
// 4096 -> 11008 at s = 431 take 18.1 us: 10.1e9 flops of hi and lo products, 9
// us at a large library product's rate on all CUs, here on the 172 of 256 that
// have a workgroup.  128 columns a workgroup fill more CUs and expand no more
// signs, but read T twice as often: 18.5 us, 512 rows 24.6 against 21.2.  More
// chunks on their way (rings of 4 and 6: 18.5, 18.8) or two words a chunk, which
// leaves a workgroup a CU (64 layers, 1542 rows: 19.2 against 15.6), are slower.
constexpr int kMidT = 8192, kMidChunk = kMidT + 2048;  // T, words
constexpr int kMidLds = 32768 + 8 * 32 * pitch2<1>() * 4;  // the sums exchanged, the epilogue's rows
static_assert(2 * kMidChunk <= kMidLds, "the chunks fit too");

template <int G>
__global__ void __launch_bounds__(512, 4)
k_bank_second_mid(BankArgs A, int slots) {
  __shared__ __align__(16) unsigned char sm[kMidLds];
  const int ncb = (A.b + 255) >> 8;
  const int tile = xcd_tile(A.span), slot = tile / ncb, cb = tile - slot * ncb;
  const int w = wave_id(), lane = threadIdx.x & 63, lr = lane & 31, lh = lane >> 5;
  const int half = w >> 2, j0 = cb * 256 + (w & 3) * 64;
  if (slot >= slots) return;

  const int nit = A.P * A.Wk;
  const int first = G == 2 ? nit : (nit + 1) >> 1;         // words of the first half; the longer one
  const int count = half ? G * nit - first : first;        // of this wave's
  const int word0 = G == 1 && half ? first : 0, side = G == 2 ? half : 0;  // its first word, within its side
  // the wave's copies of a chunk: 1 KB of its half's T (words past the last
  // read on, T has room behind it), and a word of its columns
  const uint16_t *src = A.T + ((size_t)slot * G * nit + (half ? first : 0)) * 2048 + (w & 3) * 512 + lane * 8;
  auto issue_t = [&](int at) {
    dma16(src, sm + at + w * 1024);
    src += 2048;
  };
  issue_t(0);
  int e, row0, n;
  if (!find_slot(A, A.slot0 + slot, e, row0, n)) {
    wait_loads<0>();  // the copies land before the LDS is left
    return;
  }
  const LayerDesc D = layer_of(A, side, e);
  const unsigned jw = min(j0 + lane, A.b16 - 1);
  auto issue_w = [&](int c, int at) {
    dma4((const void *)(D.su + (size_t)min(word0 + min(c, max(count - 1, 0)), nit - 1) * A.b16 + jw),
         sm + at + kMidT + w * 256);
  };
  issue_w(0, 0);
  if (first > 1) {
    issue_t(kMidChunk);
    issue_w(1, kMidChunk);
  }
  uint32_t hh[2][2];  // [path][column tile], two copies per register
#pragma unroll
  for (int pp = 0; pp < 2; ++pp)
#pragma unroll
    for (int ct = 0; ct < 2; ++ct) {
      const uint16_t h = D.h[(size_t)(pp < A.P ? pp : 0) * A.b16 + min(j0 + ct * 32 + lr, A.b16 - 1)];
      hh[pp][ct] = h | ((uint32_t)h << 16);
    }
  const int jm = j0 + half * 32;  // of its two column tiles the wave finishes this one
  float bu[1], bg[1];
  load_bias<1>(A, 0, e, jm, bu);
  load_bias<1>(A, G - 1, e, jm, bg);
  float16_t acc[2], low[2];
#pragma unroll
  for (int ct = 0; ct < 2; ++ct)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[ct][i] = low[ct][i] = 0.f;

  // chunk c is read from LDS during the products of the one before it
  struct Operands {
    u32x4 t[2][2];  // [half of the word][plane]
    uint32_t wd[2];
  };
  auto read = [&](Operands &o, int at) {
    const u32x4 *tl = reinterpret_cast<const u32x4 *>(sm + at + half * 4096) + lane;
    const uint32_t *wl = reinterpret_cast<const uint32_t *>(sm + at + kMidT + w * 256) + lr;
#pragma unroll
    for (int f = 0; f < 4; ++f) o.t[f >> 1][f & 1] = tl[f * 64];
#pragma unroll
    for (int ct = 0; ct < 2; ++ct) o.wd[ct] = wl[ct * 32];
  };
  auto multiply = [&](const Operands &o, int c) {
    if (c >= count) return;
    const int pp = word0 + c >= A.Wk;
    const int left = A.s - 32 * (word0 + c - pp * A.Wk);
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      if (st == 1 && left <= 16) break;  // padding
#pragma unroll
      for (int ct = 0; ct < 2; ++ct) {
        const half8_t b = flip(splat(pp ? hh[1][ct] : hh[0][ct]), o.wd[ct] << (4 * lh + 8 * st));
        acc[ct] = __builtin_amdgcn_mfma_f32_32x32x16_f16(as_h8(o.t[st][0]), b, acc[ct], 0, 0, 0);
        low[ct] = __builtin_amdgcn_mfma_f32_32x32x16_f16(as_h8(o.t[st][1]), b, low[ct], 0, 0, 0);
      }
    }
  };
  Operands even, odd;
  if (first > 1)  // the chunk has landed: this wave's part, then everybody's
    wait_loads<2>();
  else
    wait_loads<0>();
  lds_barrier();
  read(even, 0);
  auto step = [&](int c, const Operands &now, Operands &next, int at) {  // chunk c, which lay at `at`
    if (c + 1 < first) {
      wait_loads<0>();
      lds_barrier();  // and everybody has read chunk c
      if (c + 2 < first) {
        issue_t(at);
        issue_w(c + 2, at);
      }
      read(next, kMidChunk - at);
    }
    multiply(now, c);
  };
  for (int c = 0; c < first; c += 2) {
    step(c, even, odd, 0);
    if (c + 1 < first) step(c + 1, odd, even, kMidChunk);
  }
#pragma unroll
  for (int ct = 0; ct < 2; ++ct) acc[ct] += low[ct] * 0x1p-11f;
  __syncthreads();
  // a column tile's sums go to the wave of the other half that finishes it
  float4_t *over = reinterpret_cast<float4_t *>(sm) + lane;  // [wave][registers / 4][lane]
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float4_t v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = half ? acc[0][4 * q + i] : acc[1][4 * q + i];
    over[(w * 4 + q) * 64] = v;
  }
  __syncthreads();
  if (jm >= A.b) return;
  float16_t own[1], other[1];
#pragma unroll
  for (int i = 0; i < 16; ++i) own[0][i] = half ? acc[1][i] : acc[0][i];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float4_t v = over[((w ^ 4) * 4 + q) * 64];
#pragma unroll
    for (int i = 0; i < 4; ++i) other[0][4 * q + i] = v[i];
  }
  float *rows = reinterpret_cast<float *>(sm + 32768) + w * 32 * pitch2<1>();
  if constexpr (G == 1) {
    own[0] += other[0];
    finish<1, 1>(A, row0, n, 0, jm, own, other, bu, bg, rows);
  } else if (half) {
    finish<2, 1>(A, row0, n, 0, jm, other, own, bu, bg, rows);
  } else {
    finish<2, 1>(A, row0, n, 0, jm, own, other, bu, bg, rows);
  }
}

// The power of two (its exponent) that brings a column's h into [2^14, 2^15), so
// that 2^-11 h is exact too: that of the larger of two paths (h0 | h1 << 16), or,
// where a column of the wave has them further apart than 2^16, each path's own.
__device__ __forceinline__ int lift(uint32_t h01, int path) {
  const auto by = [](float h) { return h > 0.f && h < INFINITY ? 15 - __builtin_amdgcn_frexp_expf(h) : 0; };
  const float h0 = fabsf(h2f((uint16_t)h01)), h1 = fabsf(h2f((uint16_t)(h01 >> 16)));
  const float top = fmaxf(h0, h1), low = fminf(h0, h1);
  if (__any(low > 0.f && low < top * 0x1p-16f)) return by(path ? h1 : h0);
  return by(top);
}

// Many rows: a workgroup of 4 waves, 64 rows of one slot, every wave 64 columns
// of all G sides.  T and the sign words are copied into LDS in chunks of two
// 32-column words of a path, the next chunk during the products of one: T once
// for the workgroup, a wave's words by itself.  (Three or four chunks on their
// way, longer ones, a chunk's first operands read before the last products of
// the one before it, or 8 waves and 512 columns changed nothing or cost up to
// 8%.)  With two waves on a SIMD (G = 2; four with G = 1) a wave issues an
// instruction every four or five cycles at best, so besides the products what
// counts is instructions: per 16 columns and column tile 4 shifts and 4 sign
// flips (8 with G = 1), shared by two row tiles, and everything that is not per
// product is out of the loop.  4096 gated rows of 4096 -> 11008 at s = 133 take
// 119 to 132 us, as the clock allows: hi and lo products are 104e9 flops, 47 us
// of it.  (Without its epilogue the kernel took 98 us of 122, without products
// 59, when one sum held hi and lo.)  8192 rows of 11008 -> 4096 in 8 layers
// (G = 1) take 49 to 52 us.
// With gates the lo sums of the side in hand have registers of their own (240 of
// 256).  Without, that would leave two waves on a SIMD instead of four (58 us),
// so one sum takes hi h and lo 2^-11 h, both scaled by the column's `lift`, which
// is divided out at the end: powers of two, exact throughout.
constexpr int kW2T = 16384, kW2Chunk = kW2T + 2048;                              // T, words
constexpr int kW2Lds = 2 * kW2Chunk;
static_assert(kW2Lds >= 4 * 32 * pitch2<2>() * 4, "the epilogue's rows fit");

template <int G>
__global__ void __launch_bounds__(256, G == 1 ? 4 : 2)
k_bank_second_wide(BankArgs A, int slots) {
  __shared__ __align__(16) unsigned char sm[kW2Lds];
  const int ncb = (A.b + 255) >> 8;
  const int tile = xcd_tile(A.span), slot = tile / ncb, cb = tile - slot * ncb;
  const int w = wave_id(), lane = threadIdx.x & 63, lr = lane & 31, lh = lane >> 5;
  const int j0 = (cb * 4 + w) * 64;
  if (slot >= slots) return;

  const int nch = (A.Wk + 1) >> 1;  // chunks of a path
  // The wave's copies of a chunk, at addresses that only advance: one word of T
  // of one row tile (past a path's last word it reads on, T has room behind
  // it), and two words of its own columns (the last one again past it).  T does
  // not depend on the expert, so its first chunk is on its way before the slot
  // is looked up.
  const uint16_t *src = A.T + ((size_t)(slot * 2 + (w >> 1)) * G * A.P * A.Wk + (w & 1)) * 2048 + lane * 8;
  int fpath = 0, fc = 0, fs = 0;  // the next chunk's path (of all sides), number in it, and place
  auto issue_t = [&]() {
#pragma unroll
    for (int f = 0; f < 4; ++f) dma16(src + f * 512, sm + fs + (w * 4 + f) * 1024);
  };
  issue_t();
  int e, row0, n;
  if (!find_slot(A, A.slot0 + slot, e, row0, n)) {
    wait_loads<0>();  // the copies land before the LDS is left
    return;
  }
  const LayerDesc D0 = layer_of(A, 0, e), D1 = layer_of(A, G - 1, e);
  const unsigned jw = min(j0 + lane, A.b16 - 1);
  gu32 row = D0.su;  // of the next word
  auto issue_w = [&]() {
    const int left = A.Wk - fc * 2;  // words of the path from here on
#pragma unroll
    for (int i = 0; i < 2; ++i)
      dma4((const void *)(row + (size_t)min(i, left - 1) * A.b16 + jw), sm + fs + kW2T + (w * 2 + i) * 256);
    const int step = min(2, left);
    row += (size_t)step * A.b16;
    src += step * 2048;
    if (++fc == nch) {
      fc = 0;
      if (++fpath == A.P) row = D1.su;
    }
    fs ^= kW2Chunk;
  };
  issue_w();
  uint32_t hv[G][2];  // of the column tiles' two paths (one path: twice the same)
#pragma unroll
  for (int q = 0; q < G; ++q)
#pragma unroll
    for (int ct = 0; ct < 2; ++ct) {
      const gu16 h = (q ? D1.h : D0.h) + min(j0 + ct * 32 + lr, A.b16 - 1);
      hv[q][ct] = h[0] | ((uint32_t)h[(size_t)(A.P - 1) * A.b16] << 16);
    }
  float16_t acc[G][2][2];
#pragma unroll
  for (int q = 0; q < G; ++q)
#pragma unroll
    for (int rt = 0; rt < 2; ++rt)
#pragma unroll
      for (int ct = 0; ct < 2; ++ct)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[q][rt][ct][i] = 0.f;

  const int paths = G * A.P;
  int at = 0;
#pragma unroll
  for (int q = 0; q < G; ++q) {
    float16_t low[2][2];  // lo sums, with gates
    if constexpr (G == 2) {
#pragma unroll
      for (int rt = 0; rt < 2; ++rt)
#pragma unroll
        for (int ct = 0; ct < 2; ++ct)
#pragma unroll
          for (int i = 0; i < 16; ++i) low[rt][ct][i] = 0.f;
    }
    for (int pp = 0; pp < A.P; ++pp) {
      uint32_t hh[2], hl[2];  // the path's h and, without gates, 2^-11 h: two copies per register
#pragma unroll
      for (int ct = 0; ct < 2; ++ct) {
        uint16_t h = (uint16_t)(pp ? hv[q][ct] >> 16 : hv[q][ct]);
        if constexpr (G == 1) {
          const int by = lift(hv[q][ct], pp);
          const float hf = ldexpf(h2f(h), by);
          const uint16_t hs = f2h(hf * 0x1p-11f);
          h = f2h(hf);
          hl[ct] = hs | ((uint32_t)hs << 16);
          const int was = lift(hv[q][ct], 0);
          if (pp && __any(by != was)) {
#pragma unroll
            for (int rt = 0; rt < 2; ++rt) acc[q][rt][ct] *= ldexpf(1.f, by - was);
          }
        }
        hh[ct] = h | ((uint32_t)h << 16);
      }
      for (int c = 0; c < nch; ++c) {
        wait_loads<0>();  // the chunk has landed: this wave's part, then everybody's
        lds_barrier();
        if (fpath < paths) {  // the next, into the place that all have left behind
          issue_t();
          issue_w();
        }
        const u32x4 *tl = reinterpret_cast<const u32x4 *>(sm + at) + lane;
        const uint32_t *wl = reinterpret_cast<const uint32_t *>(sm + at + kW2T + w * 512) + lr;
        at ^= kW2Chunk;
        const int steps = (A.s - 64 * c + 15) >> 4;  // blocks of 16 columns that are not padding
        u32x4 t[2][2][2];                            // [half][row tile][plane]
        uint32_t wd[2];
        auto read = [&](int st) {
#pragma unroll
          for (int rt = 0; rt < 2; ++rt)
#pragma unroll
            for (int k = 0; k < 2; ++k) t[st & 1][rt][k] = tl[(rt * 2 + (st >> 1)) * 256 + ((st & 1) * 2 + k) * 64];
        };
        read(0);
#pragma unroll
        for (int st = 0; st < 4; ++st) {
          if (st >= steps) break;
          if (st < 3) read(st + 1);
          if ((st & 1) == 0) {
#pragma unroll
            for (int ct = 0; ct < 2; ++ct) wd[ct] = wl[(st >> 1) * 64 + ct * 32] << (4 * lh);
          }
#pragma unroll
          for (int ct = 0; ct < 2; ++ct) {
            const uint32_t sh = wd[ct] << (8 * (st & 1));
            const half8_t bh = flip(splat(hh[ct]), sh), bl = G == 1 ? flip(splat(hl[ct]), sh) : bh;
#pragma unroll
            for (int rt = 0; rt < 2; ++rt) {
              acc[q][rt][ct] = __builtin_amdgcn_mfma_f32_32x32x16_f16(as_h8(t[st & 1][rt][0]), bh, acc[q][rt][ct], 0, 0, 0);
              float16_t &lo = G == 1 ? acc[q][rt][ct] : low[rt][ct];
              lo = __builtin_amdgcn_mfma_f32_32x32x16_f16(as_h8(t[st & 1][rt][1]), bl, lo, 0, 0, 0);
            }
          }
        }
      }
    }
    if constexpr (G == 2) {
#pragma unroll
      for (int rt = 0; rt < 2; ++rt)
#pragma unroll
        for (int ct = 0; ct < 2; ++ct) acc[q][rt][ct] += low[rt][ct] * 0x1p-11f;
    } else {
#pragma unroll
      for (int ct = 0; ct < 2; ++ct) {
        const float f = ldexpf(1.f, -lift(hv[q][ct], A.P - 1));
#pragma unroll
        for (int rt = 0; rt < 2; ++rt) acc[q][rt][ct] *= f;
      }
    }
  }
  __syncthreads();
  float *lds = reinterpret_cast<float *>(sm) + w * 32 * pitch2<2>();
  float bu[2], bg[2];
  load_bias<2>(A, 0, e, j0, bu);
  load_bias<2>(A, G - 1, e, j0, bg);
#pragma unroll
  for (int rt = 0; rt < 2; ++rt)
    if (rt * 32 < n && j0 < A.b) finish<G, 2>(A, row0, n, rt, j0, acc[0][rt], acc[G - 1][rt], bu, bg, lds);
}

// ------------------------------------------------------------------ host
constexpr int kMaxExperts = 1024;
constexpr int64_t kMaxRows = (int64_t)1 << 30;
// T of at most this many bytes; longer calls run in windows of slots
constexpr size_t kTBudget = (size_t)256 << 20;

}  // namespace

struct lb_bank {
  int E = 0, G = 1, device = 0;
  lb_layer *first = nullptr;
  int64_t a = 0, b = 0;
  LayerDesc *desc = nullptr;     // [side][layer], on the device
  std::vector<LayerDesc> host;   // the same on the host
  uint16_t *T = nullptr;
  int64_t parts = 0;  // 32-row parts that T holds
  std::vector<void *> retired;
};

namespace {

size_t part_bytes(const lb_bank *B) {
  const Layer &Ly = B->first->ly;
  return (size_t)B->G * Ly.P * Ly.Wk * 2048 * 2;
}

int cu_count(const lb_bank *B) {
  const int n = device_info(B->first).cu_count;
  return n > 0 ? n : 256;
}

// Up to this many rows a call takes slots of 16: while the first product's
// 16 x 16 tiles, all slots full, are a few hundred.  16- against 32-row slots,
// both kernels, 4096 -> 11008 gated at s = 133 (20 words): 32 rows 13.7 against
// 17.6 us, 64 rows 16.5 against 17.8, 96 rows 20.5 against 18.0; at s = 431 (56
// words) 32 rows 17.6 against 24.5, 64 rows 26.8 against 25.4; 4096 -> 4096 at
// s = 86 (6 words) 256 rows 14.2 against 15.7, 512 rows 23.2 against 17.3.
// Grouped rows leave slots part empty: 8 layers 8 rows 18.3 against 22.7, 48 rows
// 25.0 against 24.2, 64 rows 26.5 against 24.1; 64 layers 1024 -> 1407 (8
// words) 96 rows 16.2 against 17.0, 180 rows 18.9 against 17.6.
int64_t few_rows(const lb_bank *B, bool grouped) {
  const Layer &Ly = B->first->ly;
  return (grouped ? 4 : 7) * (int64_t)cu_count(B) / (B->G * Ly.P * Ly.Wk);
}

// The most 32-row parts of T that a call of up to `rows` rows makes, at any
// slot size (16-row slots take a part each), within the budget (at least one
// 64-row slot).
int64_t parts_for(const lb_bank *B, int64_t rows) {
  const int64_t few = std::min(rows, few_rows(B, false)), e = std::min<int64_t>(B->E, rows);
  const int64_t most = std::max((rows / 64 + 1 + e) * 2, few / 16 + 1 + e);
  const int64_t cap = std::max<int64_t>(2, (int64_t)(kTBudget / part_bytes(B)) / 2 * 2);
  return std::min(most, cap);
}

lb_status grow(lb_bank *B, int64_t rows, const char *who, bool in_call, hipStream_t st) {
  const int64_t need = parts_for(B, rows);
  if (need <= B->parts) return LB_OK;
  const std::string pre = std::string(who) + ": ";
  if (in_call) {
    hipStreamCaptureStatus cs = hipStreamCaptureStatusNone;
    const hipError_t e = hipStreamIsCapturing(st, &cs);
    if (e != hipSuccess) return set_error(LB_EHIP, pre + hipGetErrorString(e));
    if (cs != hipStreamCaptureStatusNone)
      return set_error(LB_ENOTREADY, pre + "more rows than reserved while the stream is being captured; call "
                                           "lb_bank_reserve first");
  }
  const int64_t parts = std::max(need, std::min(2 * B->parts, parts_for(B, kMaxRows)));
  void *t = nullptr;
  // the many-row kernels read up to three words past a part's end
  const hipError_t e = hipMalloc(&t, (size_t)parts * part_bytes(B) + 16384);
  if (e != hipSuccess) return set_error(LB_ENOMEM, pre + "hipMalloc: " + hipGetErrorString(e));
  if (B->T) {
    try {
      B->retired.push_back(B->T);
    } catch (...) {
      (void)hipFree(t);
      return set_error(LB_ENOMEM, pre + "host allocation");
    }
  }
  B->T = (uint16_t *)t;
  B->parts = parts;
  return LB_OK;
}

template <int NW>
hipError_t launch_first16(const BankArgs &A, int slots, hipStream_t st) {
  const dim3 grid((unsigned)(A.G * A.P * A.Wk * 2), (unsigned)slots);
  if (A.xvec)
    k_bank_first16<NW, true><<<grid, dim3(NW * 64), 0, st>>>(A);
  else
    k_bank_first16<NW, false><<<grid, dim3(NW * 64), 0, st>>>(A);
  return hipGetLastError();
}

template <int G, int CT, int NW, int U>
hipError_t launch_second16(const BankArgs &A, int slots, hipStream_t st) {
  const dim3 grid((unsigned)((A.b + 16 * CT - 1) / (16 * CT)), (unsigned)slots);
  k_bank_second16<G, CT, NW, U><<<grid, dim3(NW * 64), 0, st>>>(A);
  return hipGetLastError();
}

// The grid of `tiles` tiles in runs for the XCDs, `width` of them to a slot: a
// run is a slot's tiles, or an eighth of all when there are few slots.
unsigned xcd_grid(BankArgs &A, int64_t tiles, int width) {
  A.span = (int)std::max<int64_t>(1, std::min<int64_t>(width, tiles / 16));
  const int64_t runs = (tiles + A.span - 1) / A.span;
  return (unsigned)((runs + 7) / 8 * 8 * A.span);
}

template <int RT, int CT, int NW>
hipError_t launch_first_wide(BankArgs A, int slots, int ncs, hipStream_t st) {
  const dim3 grid(xcd_grid(A, (int64_t)slots * A.G * A.P * ncs, A.G * A.P * ncs));
  constexpr int lds = w1_lds<RT, CT, NW>();
  const void *f = A.xvec ? (const void *)k_bank_first_wide<RT, CT, NW, true> : (const void *)k_bank_first_wide<RT, CT, NW, false>;
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  if (A.xvec)
    k_bank_first_wide<RT, CT, NW, true><<<grid, dim3(NW * 64), lds, st>>>(A, slots, ncs);
  else
    k_bank_first_wide<RT, CT, NW, false><<<grid, dim3(NW * 64), lds, st>>>(A, slots, ncs);
  return hipGetLastError();
}

template <int RT, int NW>
hipError_t launch_first_wide(const BankArgs &A, int slots, int ct, hipStream_t st) {
  const int ncs = (A.Wk + ct - 1) / ct;
  switch (ct) {
    case 1: return launch_first_wide<RT, 1, NW>(A, slots, ncs, st);
    case 2: return launch_first_wide<RT, 2, NW>(A, slots, ncs, st);
    case 3: return launch_first_wide<RT, 3, NW>(A, slots, ncs, st);
    case 4: return launch_first_wide<RT, 4, NW>(A, slots, ncs, st);
    default: return launch_first_wide<RT, 5, NW>(A, slots, ncs, st);
  }
}

// The first product of 32- and 64-row slots: column tiles per workgroup (at most
// five: with RT = 2 160 of 256 registers are sums then), and what a launch
// costs, in workgroups' times of a column tile.  What counts first is how often
// all CUs are filled, then the tiles a workgroup has: the fewest rounds, then
// the fewest tiles.  A round is a workgroup a CU, which is what LDS leaves room
// for with three tiles or more (with 8 waves); two of one or two tiles fit (74 KB
// of LDS at RT = 1), but then share the CU's time: 288 workgroups of two tiles
// take 17.7 us where 256 take 11.4.  4096 -> 11008, gated, s = 133: 256 rows 9.4
// us with one tile, 17 with five; 768 rows 14.0 with three (one round), 17.7 with
// two, 17.9 with five; 2048 rows 21 with five (one round), 30 with two or three.
// A tile alone costs as much as 1.5.  Of grouped calls `slots` is the most that
// their rows can make.
struct FirstPlan {
  int ct;
  int64_t cost;
};
FirstPlan first_plan(const BankArgs &A, int64_t slots, int rt, int cus) {
  FirstPlan best = {1, 0};
  int64_t fewest = INT64_MAX;
  for (int c = 1; c <= 5 && c <= A.Wk; ++c) {
    const int64_t wgs = slots * A.G * A.P * ((A.Wk + c - 1) / c), rounds = (wgs + cus - 1) / cus;
    if (rounds < fewest) {
      fewest = rounds;
      best = {c, rounds * rt * std::max(3, 2 * c)};
    }
  }
  return best;
}

// With more than a round of 64-row workgroups they have 4 waves, so that two
// run on a CU and one's end overlaps the other's products (8192 rows of 4096,
// gated: 54 us against 63 with 8 waves; 270 workgroups of 8192 expert rows of
// 11008: 113 against 122; one round of 4096 rows: 36 against 33).
template <int RT>
hipError_t launch_first_wide(const BankArgs &A, int slots, int cus, hipStream_t st) {
  const int ct = first_plan(A, slots, RT, cus).ct, ncs = (A.Wk + ct - 1) / ct;
  if constexpr (RT == 2)
    if ((int64_t)slots * A.G * A.P * ncs > cus) return launch_first_wide<RT, 4>(A, slots, ct, st);
  return launch_first_wide<RT, 8>(A, slots, ct, st);
}

template <int G>
hipError_t launch_second_mid(BankArgs A, int slots, hipStream_t st) {
  const int ncb = (A.b + 255) / 256;
  const dim3 grid(xcd_grid(A, (int64_t)slots * ncb, ncb));
  k_bank_second_mid<G><<<grid, dim3(512), 0, st>>>(A, slots);
  return hipGetLastError();
}

template <int G>
hipError_t launch_second_wide(BankArgs A, int slots, hipStream_t st) {
  const int ncb = (A.b + 255) / 256;
  const dim3 grid(xcd_grid(A, (int64_t)slots * ncb, ncb));
  k_bank_second_wide<G><<<grid, dim3(256), 0, st>>>(A, slots);
  return hipGetLastError();
}

lb_status run(lb_bank *B, BankArgs A, const char *who, hipStream_t st) {
  const Layer &Ly = B->first->ly;
  const int cus = cu_count(B);
  lb_status gs = grow(B, A.rows, who, true, st);
  if (gs != LB_OK) return gs;
  A.desc = B->desc;
  A.one[0] = B->host[A.e0];
  A.one[1] = B->host[(size_t)(B->G - 1) * B->E + A.e0];
  A.T = B->T;
  A.zero = device_zero(B->first);
  A.E = B->E;
  A.a = (int)Ly.a; A.a16 = (int)Ly.a16; A.b = (int)Ly.b; A.b16 = (int)Ly.b16;
  A.s = (int)Ly.s; A.L = (int)Ly.L; A.P = Ly.P; A.G = B->G; A.R1 = (int)Ly.R1; A.Wk = (int)Ly.Wk;
  A.xvec = A.a % 8 == 0 && A.ldx % 8 == 0 && (uintptr_t)A.x % 16 == 0;
  const int64_t avg = A.offsets ? (A.rows + A.E - 1) / A.E : A.rows;
  // pieces of 64 rows and 512 columns of y: two workgroups of the second product
  const int64_t pieces = (int64_t)(A.rows / 64) * ((A.b + 511) / 512);
  // Slots of 64 share an expanded sign operand between two row tiles, but make
  // half the workgroups, and the second product's have half the waves.  64-
  // against 32-row slots, both kernels: 4096 -> 11008 gated 1024 rows (352 pieces)
  // 56 against 51 us, 2048 rows (704) 101 against 96, 3000 rows (1012) 137 against
  // 149, 4096 rows (1408) 168 against 185; 4096 -> 4096 4096 rows (512) 64 against
  // 57, 8192 rows (1024) 106 against 113, 16384 rows 193 against 218.  Below four a
  // CU they win where 32-row slots cost the first product a round more: 8 layers
  // 11008 -> 4096, 4096 rows (512) 90 against 114 us; not 4096 rows of one layer
  // (102 against 91).
  const auto plan = [&](int lg) {
    const int64_t n = A.offsets ? (A.rows >> lg) + std::min<int64_t>(A.E, A.rows) : (A.rows + (1 << lg) - 1) >> lg;
    return first_plan(A, n, 1 << (lg - 5), cus).cost;
  };
  A.lg = A.rows <= few_rows(B, A.offsets != nullptr) ? 4
         : avg >= 64 && (pieces >= 4 * cus || (pieces >= 2 * cus && plan(6) <= plan(5))) ? 6 : 5;
  const int64_t slots = A.offsets ? (A.rows >> A.lg) + std::min<int64_t>(A.E, A.rows)
                                  : (A.rows + (1 << A.lg) - 1) >> A.lg;
  const int per = A.lg == 6 ? 2 : 1;  // 32-row parts of T per slot
  const int64_t tiles = std::max<int64_t>((int64_t)A.G * A.P * A.Wk, (A.b + 127) / 128);
  const int64_t window =
      std::max<int64_t>(1, std::min<int64_t>({B->parts / per, (int64_t)0x7fffffff / 1024 / tiles, 65535}));
  for (int64_t s0 = 0; s0 < slots; s0 += window) {
    const int ns = (int)std::min<int64_t>(window, slots - s0);
    A.slot0 = (int)s0;
    hipError_t e;
    if (A.lg == 4) {
      e = A.R1 > 4 * kF1U ? launch_first16<8>(A, ns, st) : launch_first16<4>(A, ns, st);
      // 32 columns a workgroup when all of them start at once, else 64 (8
      // experts of 4096 -> 11008, gated, a row each: 9.1 against 11.0 us; one
      // row alone: 5.6 against 5.0 us)
      const bool many = (int64_t)ns * ((A.b + 31) / 32) > 4 * cus;
      if (e == hipSuccess)
        e = A.G == 1 ? (many ? launch_second16<1, 4, 4, 3>(A, ns, st) : launch_second16<1, 2, 4, 3>(A, ns, st))
                     : (many ? launch_second16<2, 4, 4, 3>(A, ns, st) : launch_second16<2, 2, 4, 3>(A, ns, st));
    } else if (A.lg == 5) {
      e = launch_first_wide<1>(A, ns, cus, st);
      if (e == hipSuccess)
        e = A.G == 1 ? launch_second_mid<1>(A, ns, st) : launch_second_mid<2>(A, ns, st);
    } else {
      e = launch_first_wide<2>(A, ns, cus, st);
      if (e == hipSuccess)
        e = A.G == 1 ? launch_second_wide<1>(A, ns, st) : launch_second_wide<2>(A, ns, st);
    }
    if (e != hipSuccess) return set_error(LB_EHIP, std::string(who) + ": " + hipGetErrorString(e));
  }
  return LB_OK;
}

// The checks both calls share.
lb_status check(const lb_bank *B, const BankArgs &A, int64_t rows, int64_t x_rows, int y_type, const char *who) {
  const auto refuse = [who](const char *why) { return set_error(LB_EINVAL, std::string(who) + ": " + why); };
  if (y_type != LB_F16 && y_type != LB_F32) return refuse("y_type must be LB_F16 or LB_F32");
  if (A.act < LB_ACT_NONE || A.act > LB_ACT_SILU) return refuse("unknown activation");
  if (rows < 0 || x_rows < 0 || rows > kMaxRows || x_rows > kMaxRows)
    return refuse("row counts must be in [0, 2^30]");
  if (rows == 0) return LB_OK;
  if (!A.x || !A.y) return refuse("NULL x or y");
  if (x_rows == 0) return refuse("x has no rows");
  if (A.bias[1] && B->G == 1) return refuse("a gate bias needs a bank with gates");
  if (A.ldx < B->a || A.ldy < B->b || (A.res && A.ldr < B->b))
    return refuse("a row stride is smaller than the row");
  if (A.ldx > ((int64_t)1 << 31) || A.ldy > ((int64_t)1 << 31) || A.ldr > ((int64_t)1 << 31))
    return refuse("a row stride exceeds 2^31");
  const int ys = y_type == LB_F32 ? 4 : 2;
  if (((uintptr_t)A.x | (uintptr_t)A.bias[0] | (uintptr_t)A.bias[1]) % 2 || ((uintptr_t)A.y | (uintptr_t)A.res) % ys ||
      ((uintptr_t)A.index | (uintptr_t)A.offsets) % 4)
    return refuse("misaligned pointer");
  const auto strided = [](const void *p, int64_t r, int64_t ld, int64_t n, int size) {
    return Rows{p, r, (size_t)ld * size, (size_t)n * size};
  };
  const auto flat = [](const void *p, int64_t n, int size) { return Rows{p, 1, 0, (size_t)n * size}; };
  const Rows y = strided(A.y, rows, A.ldy, B->b, ys);
  if (meet(strided(A.x, x_rows, A.ldx, B->a, 2), y)) return refuse("x and y overlap");
  if (A.res && !(A.res == A.y && A.ldr == A.ldy) && meet(strided(A.res, rows, A.ldr, B->b, ys), y))
    return refuse("residual and y overlap (they may be the same rows)");
  for (const uint16_t *bias : A.bias)
    if (bias && meet(flat(bias, B->E * B->b, 2), y)) return refuse("a bias and y overlap");
  if ((A.index && meet(flat(A.index, rows, 4), y)) || (A.offsets && meet(flat(A.offsets, B->E + 1, 4), y)))
    return refuse("index or offsets and y overlap");
  return LB_OK;
}

}  // namespace

extern "C" lb_status lb_bank_create(lb_layer *const *layers, lb_layer *const *gates, int n, lb_bank **out) {
  if (!out) return set_error(LB_EINVAL, "lb_bank_create: out is NULL");
  if (!layers) return set_error(LB_EINVAL, "lb_bank_create: layers is NULL");
  if (n < 1 || n > kMaxExperts) return set_error(LB_EINVAL, "lb_bank_create: need 1 to 1024 layers");
  const int G = gates ? 2 : 1;
  for (int i = 0; i < G * n; ++i) {
    const lb_layer *L = i < n ? layers[i] : gates[i - n];
    if (!L) return set_error(LB_EINVAL, "lb_bank_create: NULL layer");
    const Layer &Ly = L->ly, &L0 = layers[0]->ly;
    if (Ly.a != L0.a || Ly.b != L0.b || Ly.s != L0.s || Ly.P != L0.P)
      return set_error(LB_EINVAL, "lb_bank_create: all layers must have the same a, b, s and paths");
    if (Ly.device != L0.device) return set_error(LB_EINVAL, "lb_bank_create: layers on different devices");
    if (!Ly.ready()) return set_error(LB_ENOTREADY, "lb_bank_create: signs/scales not set for every path");
  }
  DeviceGuard dg(layers[0]->ly.device);
  lb_bank *B = nullptr;
  try {
    B = new lb_bank();
    B->host.resize((size_t)G * n);
  } catch (...) {
    delete B;
    return set_error(LB_ENOMEM, "lb_bank_create: host allocation");
  }
  B->E = n;
  B->G = G;
  B->first = layers[0];
  B->device = layers[0]->ly.device;
  B->a = layers[0]->ly.a;
  B->b = layers[0]->ly.b;
  for (int i = 0; i < G * n; ++i) {
    lb_layer *L = i < n ? layers[i] : gates[i - n];
    const lb_status st = ensure_mfma_copies(L, nullptr, true, "lb_bank_create");
    if (st != LB_OK) {
      lb_bank_destroy(B);
      return st;
    }
    B->host[i] = {LB_G(gu32, L->ly.sv1m), LB_G(gu32, L->ly.su2m), LB_G(gu16, L->ly.g), LB_G(gu16, L->ly.l), LB_G(gu16, L->ly.h)};
  }
  hipError_t e = hipMalloc(&B->desc, B->host.size() * sizeof(LayerDesc));
  if (e != hipSuccess) {
    lb_bank_destroy(B);
    return set_error(LB_ENOMEM, std::string("lb_bank_create: hipMalloc: ") + hipGetErrorString(e));
  }
  e = hipMemcpy(B->desc, B->host.data(), B->host.size() * sizeof(LayerDesc), hipMemcpyHostToDevice);
  if (e == hipSuccess) e = hipDeviceSynchronize();
  if (e != hipSuccess) {
    lb_bank_destroy(B);
    return set_error(LB_EHIP, std::string("lb_bank_create: ") + hipGetErrorString(e));
  }
  *out = B;
  return LB_OK;
}

extern "C" lb_status lb_bank_destroy(lb_bank *B) {
  if (!B) return LB_OK;
  DeviceGuard dg(B->device);
  if (B->desc) (void)hipFree(B->desc);
  if (B->T) (void)hipFree(B->T);
  for (void *p : B->retired) (void)hipFree(p);
  delete B;
  return LB_OK;
}

extern "C" lb_status lb_bank_shape(const lb_bank *B, int *n, int *gated, int64_t *a, int64_t *b, int *device) {
  if (!B) return set_error(LB_EINVAL, "lb_bank_shape: NULL bank");
  if (n) *n = B->E;
  if (gated) *gated = B->G == 2;
  if (a) *a = B->a;
  if (b) *b = B->b;
  if (device) *device = B->device;
  return LB_OK;
}

extern "C" lb_status lb_bank_reserve(lb_bank *B, int64_t rows) {
  if (!B) return set_error(LB_EINVAL, "lb_bank_reserve: NULL bank");
  if (rows < 0 || rows > kMaxRows) return set_error(LB_EINVAL, "lb_bank_reserve: rows must be in [0, 2^30]");
  if (rows == 0) return LB_OK;
  DeviceGuard dg(B->device);
  return grow(B, rows, "lb_bank_reserve", false, nullptr);
}

extern "C" lb_status lb_bank_forward(lb_bank *B, int expert, const void *x, int64_t ldx, void *y, int64_t ldy,
                                     int y_type, int64_t M, int act, const void *bias, const void *gate_bias,
                                     const void *residual, int64_t ldr, void *stream) {
  if (!B) return set_error(LB_EINVAL, "lb_bank_forward: NULL bank");
  if (expert < 0 || expert >= B->E) return set_error(LB_EINVAL, "lb_bank_forward: expert out of range");
  BankArgs A = {};
  A.x = (const uint16_t *)x;
  A.y = y;
  A.res = residual;
  A.bias[0] = (const uint16_t *)bias;
  A.bias[1] = (const uint16_t *)gate_bias;
  A.ldx = ldx; A.ldy = ldy; A.ldr = ldr;
  A.act = act;
  A.f32 = y_type == LB_F32;
  A.e0 = expert;
  const lb_status st = check(B, A, M, M, y_type, "lb_bank_forward");
  if (st != LB_OK || M == 0) return st;
  A.rows = A.x_rows = (int)M;
  DeviceGuard dg(B->device);
  return run(B, A, "lb_bank_forward", (hipStream_t)stream);
}

extern "C" lb_status lb_bank_grouped(lb_bank *B, const void *x, int64_t x_rows, int64_t ldx, const int32_t *index,
                                     const int32_t *offsets, int64_t rows, void *y, int64_t ldy, int y_type,
                                     int act, const void *bias, const void *gate_bias, const void *residual,
                                     int64_t ldr, void *stream) {
  if (!B) return set_error(LB_EINVAL, "lb_bank_grouped: NULL bank");
  if (!offsets) return set_error(LB_EINVAL, "lb_bank_grouped: NULL offsets");
  BankArgs A = {};
  A.x = (const uint16_t *)x;
  A.y = y;
  A.res = residual;
  A.index = index;
  A.offsets = offsets;
  A.bias[0] = (const uint16_t *)bias;
  A.bias[1] = (const uint16_t *)gate_bias;
  A.ldx = ldx; A.ldy = ldy; A.ldr = ldr;
  A.act = act;
  A.f32 = y_type == LB_F32;
  const lb_status st = check(B, A, rows, x_rows, y_type, "lb_bank_grouped");
  if (st != LB_OK || rows == 0) return st;
  if (!index && x_rows < rows) return set_error(LB_EINVAL, "lb_bank_grouped: without an index x needs a row for each of the rows");
  A.rows = (int)rows;
  A.x_rows = (int)x_rows;
  DeviceGuard dg(B->device);
  return run(B, A, "lb_bank_grouped", (hipStream_t)stream);
}
