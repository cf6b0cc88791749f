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
// two fp16 numbers, hi = fp16(w) and lo = fp16(2^11 (w - hi)), multiplied
// by +-h and +-2^-11 h: the pair carries 22 bits of w for every |w| < 65504
// down to 2^-14 (an absolute 2^-36 below), so y is rounded once, at
// the end, whatever the batch size.  With w as one fp16 number the error of
// an fp16 y is 1.4 times that of its own rounding (1.75 times when gated).
//
// Rows are cut into slots of tm rows (32 or 64) of one expert.  Without
// offsets slot i is rows [i tm, (i + 1) tm); with offsets every wave finds
// its slot from the experts' row counts, so the host never waits for them:
// the grid is sized for the most slots that `rows` rows can make,
// rows / tm + min(experts, rows), and workgroups past the last slot leave.
//
// Latent workspace T, per 32-row part of a slot (ps), segment and block of 16
// columns: [hi, lo][column half 2][32 rows][8 fp16], so that an operand load
// of a wave is 1 KB contiguous:
//   T[(((ps nseg + seg) 2 Wk + k16) 2 + plane) 512 + (c8 32 + row) 8 + c].
// Columns past s are zero.
//
// Instruction: v_mfma_f32_32x32x16_f16.  Operand lanes: A[i][k] in lane
// i + 32 (k / 8), element k % 8; B[k][j] in lane j + 32 (k / 8), element
// k % 8; D[i][j] in lane j + 32 ((i / 4) % 2), register 4 (i / 8) + i % 4.
#include <hip/hip_fp16.h>

#include <algorithm>
#include <new>
#include <string>
#include <type_traits>
#include <vector>

#include "lb_internal.h"

#ifndef SD1
#define SD1 3
#endif
#ifndef SD2
#define SD2 4
#endif
#ifndef SCT
#define SCT 4
#endif
namespace {

using namespace lbi;

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
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
  int tm, slot0;  // rows per slot, first slot of this launch
  int act, f32, xvec, yvec;
};

#define LB_G(T, p) ((T)(uintptr_t)(p))

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

// Slot `slot` of the call: its expert, first row and row count (1..tm).
// Uniform over the wave; false past the last slot.  Offsets are clamped to
// [0, rows], so no row outside the call is touched whatever they hold.
__device__ __forceinline__ bool find_slot(const BankArgs &A, int slot, int &e, int &row0, int &n) {
  if (!A.offsets) {
    const int64_t r = (int64_t)slot * A.tm;
    if (r >= A.rows) return false;
    e = A.e0;
    row0 = (int)r;
    n = min(A.tm, A.rows - row0);
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
    const int t = (c + A.tm - 1) / A.tm;
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
      row0 = __builtin_amdgcn_readfirstlane(__shfl(lo, src) + ks * A.tm);
      n = __builtin_amdgcn_readfirstlane(min(A.tm, __shfl(c, src) - ks * A.tm));
      return true;
    }
    base += __shfl(inc, 63);
  }
  return false;
}

// 8 fp16 of an x row from element i on; zeros past a or for a row that is
// not there.
template <bool XV>
__device__ __forceinline__ u32x4 load_x(const BankArgs &A, const uint16_t *row, bool ok, int i) {
  if constexpr (XV) {
    return *LB_G(gu128, ok && i < A.a ? (const void *)(row + i) : A.zero);
  } else {
    uint32_t v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] = *LB_G(gu16, ok && i + e < A.a ? (const void *)(row + i + e) : A.zero);
    }
    u32x4 o;
    o.x = v[0] | (v[1] << 16);
    o.y = v[2] | (v[3] << 16);
    o.z = v[4] | (v[5] << 16);
    o.w = v[6] | (v[7] << 16);
    return o;
  }
}

// ------------------------------------------------------- first product
// One workgroup of 16 waves: 32 rows x 32 latent columns over the whole
// input dimension, wave w on the 32-row chunks w, w + 16, ...; the waves'
// sums are added in wave order through LDS.  Four chunks' operands are
// requested together.
constexpr int kN1Waves = 16, kN1U = 4;

template <bool XV>
__global__ void __launch_bounds__(kN1Waves * 64)
k_bank_first(BankArgs A) {
  __shared__ __align__(16) float red[kN1Waves * 1024];
  const int ntile = A.G * A.P * A.Wk;
  const int sub = blockIdx.x / ntile, tile = blockIdx.x - sub * ntile;
  const int per = A.tm >> 5;
  int e, row0, n;
  if (!find_slot(A, A.slot0 + sub / per, e, row0, n)) return;
  const int part = sub % per;
  row0 += 32 * part;
  n = min(n - 32 * part, 32);
  if (n <= 0) return;
  const int seg = tile / A.Wk, ct = tile - seg * A.Wk;
  const int side = seg / A.P, p = seg - side * A.P;
  const LayerDesc D = A.desc[side * A.E + e];

  const int w = wave_id(), lane = threadIdx.x & 63, lr = lane & 31, lh = lane >> 5;
  const int k = ct * 32 + lr;
  const bool cval = k < A.s;
  const gu32 bw = D.sv + (size_t)p * A.s + k;
  const gu16 g = D.g + (size_t)p * A.a16;
  bool rv = lr < n;
  int64_t r = row0 + lr;
  if (A.index && rv) {
    r = A.index[r];
    rv = r >= 0 && r < A.x_rows;
  }
  const uint16_t *xr = A.x + (rv ? r * A.ldx : 0);

  float16_t acc;
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;
  for (int c0 = w; c0 < A.R1; c0 += kN1Waves * kN1U) {
    uint32_t wd[kN1U];
    u32x4 xv[kN1U][2], gv[kN1U][2];
#pragma unroll
    for (int u = 0; u < kN1U; ++u) {
      const int c = c0 + u * kN1Waves;
      const bool ok = c < A.R1;
      wd[u] = *(ok && cval ? bw + (size_t)c * A.L : LB_G(gu32, A.zero));
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        const int i = c * 32 + st * 16 + lh * 8;
        gv[u][st] = *(i < A.a16 ? (gu128)(g + i) : LB_G(gu128, A.zero));
        xv[u][st] = load_x<XV>(A, xr, rv, i);
      }
    }
#pragma unroll
    for (int u = 0; u < kN1U; ++u)
#pragma unroll
      for (int st = 0; st < 2; ++st)
        acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(
            as_h8(xv[u][st]), flip(gv[u][st], (wd[u] << (4 * lh)) << (8 * st)), acc, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) red[(w * 16 + i) * 64 + lane] = acc[i];
  __syncthreads();
  // thread (w, lane) finishes register w of the tile
  float v = 0.f;
#pragma unroll
  for (int q = 0; q < kN1Waves; ++q) v += red[(q * 16 + w) * 64 + lane];
  __syncthreads();
  v = cval ? v * h2f(D.l[(size_t)p * ((A.s + 7) / 8 * 8) + k]) : 0.f;
  uint16_t *tl = reinterpret_cast<uint16_t *>(red);  // [k16 2][plane 2][c8 2][row 32][8]
  {
    const int row = 8 * (w >> 2) + 4 * lh + (w & 3);
    const int o = (lr >> 4) * 1024 + (((lr >> 3) & 1) * 32 + row) * 8 + (lr & 7);
    const uint16_t hi = f2h(v);
    const float hf = h2f(hi);
    tl[o] = hi;
    tl[o + 512] = isinf(hf) ? (uint16_t)0 : f2h((v - hf) * 2048.f);
  }
  __syncthreads();
  if (threadIdx.x < 256) {
    u32x4 *dst = reinterpret_cast<u32x4 *>(A.T + ((size_t)sub * (A.G * A.P) * A.Wk + tile) * 2048);
    dst[threadIdx.x] = reinterpret_cast<const u32x4 *>(red)[threadIdx.x];
  }
}

// Workgroup barrier for LDS alone: global loads in flight stay in flight.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
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

// Many rows: a workgroup of 8 waves computes 32 RT rows x 32 CT columns of one
// segment over the whole input dimension, wave w on the blocks of 32 inputs
// 2 w, 2 w + 1, 2 w + 16, ... (pairs: whole 128-byte lines of x).  A wave
// shares its operands with no other, so it stages them itself, without
// barriers: x rows, the block's g and its columns' sign words are copied into
// a ring of kW1Ring blocks in the wave's own LDS, all but one in flight (piece
// c of row r in slot c ^ (r / 2) % 4, so that the operand reads meet no bank
// twice).  One expanded sign operand serves RT products.  The waves' sums are
// added in wave order through LDS, 32 columns at a time.  The workgroups of
// one slot run on one XCD (workgroup i runs on XCD i % 8) one after another,
// so its x rows come from that XCD's L2 after the first.
constexpr int kW1Waves = 8, kW1Ring = 4;
template <int RT, int CT>
constexpr int w1_block() { return RT * 2048 + (CT + 1) / 2 * 256 + 64; }  // x, words, g
template <int RT, int CT>
constexpr int w1_lds() {
  return std::max(kW1Waves * kW1Ring * w1_block<RT, CT>(), RT * (kW1Waves * 4096 + 4096));
}

template <int RT, int CT, bool XV>
__global__ void __launch_bounds__(kW1Waves * 64)
k_bank_first_wide(BankArgs A, int slots, int ncs) {
  extern __shared__ __align__(16) unsigned char sm[];
  constexpr int kBlock = w1_block<RT, CT>(), kWords = RT * 2048, kG = kBlock - 64, kPer = 2 * RT + (CT + 1) / 2 + 1;
  const int ncg = A.G * A.P * ncs;
  const int xcd = blockIdx.x & 7, jj = blockIdx.x >> 3;
  const int slot = (jj / ncg) * 8 + xcd, cg = jj % ncg;
  int e, row0, n;
  if (slot >= slots || !find_slot(A, A.slot0 + slot, e, row0, n)) return;
  const int seg = cg / ncs, ct0 = (cg - seg * ncs) * CT;
  const int side = seg / A.P, p = seg - side * A.P;
  const LayerDesc D = A.desc[side * A.E + e];

  const int w = wave_id(), lane = threadIdx.x & 63, lr = lane & 31, lh = lane >> 5;
  unsigned char *ring = sm + w * kW1Ring * kBlock;
  const gu16 g = D.g + (size_t)p * A.a16;
  const gu32 bw = D.sv + (size_t)p * A.s;  // uniform
  unsigned col[(CT + 1) / 2];              // the columns whose words the lane copies
#pragma unroll
  for (int q = 0; q < (CT + 1) / 2; ++q) col[q] = min(ct0 * 32 + q * 64 + lane, A.s - 1);
  // the lane's rows: 16 u + lane / 4, 16 bytes of each
  const int piece = (lane & 3) ^ ((lane >> 3) & 3);
  int xrow[2 * RT];
#pragma unroll
  for (int u = 0; u < 2 * RT; ++u) {
    const int r = 16 * u + (lane >> 2);
    int v = r < n ? row0 + r : -1;
    if (A.index && v >= 0) {
      v = A.index[v];
      if (v >= A.x_rows) v = -1;
    }
    xrow[u] = v;
  }

  float16_t acc[RT][CT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[rt][ct][i] = 0.f;

  // the wave's block number i is block 16 (i / 2) + 2 w + i % 2 of the input
  auto block_of = [&](int i) { return 16 * (i >> 1) + 2 * w + (i & 1); };
  const int nblk = A.R1;
  const int mine = max(0, (nblk - 2 * w + 15) / 16 * 2 - ((nblk - 2 * w) % 16 == 1 ? 1 : 0));
  // copies block i of the wave (kPer loads)
  auto issue = [&](int i) {
    const int kb = block_of(i);
    unsigned char *dst = ring + (i & (kW1Ring - 1)) * kBlock;
    const int k0 = kb * 32 + piece * 8;
#pragma unroll
    for (int u = 0; u < 2 * RT; ++u) {
      const uint16_t *row = A.x + (int64_t)xrow[u] * A.ldx;
      if constexpr (XV)
        dma16(xrow[u] >= 0 && k0 < A.a ? (const void *)(row + k0) : A.zero, dst + u * 1024);
      else
        *reinterpret_cast<u32x4 *>(dst + u * 1024 + lane * 16) = load_x<false>(A, row, xrow[u] >= 0, k0);
    }
    const gu32 wrow = bw + (size_t)kb * A.L;
#pragma unroll
    for (int q = 0; q < (CT + 1) / 2; ++q) dma4((const void *)(wrow + col[q]), dst + kWords + q * 256);
    if (lane < 4) {
      const int i8 = kb * 32 + lane * 8;
      dma16(i8 < A.a16 ? (const void *)(g + i8) : A.zero, dst + kG);
    }
  };
#pragma unroll
  for (int i = 0; i < kW1Ring - 1; ++i)
    if (i < mine) issue(i);
  for (int i = 0; i < mine; ++i) {
    // block i has landed; the later ones may be in flight
    if (XV && i + 2 < mine)
      wait_loads<2 * kPer>();
    else if (XV && i + 1 < mine)
      wait_loads<kPer>();
    else
      wait_loads<0>();
    const unsigned char *blk = ring + (i & (kW1Ring - 1)) * kBlock;
    const u32x4 *xs = reinterpret_cast<const u32x4 *>(blk);
    const uint32_t *ws = reinterpret_cast<const uint32_t *>(blk + kWords);
    const u32x4 *gs = reinterpret_cast<const u32x4 *>(blk + kG);
    uint32_t wd[CT];
    u32x4 gv[2], xv[2][RT];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      gv[t] = gs[2 * t + lh];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) xv[t][rt] = xs[(rt * 32 + lr) * 4 + ((2 * t + lh) ^ ((lr >> 1) & 3))];
    }
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) wd[ct] = ws[ct * 32 + lr] << (4 * lh);
    // into the block read in the round before this
    if (i + kW1Ring - 1 < mine) issue(i + kW1Ring - 1);
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        const half8_t b = flip(gv[t], wd[ct] << (8 * t));
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
          acc[rt][ct] = __builtin_amdgcn_mfma_f32_32x32x16_f16(as_h8(xv[t][rt]), b, acc[rt][ct], 0, 0, 0);
      }
  }
  // sums over the waves and w = l t, a column tile at a time
  float *red = reinterpret_cast<float *>(sm);                                       // [wave][rt][register][lane]
  uint16_t *tl = reinterpret_cast<uint16_t *>(sm + RT * kW1Waves * 4096);           // [rt][2048]
  const int nseg = A.G * A.P;
  __syncthreads();
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    const int tile = ct0 + ct;
    if (tile >= A.Wk) break;  // uniform
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int i = 0; i < 16; ++i) red[((w * RT + rt) * 16 + i) * 64 + lane] = acc[rt][ct][i];
    __syncthreads();
    const int k = tile * 32 + lr;
    const float lk = k < A.s ? h2f(D.l[(size_t)p * ((A.s + 7) / 8 * 8) + k]) : 0.f;
#pragma unroll
    for (int q = 0; q < 2 * RT; ++q) {
      const int idx = q * 512 + threadIdx.x, rt = idx >> 10, i = (idx >> 6) & 15;
      float v = 0.f;
#pragma unroll
      for (int z = 0; z < kW1Waves; ++z) v += red[z * RT * 1024 + idx];
      v = k < A.s ? v * lk : 0.f;
      const int row = 8 * (i >> 2) + 4 * lh + (i & 3);
      const int o = rt * 2048 + (lr >> 4) * 1024 + (((lr >> 3) & 1) * 32 + row) * 8 + (lr & 7);
      const uint16_t hi = f2h(v);
      const float hf = h2f(hi);
      tl[o] = hi;
      tl[o + 512] = isinf(hf) ? (uint16_t)0 : f2h((v - hf) * 2048.f);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < RT * 256; i += 512) {
      const int rt = i >> 8;
      u32x4 *dst = reinterpret_cast<u32x4 *>(A.T + (((size_t)(slot * RT + rt) * nseg + seg) * A.Wk + tile) * 2048);
      dst[i & 255] = reinterpret_cast<const u32x4 *>(tl)[i];
    }
  }
}

// ------------------------------------------------------ second product
// Activations in fp32 on the hardware's exp2 and reciprocal (a step of error
// each): v / (1 + exp(-c)) takes six instructions, where expf and a division
// take some forty, and a wave has 64 of them against 288 matrix products.
__device__ __forceinline__ float exp2_hw(float v) { return __builtin_amdgcn_exp2f(v); }
__device__ __forceinline__ float rcp_hw(float v) { return __builtin_amdgcn_rcpf(v); }
constexpr float kLog2e = 1.4426950408889634f;

template <int ACT>
__device__ __forceinline__ float activate(float v) {
  if constexpr (ACT == LB_ACT_RELU) {
    return v > 0.f || v != v ? v : 0.f;
  } else if constexpr (ACT == LB_ACT_GELU) {
    // v/2 erfc(-v / sqrt 2), erfc by Abramowitz and Stegun 7.1.26 (within 1.5e-7)
    const float z = fabsf(v) * 0.70710678118654752f;
    const float t = rcp_hw(fmaf(0.3275911f, z, 1.f));
    float q = fmaf(1.061405429f, t, -1.453152027f);
    q = fmaf(q, t, 1.421413741f);
    q = fmaf(q, t, -0.284496736f);
    q = fmaf(q, t, 0.254829592f) * t * exp2_hw(-kLog2e * z * z);  // erfc(z)
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

// The epilogue of one 32-row tile (rows 32 rt .. of the slot) and 32 CT columns
// from j0 on: up and gate hold the wave's accumulators (gate unused unless
// G = 2), lds 32 x (32 CT + 4) floats of the wave's own.
template <int G, int CT>
__device__ __forceinline__ void finish(const BankArgs &A, int e, int row0, int n, int rt, int j0,
                                       const float16_t (&up)[CT], const float16_t (&gate)[CT], float *lds) {
  constexpr int kPitch = pitch2<CT>();
  const int lane = threadIdx.x & 63, lr = lane & 31, lh = lane >> 5;
  float bu[CT], bg[CT];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    const int j = j0 + ct * 32 + lr;
    bu[ct] = A.bias[0] && j < A.b ? h2f(A.bias[0][(size_t)e * A.b + j]) : 0.f;
    bg[ct] = G == 2 && A.bias[1] && j < A.b ? h2f(A.bias[1][(size_t)e * A.b + j]) : 0.f;
  }
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
    if (A.yvec && j + 8 <= A.b) {
      if (A.f32) {
        if (A.res) {
          const float4 r0 = reinterpret_cast<const float4 *>((const float *)A.res + ro)[0];
          const float4 r1 = reinterpret_cast<const float4 *>((const float *)A.res + ro)[1];
          v[0] += r0.x; v[1] += r0.y; v[2] += r0.z; v[3] += r0.w;
          v[4] += r1.x; v[5] += r1.y; v[6] += r1.z; v[7] += r1.w;
        }
        float4 *dst = reinterpret_cast<float4 *>((float *)A.y + yo);
        dst[0] = make_float4(v[0], v[1], v[2], v[3]);
        dst[1] = make_float4(v[4], v[5], v[6], v[7]);
      } else {
        if (A.res) {
          const u32x4 r = *reinterpret_cast<const u32x4 *>((const uint16_t *)A.res + ro);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[2 * i] += h2f((uint16_t)(r[i] & 0xffffu));
            v[2 * i + 1] += h2f((uint16_t)(r[i] >> 16));
          }
        }
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = f2h(v[2 * i]) | ((uint32_t)f2h(v[2 * i + 1]) << 16);
        *reinterpret_cast<u32x4 *>((uint16_t *)A.y + yo) = o;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (j + i >= A.b) break;
        if (A.f32) {
          ((float *)A.y)[yo + i] = v[i] + (A.res ? ((const float *)A.res)[ro + i] : 0.f);
        } else {
          ((uint16_t *)A.y)[yo + i] = f2h(v[i] + (A.res ? h2f(((const uint16_t *)A.res)[ro + i]) : 0.f));
        }
      }
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// A workgroup of 4 waves, each 32 RT rows of one slot x 32 CT outputs of all G
// sides, operands straight from T (1 KB contiguous per load) and su2m (one
// word per column and 32 latent columns); the workgroups of a slot lie side
// by side.  The epilogue turns each 32-row tile through the wave's own LDS,
// so that residual loads and y stores are whole 16-byte pieces of rows.
template <int G, int RT, int CT>
__global__ void __launch_bounds__(256)
k_bank_second(BankArgs A) {
  constexpr int kPitch = pitch2<CT>();
  extern __shared__ __align__(16) float smem[];
  const int ncb = (A.b + 128 * CT - 1) / (128 * CT);
  const int slot = blockIdx.x / ncb, cb = blockIdx.x - slot * ncb;
  const int w = wave_id(), lane = threadIdx.x & 63, lr = lane & 31, lh = lane >> 5;
  const int j0 = (cb * 4 + w) * 32 * CT;
  if (j0 >= A.b) return;
  int e, row0, n;
  if (!find_slot(A, A.slot0 + slot, e, row0, n)) return;

  const int nit = A.P * A.Wk;
  float16_t acc[G][RT][CT];
#pragma unroll
  for (int q = 0; q < G; ++q)
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[q][rt][ct][i] = 0.f;

  int jc[CT];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) jc[ct] = min(j0 + ct * 32 + lr, A.b16 - 1);
#pragma unroll
  for (int q = 0; q < G; ++q) {
    const LayerDesc D = A.desc[q * A.E + e];
    const u32x4 *tp[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
      tp[rt] = reinterpret_cast<const u32x4 *>(A.T) + ((size_t)(slot * RT + rt) * G + q) * nit * 256 + lane;
    struct Ops {
      u32x4 t[RT][2][2];  // [k16][plane]
      uint32_t wd[CT];
    };
    auto fetch = [&](int it, Ops &o) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int f = 0; f < 4; ++f) o.t[rt][f >> 1][f & 1] = tp[rt][it * 256 + f * 64];
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) o.wd[ct] = D.su[(size_t)it * A.b16 + jc[ct]];
    };
    Ops c;
    fetch(0, c);
    uint32_t hh[CT], hl[CT];
    for (int it = 0; it < nit; ++it) {
      if (it == 0 || it == A.Wk) {  // a path's h: two copies of it per register
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
          const uint16_t h = D.h[(size_t)(it ? A.b16 : 0) + jc[ct]];
          const uint16_t hs = f2h(h2f(h) * 0x1p-11f);
          hh[ct] = h | ((uint32_t)h << 16);
          hl[ct] = hs | ((uint32_t)hs << 16);
        }
      }
      Ops nx;
      fetch(min(it + 1, nit - 1), nx);
      const int left = A.s - 32 * (it < A.Wk ? it : it - A.Wk);
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        if (st == 1 && left <= 16) break;  // the block's second half is padding
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
          const uint32_t wl = (c.wd[ct] << (4 * lh)) << (8 * st);
          const half8_t bh = flip(splat(hh[ct]), wl);
          const half8_t bl = flip(splat(hl[ct]), wl);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            acc[q][rt][ct] = __builtin_amdgcn_mfma_f32_32x32x16_f16(as_h8(c.t[rt][st][0]), bh, acc[q][rt][ct], 0, 0, 0);
            acc[q][rt][ct] = __builtin_amdgcn_mfma_f32_32x32x16_f16(as_h8(c.t[rt][st][1]), bl, acc[q][rt][ct], 0, 0, 0);
          }
        }
      }
      c = nx;
    }
  }

  float *lds = smem + w * 32 * kPitch;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
    if (rt * 32 < n) finish<G, CT>(A, e, row0, n, rt, j0, acc[0][rt], acc[G - 1][rt], lds);
}

// Many rows: a workgroup of 4 waves, 64 rows of one slot, every wave 32 CT
// columns of all G sides.  T and the sign words are copied into a ring of
// chunks of 64 latent columns in LDS, D - 1 of them in flight: T once for the
// workgroup (a wave a 32-column part of one row tile), a wave's words by
// itself.  An operand read serves CT expanded sign operands, one of those two
// row tiles.
template <int CT>
constexpr int w2_chunk() { return 16384 + CT * 1024; }
template <int CT, int D>
constexpr int w2_lds() { return std::max(D * w2_chunk<CT>(), 4 * 32 * 68 * 4); }

template <int G, int CT, int D>
__global__ void __launch_bounds__(256, 2)
k_bank_second_wide(BankArgs A, int slots) {
  constexpr int kPitch = 68, kPer = 4 + CT;
  extern __shared__ __align__(16) unsigned char sm[];
  const int ncb = (A.b + 128 * CT - 1) / (128 * CT);
  const int xcd = blockIdx.x & 7, jj = blockIdx.x >> 3;  // a slot's workgroups on one XCD, as in the first product
  const int slot = (jj / ncb) * 8 + xcd, cb = jj % ncb;
  const int w = wave_id(), lane = threadIdx.x & 63, lr = lane & 31, lh = lane >> 5;
  const int j0 = (cb * 4 + w) * 32 * CT;
  int e, row0, n;
  if (slot >= slots || !find_slot(A, A.slot0 + slot, e, row0, n)) return;

  const int nit = A.P * A.Wk, nch = (nit + 1) / 2, total = G * nch;  // words, chunks of a side, chunks
  const LayerDesc D0 = A.desc[e], D1 = A.desc[(G - 1) * A.E + e];
  // h (and 2^-11 h) of the lane's columns, two copies per register
  uint32_t hh[G][2][CT], hl[G][2][CT];
#pragma unroll
  for (int q = 0; q < G; ++q)
#pragma unroll
    for (int pp = 0; pp < 2; ++pp)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        const uint16_t h = (q ? D1.h : D0.h)[(size_t)(pp < A.P ? pp : 0) * A.b16 + min(j0 + ct * 32 + lr, A.b16 - 1)];
        const uint16_t hs = f2h(h2f(h) * 0x1p-11f);
        hh[q][pp][ct] = h | ((uint32_t)h << 16);
        hl[q][pp][ct] = hs | ((uint32_t)hs << 16);
      }
  float16_t acc[G][2][CT];
#pragma unroll
  for (int q = 0; q < G; ++q)
#pragma unroll
    for (int rt = 0; rt < 2; ++rt)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[q][rt][ct][i] = 0.f;

  const uint16_t *tb = A.T + ((size_t)(slot * 2 + (w >> 1)) * G) * nit * 2048 + lane * 8;
  unsigned jw[CT / 2];  // the columns whose words the lane copies
#pragma unroll
  for (int c = 0; c < CT / 2; ++c) jw[c] = min(j0 + c * 64 + lane, A.b16 - 1);
  int fq = 0, fc = 0, fslot = 0;  // the next chunk to be copied, and where to
  auto issue = [&]() {  // kPer loads
    unsigned char *dst = sm + fslot * w2_chunk<CT>();
    const uint16_t *src = tb + ((size_t)fq * nit + min(2 * fc + (w & 1), nit - 1)) * 2048;
#pragma unroll
    for (int f = 0; f < 4; ++f) dma16(src + f * 512, dst + (w * 4 + f) * 1024);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const gu32 row = (fq ? D1.su : D0.su) + (size_t)min(2 * fc + i, nit - 1) * A.b16;
#pragma unroll
      for (int c = 0; c < CT / 2; ++c)
        dma4((const void *)(row + jw[c]), dst + 16384 + (w * 2 + i) * CT * 128 + c * 256);
    }
    if (++fc == nch) {
      fc = 0;
      ++fq;
    }
    if (++fslot == D) fslot = 0;
  };
#pragma unroll
  for (int i = 0; i < D - 1; ++i)
    if (i < total) issue();
  int at = 0, done = 0;
#pragma unroll
  for (int q = 0; q < G; ++q) {
    for (int c = 0; c < nch; ++c, ++done) {
      // chunk `done` has landed (this wave's part, then everybody's)
      if (D > 2 && done + D - 2 < total)
        wait_loads<(D - 2) * kPer>();
      else if (D > 3 && done + D - 3 < total)
        wait_loads<(D > 3 ? D - 3 : 0) * kPer>();
      else
        wait_loads<0>();
      lds_barrier();
      if (done + D - 1 < total) issue();  // into the chunk that all have left behind
      const u32x4 *tl = reinterpret_cast<const u32x4 *>(sm + at * w2_chunk<CT>());
      const uint32_t *wl = reinterpret_cast<const uint32_t *>(sm + at * w2_chunk<CT>() + 16384) + w * CT * 64 + lr;
      if (++at == D) at = 0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int it = 2 * c + i;
        if (it >= nit) break;
        const int pp = it >= A.Wk;
        uint32_t wd[CT], ph[CT], pl[CT];
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
          wd[ct] = wl[i * CT * 32 + ct * 32] << (4 * lh);
          ph[ct] = pp ? hh[q][1][ct] : hh[q][0][ct];
          pl[ct] = pp ? hl[q][1][ct] : hl[q][0][ct];
        }
#pragma unroll
        for (int st = 0; st < 2; ++st) {
          if (st == 1 && A.s - 32 * (it - pp * A.Wk) <= 16) break;  // the word's second half is padding
          u32x4 t[2][2];
#pragma unroll
          for (int rt = 0; rt < 2; ++rt)
#pragma unroll
            for (int k = 0; k < 2; ++k) t[rt][k] = tl[(rt * 2 + i) * 256 + (st * 2 + k) * 64 + lane];
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) {
            const half8_t bh = flip(splat(ph[ct]), wd[ct] << (8 * st)), bl = flip(splat(pl[ct]), wd[ct] << (8 * st));
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int rt = 0; rt < 2; ++rt)
                acc[q][rt][ct] = __builtin_amdgcn_mfma_f32_32x32x16_f16(as_h8(t[rt][k]), k ? bl : bh, acc[q][rt][ct],
                                                                        0, 0, 0);
          }
        }
      }
    }
  }
  __syncthreads();
  float *lds = reinterpret_cast<float *>(sm) + w * 32 * kPitch;
#pragma unroll
  for (int rt = 0; rt < 2; ++rt) {
    if (rt * 32 >= n) break;
#pragma unroll
    for (int cp = 0; cp < CT; cp += 2) {
      const float16_t up[2] = {acc[0][rt][cp], acc[0][rt][cp + 1]};
      const float16_t gate[2] = {acc[G - 1][rt][cp], acc[G - 1][rt][cp + 1]};
      if (j0 + cp * 32 < A.b) finish<G, 2>(A, e, row0, n, rt, j0 + cp * 32, up, gate, lds);
    }
  }
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
  LayerDesc *desc = nullptr;
  uint16_t *T = nullptr;
  int64_t parts = 0;  // 32-row parts that T holds
  std::vector<void *> retired;
};

namespace {

size_t part_bytes(const lb_bank *B) {
  const Layer &Ly = B->first->ly;
  return (size_t)B->G * Ly.P * Ly.Wk * 2048 * 2;
}

// The most 32-row parts a call of up to `rows` rows makes, at either slot
// size, within the budget (at least one 64-row slot).
int64_t parts_for(const lb_bank *B, int64_t rows) {
  const int64_t most = (rows / 64 + 1 + std::min<int64_t>(B->E, rows)) * 2;
  const int64_t cap = std::max<int64_t>(2, (int64_t)(kTBudget / part_bytes(B)) / 2 * 2);
  return std::min(most, cap);
}

lb_status grow(lb_bank *B, int64_t rows, const char *who, bool in_call, hipStream_t st) {
  const std::string pre = std::string(who) + ": ";
  const int64_t need = parts_for(B, rows);
  if (need <= B->parts) return LB_OK;
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
  const hipError_t e = hipMalloc(&t, (size_t)parts * part_bytes(B));
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

template <int G, int RT, int CT>
hipError_t launch_second(const BankArgs &A, int slots, hipStream_t st) {
  const int ncb = (A.b + 128 * CT - 1) / (128 * CT);
  const size_t lds = (size_t)4 * 32 * pitch2<CT>() * sizeof(float);
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute((const void *)k_bank_second<G, RT, CT>,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  k_bank_second<G, RT, CT><<<dim3((unsigned)(slots * ncb)), dim3(256), lds, st>>>(A);
  return hipGetLastError();
}

template <int RT, int CT>
hipError_t launch_first_wide(const BankArgs &A, int slots, int ncs, hipStream_t st) {
  const dim3 grid((unsigned)((slots + 7) / 8 * 8 * A.G * A.P * ncs));
  constexpr int lds = w1_lds<RT, CT>();
  const void *f = A.xvec ? (const void *)k_bank_first_wide<RT, CT, true> : (const void *)k_bank_first_wide<RT, CT, false>;
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  if (A.xvec)
    k_bank_first_wide<RT, CT, true><<<grid, dim3(kW1Waves * 64), lds, st>>>(A, slots, ncs);
  else
    k_bank_first_wide<RT, CT, false><<<grid, dim3(kW1Waves * 64), lds, st>>>(A, slots, ncs);
  return hipGetLastError();
}

// Column tiles per workgroup: a segment's tiles in the fewest groups of at
// most five (160 of 256 registers are sums then), spread evenly.
template <int RT>
hipError_t launch_first_wide(const BankArgs &A, int slots, hipStream_t st) {
  const int ncs = (A.Wk + 4) / 5;
  switch ((A.Wk + ncs - 1) / ncs) {
    case 1: return launch_first_wide<RT, 1>(A, slots, ncs, st);
    case 2: return launch_first_wide<RT, 2>(A, slots, ncs, st);
    case 3: return launch_first_wide<RT, 3>(A, slots, ncs, st);
    case 4: return launch_first_wide<RT, 4>(A, slots, ncs, st);
    default: return launch_first_wide<RT, 5>(A, slots, ncs, st);
  }
}

template <int G, int CT, int D>
hipError_t launch_second_wide(const BankArgs &A, int slots, hipStream_t st) {
  const int ncb = (A.b + 128 * CT - 1) / (128 * CT);
  constexpr int lds = w2_lds<CT, D>();
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute((const void *)k_bank_second_wide<G, CT, D>,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  k_bank_second_wide<G, CT, D><<<dim3((unsigned)((slots + 7) / 8 * 8 * ncb)), dim3(256), lds, st>>>(A, slots);
  return hipGetLastError();
}

lb_status run(lb_bank *B, BankArgs A, const char *who, hipStream_t st) {
  const Layer &Ly = B->first->ly;
  const int cus = device_info(B->first).cu_count > 0 ? device_info(B->first).cu_count : 256;
  lb_status gs = grow(B, A.rows, who, true, st);
  if (gs != LB_OK) return gs;
  A.desc = B->desc;
  A.T = B->T;
  A.zero = device_zero(B->first);
  A.E = B->E;
  A.a = (int)Ly.a; A.a16 = (int)Ly.a16; A.b = (int)Ly.b; A.b16 = (int)Ly.b16;
  A.s = (int)Ly.s; A.L = (int)Ly.L; A.P = Ly.P; A.G = B->G; A.R1 = (int)Ly.R1; A.Wk = (int)Ly.Wk;
  A.xvec = A.a % 8 == 0 && A.ldx % 8 == 0 && (uintptr_t)A.x % 16 == 0;
  const int wide = A.f32 ? 4 : 8;
  A.yvec = A.ldy % wide == 0 && (uintptr_t)A.y % 16 == 0 &&
           (!A.res || (A.ldr % wide == 0 && (uintptr_t)A.res % 16 == 0));

  const int64_t avg = A.offsets ? (A.rows + A.E - 1) / A.E : A.rows;
  const int64_t big_wg = (int64_t)(A.rows / 64) * ((A.b + 511) / 512);
  const bool big = avg >= 64 && big_wg >= cus;
  A.tm = big ? 64 : 32;
  const int64_t slots = A.offsets ? A.rows / A.tm + std::min<int64_t>(A.E, A.rows) : (A.rows + A.tm - 1) / A.tm;
  const int per = A.tm / 32, ntile = A.G * A.P * A.Wk;
  const int64_t window = std::min<int64_t>(B->parts / per, (int64_t)0x7fffffff / 64 / std::max(ntile * per, (A.b + 127) / 128));
  for (int64_t s0 = 0; s0 < slots; s0 += window) {
    const int ns = (int)std::min<int64_t>(window, slots - s0);
    A.slot0 = (int)s0;
    const dim3 grid((unsigned)(ns * per * ntile));
    hipError_t e = hipSuccess;
    if (big)
      e = launch_first_wide<2>(A, ns, st);
    else if (A.xvec)
      k_bank_first<true><<<grid, dim3(kN1Waves * 64), 0, st>>>(A);
    else
      k_bank_first<false><<<grid, dim3(kN1Waves * 64), 0, st>>>(A);
    if (e == hipSuccess) e = hipGetLastError();
    if (e == hipSuccess) {
      if (A.G == 1)
        e = big ? launch_second_wide<1, SCT, SD1>(A, ns, st) : launch_second<1, 1, 1>(A, ns, st);
      else
        e = big ? launch_second_wide<2, 2, SD2>(A, ns, st) : launch_second<2, 1, 1>(A, ns, st);
    }
    if (e != hipSuccess) return set_error(LB_EHIP, std::string(who) + ": " + hipGetErrorString(e));
  }
  return LB_OK;
}

// Bytes from the first to the last element of `rows` rows of `n` elements.
size_t extent(int64_t rows, int64_t ld, int64_t n, int size) { return (size_t)((rows - 1) * ld + n) * size; }

// The checks both calls share.
lb_status check(const lb_bank *B, const BankArgs &A, int64_t rows, int64_t x_rows, int y_type, const char *who) {
  const std::string pre = std::string(who) + ": ";
  if (y_type != LB_F16 && y_type != LB_F32) return set_error(LB_EINVAL, pre + "y_type must be LB_F16 or LB_F32");
  if (A.act < LB_ACT_NONE || A.act > LB_ACT_SILU) return set_error(LB_EINVAL, pre + "unknown activation");
  if (rows < 0 || x_rows < 0 || rows > kMaxRows || x_rows > kMaxRows)
    return set_error(LB_EINVAL, pre + "row counts must be in [0, 2^30]");
  if (rows == 0) return LB_OK;
  if (!A.x || !A.y) return set_error(LB_EINVAL, pre + "NULL x or y");
  if (x_rows == 0) return set_error(LB_EINVAL, pre + "x has no rows");
  if (A.bias[1] && B->G == 1) return set_error(LB_EINVAL, pre + "a gate bias needs a bank with gates");
  if (A.ldx < B->a || A.ldy < B->b || (A.res && A.ldr < B->b))
    return set_error(LB_EINVAL, pre + "a row stride is smaller than the row");
  if (A.ldx > ((int64_t)1 << 31) || A.ldy > ((int64_t)1 << 31) || A.ldr > ((int64_t)1 << 31))
    return set_error(LB_EINVAL, pre + "a row stride exceeds 2^31");
  const int ys = y_type == LB_F32 ? 4 : 2;
  if (((uintptr_t)A.x | (uintptr_t)A.bias[0] | (uintptr_t)A.bias[1]) % 2 || ((uintptr_t)A.y | (uintptr_t)A.res) % ys ||
      ((uintptr_t)A.index | (uintptr_t)A.offsets) % 4)
    return set_error(LB_EINVAL, pre + "misaligned pointer");
  const size_t yn = extent(rows, A.ldy, B->b, ys);
  if (overlaps(A.x, extent(x_rows, A.ldx, B->a, 2), A.y, yn)) return set_error(LB_EINVAL, pre + "x and y overlap");
  if (A.res && !(A.res == A.y && A.ldr == A.ldy) && overlaps(A.res, extent(rows, A.ldr, B->b, ys), A.y, yn))
    return set_error(LB_EINVAL, pre + "residual and y overlap (they may be the same rows)");
  for (const uint16_t *bias : A.bias)
    if (bias && overlaps(bias, (size_t)B->E * B->b * 2, A.y, yn))
      return set_error(LB_EINVAL, pre + "a bias and y overlap");
  if ((A.index && overlaps(A.index, (size_t)rows * 4, A.y, yn)) ||
      (A.offsets && overlaps(A.offsets, (size_t)(B->E + 1) * 4, A.y, yn)))
    return set_error(LB_EINVAL, pre + "index or offsets and y overlap");
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
  std::vector<LayerDesc> desc;
  try {
    desc.resize((size_t)G * n);
    B = new lb_bank();
  } catch (...) {
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
    desc[i] = {LB_G(gu32, L->ly.sv1m), LB_G(gu32, L->ly.su2m), LB_G(gu16, L->ly.g), LB_G(gu16, L->ly.l), LB_G(gu16, L->ly.h)};
  }
  hipError_t e = hipMalloc(&B->desc, desc.size() * sizeof(LayerDesc));
  if (e != hipSuccess) {
    lb_bank_destroy(B);
    return set_error(LB_ENOMEM, std::string("lb_bank_create: hipMalloc: ") + hipGetErrorString(e));
  }
  e = hipMemcpy(B->desc, desc.data(), desc.size() * sizeof(LayerDesc), hipMemcpyHostToDevice);
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
