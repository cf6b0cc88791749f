// The end of a block and the beginning of the next, a row at a time: lb_norm.
//
//   u = y, or N(y) post_weight + post_bias       the block's output, normed
//   r' = scale r + gate u                        the residual stream
//   x = N(r') weight + bias                      the next block's input
//
// with N(v) = v / sqrt(mean(v^2) + eps), or (v - m) / sqrt(mean((v - m)^2) +
// eps) about the mean m; every part but y or r may be missing.  All of it is
// fp32: the sums run over the row as it lies in registers (the squares about
// the mean in a second pass over the registers, so nothing cancels), r' is
// normed as it was summed, before its own rounding, and out and x are rounded
// once each.
//
// Bound by reading y and r and writing out and x, each once (4096 rows of 8192
// with a norm on each side: 403 MB in 78 us, 5.1 TB/s, a copy's rate); a single row
// by latency (3.3 us of 4096, of which 2 are a launch).  A thread holds pieces of 8
// neighbouring columns (16 bytes of fp16), so that a row is read and written in wide
// accesses at any alignment.
#include <hip/hip_fp16.h>

#include <algorithm>
#include <string>

#include "lb_internal.h"
#include "lb_norm.h"

namespace {

using namespace lbi;

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
// 16 bytes at an element's alignment (global memory takes them as one access).
typedef u32x4 __attribute__((aligned(2), address_space(1))) loose128;
#define LB_LOOSE(p) ((loose128 *)(uintptr_t)(p))

constexpr int64_t kMaxWidth = 32768;
constexpr int64_t kMaxRows = (int64_t)1 << 30;

struct NormArgs {
  const void *y, *r;
  const uint16_t *gate, *post_weight, *post_bias, *weight, *bias;
  void *out;
  uint16_t *x;
  int64_t ldy, ldr, ldg, ldo, ldx;
  float scale, eps;
  int rows, width, y32, r32, layer, post;
};

__device__ __forceinline__ float h2f(uint16_t v) { return __half2float(__ushort_as_half(v)); }
__device__ __forceinline__ uint32_t f2h(float v) { return __half_as_ushort(__float2half_rn(v)); }

// A thread's piece: the 8 columns from `at` on, of which those from `own` on are
// its own.  The row's last, incomplete piece begins further left instead, among
// its neighbour's columns (a row of 1031 took 5.7 us with single loads for it), as
// do pieces past the row, which own nothing.  A row of fewer than 8 columns is one
// piece at 0.
struct Piece {
  int at, own;
};
__device__ __forceinline__ Piece piece_at(int c, int width) { return {max(0, min(c, width - 8)), c}; }

// 8 fp16 numbers as they lie in memory.
__device__ __forceinline__ u32x4 pack8(const uint16_t *p, int64_t row, Piece a, int width) {
  if (width >= 8) return *LB_LOOSE(p + row + a.at);
  u32x4 q = {0, 0, 0, 0};
  for (int i = 0; i < width; ++i) {
    const uint32_t v = (uint32_t)p[row + i] << (16 * (i & 1));
    if (i < 2)
      q[0] |= v;
    else if (i < 4)
      q[1] |= v;
    else if (i < 6)
      q[2] |= v;
    else
      q[3] |= v;
  }
  return q;
}
__device__ __forceinline__ float unpack(const u32x4 &q, int i) { return h2f((uint16_t)(q[i >> 1] >> (16 * (i & 1)))); }

// The piece of a row at p, fp32 or fp16.
__device__ __forceinline__ void load8(const void *p, int f32, int64_t row, Piece a, int width, float (&v)[8]) {
  if (!f32) {
    const u32x4 q = pack8((const uint16_t *)p, row, a, width);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = unpack(q, i);
  } else if (width >= 8) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const u32x4 q = *LB_LOOSE((const float *)p + row + a.at + 4 * h);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * h + i] = __uint_as_float(q[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < width ? ((const float *)p)[row + i] : 0.f;
  }
}

// Whether column i of the piece is its own; ODD: the width is no multiple of 8.
template <bool ODD>
__device__ __forceinline__ bool owns(Piece a, int i, int width) {
  return ODD ? a.at + i >= a.own && a.at + i < width : a.own < width;
}

__device__ __forceinline__ void store8(void *p, int f32, int64_t row, Piece a, int width, const float (&v)[8]) {
  if (a.at == a.own && width >= 8) {
    if (f32) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        u32x4 q;
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = __float_as_uint(v[4 * h + i]);
        *LB_LOOSE((float *)p + row + a.at + 4 * h) = q;
      }
    } else {
      u32x4 q;
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = f2h(v[2 * i]) | (f2h(v[2 * i + 1]) << 16);
      *LB_LOOSE((uint16_t *)p + row + a.at) = q;
    }
    return;
  }
  if (a.own >= width) return;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (owns<true>(a, i, width)) {
      if (f32)
        ((float *)p)[row + a.at + i] = v[i];
      else
        ((uint16_t *)p)[row + a.at + i] = (uint16_t)f2h(v[i]);
    }
}

// The sum over the wave by DPP moves, in every lane.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, ROWS, 0xf, false));
}
__device__ __forceinline__ float wave_sum(float v) {
  v = dpp_add<0x111, 0xf>(v);  // one, two, four and eight lanes down the row of 16
  v = dpp_add<0x112, 0xf>(v);
  v = dpp_add<0x114, 0xf>(v);
  v = dpp_add<0x118, 0xf>(v);
  v = dpp_add<0x142, 0xa>(v);  // the last lane of a row to the next row
  v = dpp_add<0x143, 0xc>(v);  // that of the first half to the second
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}

// The sum over the NT threads of a row.  part: NT / 64 floats of LDS, another
// set for every call, so that one barrier is enough.
template <int NT>
__device__ __forceinline__ float row_sum(float v, float *part) {
  v = wave_sum(v);
  if constexpr (NT > 64) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int i = 1; i < NT / 64; ++i) v += part[i];
  }
  return v;
}

// A norm's weight and bias, requested with the row itself where registers allow
// it (K < 4): behind the row's sums they would be waited for on their own.
template <int K>
struct Affine {
  u32x4 w[K], b[K];
};
template <int NT, int K>
__device__ __forceinline__ void load_affine(const uint16_t *w, const uint16_t *b, int t, int width, Affine<K> &f) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const Piece a = piece_at((k * NT + t) * 8, width);
    if (w) f.w[k] = pack8(w, 0, a, width);
    if (b) f.b[k] = pack8(b, 0, a, width);
  }
}

// v = N(v) w + b over the row.
template <int NT, int K, bool ODD>
__device__ __forceinline__ void norm_row(const NormArgs &A, float (&v)[K][8], const uint16_t *w, const uint16_t *b,
                                         Affine<K> &f, int t, float *part) {
  float mean = 0.f;
  if (A.layer) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) s += owns<ODD>(piece_at((k * NT + t) * 8, A.width), i, A.width) ? v[k][i] : 0.f;
    mean = row_sum<NT>(s, part) / (float)A.width;
    part += NT / 64;
  }
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const Piece a = piece_at((k * NT + t) * 8, A.width);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float d = v[k][i] - mean;
      v[k][i] = d;
      if (owns<ODD>(a, i, A.width)) s = fmaf(d, d, s);
    }
  }
  const float r = 1.f / sqrtf(row_sum<NT>(s, part) / (float)A.width + A.eps);
  if constexpr (K >= 4) load_affine<NT, K>(w, b, t, A.width, f);
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[k][i] *= r;
      if (w) v[k][i] *= unpack(f.w[k], i);
      if (b) v[k][i] += unpack(f.b[k], i);
    }
}

// NT threads a row, K pieces of 8 columns a thread; a workgroup of 64-thread
// rows has four of them.
template <int NT, int K, bool ODD>
__global__ void __launch_bounds__(NT < 256 ? 256 : NT) k_norm(NormArgs A) {
  constexpr int kRows = NT < 256 ? 256 / NT : 1;
  __shared__ float part[4 * (NT / 64)];
  const int t = threadIdx.x % NT;
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / NT;
  if (kRows > 1 && row >= A.rows) return;  // whole waves, which share nothing
  Affine<K> before, after;
  if constexpr (K < 4) {
    if (A.post) load_affine<NT, K>(A.post_weight, A.post_bias, t, A.width, before);
    if (A.x) load_affine<NT, K>(A.weight, A.bias, t, A.width, after);
  }
  float u[K][8], r[K][8];
  if (A.y) {
#pragma unroll
    for (int k = 0; k < K; ++k) load8(A.y, A.y32, row * A.ldy, piece_at((k * NT + t) * 8, A.width), A.width, u[k]);
  }
  if (A.r) {
#pragma unroll
    for (int k = 0; k < K; ++k) load8(A.r, A.r32, row * A.ldr, piece_at((k * NT + t) * 8, A.width), A.width, r[k]);
  }
  if (A.y) {
    if (A.post) norm_row<NT, K, ODD>(A, u, A.post_weight, A.post_bias, before, t, part);
    if (A.gate) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        float g[8];
        load8(A.gate, 0, row * A.ldg, piece_at((k * NT + t) * 8, A.width), A.width, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[k][i] *= g[i];
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) u[k][i] = 0.f;
  }
  if (A.r) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) u[k][i] = fmaf(A.scale, r[k][i], u[k][i]);
  }
  if (A.out) {
#pragma unroll
    for (int k = 0; k < K; ++k) store8(A.out, A.r32, row * A.ldo, piece_at((k * NT + t) * 8, A.width), A.width, u[k]);
  }
  if (!A.x) return;
  norm_row<NT, K, ODD>(A, u, A.weight, A.bias, after, t, part + 2 * (NT / 64));
#pragma unroll
  for (int k = 0; k < K; ++k) store8(A.x, 0, row * A.ldx, piece_at((k * NT + t) * 8, A.width), A.width, u[k]);
}

template <int NT, int K>
hipError_t launch(const NormArgs &A, hipStream_t st) {
  constexpr int kRows = NT < 256 ? 256 / NT : 1;
  const dim3 grid((unsigned)((A.rows + kRows - 1) / kRows));
  if (A.width % 8)
    k_norm<NT, K, true><<<grid, dim3(NT * kRows), 0, st>>>(A);
  else
    k_norm<NT, K, false><<<grid, dim3(NT * kRows), 0, st>>>(A);
  return hipGetLastError();
}

}  // namespace

extern "C" lb_status lb_norm(int kind, const void *y, int y_type, int64_t ldy, int post, const void *post_weight,
                             const void *post_bias, const void *gate, int64_t ldg, const void *r, int64_t ldr,
                             float scale, int r_type, const void *weight, const void *bias, float eps, void *out,
                             int64_t ldo, void *x, int64_t ldx, int64_t rows, int64_t width, void *stream) {
  const auto refuse = [](const char *why) { return set_error(LB_EINVAL, std::string("lb_norm: ") + why); };
  if (kind != LB_NORM_RMS && kind != LB_NORM_LAYER) return refuse("unknown kind of norm");
  if (y_type != LB_F16 && y_type != LB_F32) return refuse("y_type must be LB_F16 or LB_F32");
  if (r_type != LB_F16 && r_type != LB_F32) return refuse("r_type must be LB_F16 or LB_F32");
  if (rows < 0 || rows > kMaxRows) return refuse("rows must be in [0, 2^30]");
  if (width < 1 || width > kMaxWidth) return refuse("need 1 <= width <= 32768");
  if (!(eps >= 0.f) || !(eps < INFINITY)) return refuse("eps must be finite and not negative");
  if (rows == 0) return LB_OK;
  if (!y && !r) return refuse("needs y or r");
  if (!out && !x) return refuse("needs out or x");
  if (!y && (post || gate)) return refuse("a norm or a gate of y needs y");
  if (!post && (post_weight || post_bias)) return refuse("post_weight and post_bias belong to post");
  if (!x && (weight || bias)) return refuse("weight and bias belong to x");
  const int64_t most = (int64_t)1 << 31;
  if ((y && ldy < width) || (r && ldr < width) || (gate && ldg != 0 && ldg < width) || (out && ldo < width) ||
      (x && ldx < width))
    return refuse("a row stride is smaller than the row");
  if ((y && ldy > most) || (r && ldr > most) || (gate && ldg > most) || (out && ldo > most) || (x && ldx > most))
    return refuse("a row stride exceeds 2^31");
  const int ys = y_type == LB_F32 ? 4 : 2, rs = r_type == LB_F32 ? 4 : 2;
  if ((uintptr_t)y % ys || ((uintptr_t)r | (uintptr_t)out) % rs ||
      ((uintptr_t)gate | (uintptr_t)post_weight | (uintptr_t)post_bias | (uintptr_t)weight | (uintptr_t)bias |
       (uintptr_t)x) % 2)
    return refuse("misaligned pointer");
  const auto strided = [&](const void *p, int64_t ld, int size) {
    return Rows{p, p ? rows : 0, (size_t)ld * size, (size_t)width * size};
  };
  const auto flat = [&](const void *p) { return Rows{p, p ? 1 : 0, 0, (size_t)width * 2}; };
  const Rows yr = strided(y, ldy, ys), rr = strided(r, ldr, rs), orows = strided(out, ldo, rs), xr = strided(x, ldx, 2);
  // a row is read whole before it is written, so the same rows may be both
  const auto same = [](const Rows &a, const Rows &b) { return a.p == b.p && a.pitch == b.pitch && a.width == b.width; };
  if (meet(orows, xr)) return refuse("out and x overlap");
  for (const Rows &w : {orows, xr}) {
    if (meet(yr, w) && !same(yr, w)) return refuse("y and an output overlap (they may be the same rows)");
    if (meet(rr, w) && !same(rr, w)) return refuse("r and an output overlap (they may be the same rows)");
    if (meet(ldg ? strided(gate, ldg, 2) : flat(gate), w)) return refuse("the gate and an output overlap");
    for (const void *p : {post_weight, post_bias, weight, bias})
      if (meet(flat(p), w)) return refuse("a weight or bias and an output overlap");
  }
  NormArgs A = {};
  A.y = y;
  A.r = r;
  A.gate = (const uint16_t *)gate;
  A.post_weight = (const uint16_t *)post_weight;
  A.post_bias = (const uint16_t *)post_bias;
  A.weight = (const uint16_t *)weight;
  A.bias = (const uint16_t *)bias;
  A.out = out;
  A.x = (uint16_t *)x;
  A.ldy = ldy; A.ldr = ldr; A.ldg = ldg; A.ldo = ldo; A.ldx = ldx;
  A.scale = scale;
  A.eps = eps;
  A.width = (int)width;
  A.y32 = y_type == LB_F32;
  A.r32 = r_type == LB_F32;
  A.layer = kind == LB_NORM_LAYER;
  A.post = post != 0;
  // windows of rows keep the grid below 2^31 threads
  const int64_t window = (int64_t)1 << 20;
  for (int64_t r0 = 0; r0 < rows; r0 += window) {
    NormArgs W = A;
    W.rows = (int)std::min(window, rows - r0);
    const auto at = [&](const void *p, int64_t ld, int size) { return p ? (const char *)p + (size_t)r0 * ld * size : nullptr; };
    W.y = at(y, ldy, ys);
    W.r = at(r, ldr, rs);
    W.gate = (const uint16_t *)at(gate, ldg, 2);
    W.out = (void *)at(out, ldo, rs);
    W.x = (uint16_t *)at(x, ldx, 2);
    hipStream_t st = (hipStream_t)stream;
    hipError_t e;
    const NormShape shape = norm_shape(width, W.rows);
    switch (shape.threads * 8 + shape.pieces) {
      case 64 * 8 + 1: e = launch<64, 1>(W, st); break;
      case 64 * 8 + 3: e = launch<64, 3>(W, st); break;
      case 256 * 8 + 1: e = launch<256, 1>(W, st); break;
      case 512 * 8 + 1: e = launch<512, 1>(W, st); break;
      case 512 * 8 + 2: e = launch<512, 2>(W, st); break;
      case 1024 * 8 + 1: e = launch<1024, 1>(W, st); break;
      case 1024 * 8 + 2: e = launch<1024, 2>(W, st); break;
      default: e = launch<1024, 4>(W, st);
    }
    if (e != hipSuccess) return set_error(LB_EHIP, std::string("lb_norm: ") + hipGetErrorString(e));
  }
  return LB_OK;
}
