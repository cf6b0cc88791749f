// The paged 8-bit cache of keys and values: its storage and what the kernels
// of lb_cache.hip (append, read) and lb_attend.hip (attention) share.
//
// A page holds P tokens (a power of two, 16 to 256) of KV heads.  Every head
// of a page is a block of its own, keys and values alike: one fp32 scale, and
// P / 16 units of 16 tokens x Dp values, Dp = head_dim rounded up to 32.  A
// value v is kept as the byte rint(v / scale) + 128.  Within a unit the bytes
// lie in the order in which the lanes of a wave want them as operands of the
// 16x16x32 matrix instruction, so that a wave reads a unit in loads of 1 KB
// (a pair of 32 dims: 16 bytes a lane) and, when Dp / 32 is odd, one of 512
// bytes (8 a lane) behind them; lane = 16 G + x, G = 0..3, x = 0..15:
//
//   keys    byte 8 h + j of the lane in pair c: token x, dim 64 c + 32 h + 8 G + j
//   values  byte 4 i + j: token 4 G + j, dim 64 c + 16 i + x
//
// (the last, odd 32 dims: keys byte j, values i = 0, 1 only).  Keys are the
// operand K of S^T = K Q^T with dims as the summed index; values that of
// O^T = V^T P^T with tokens as the summed index, in the order in which S^T's
// result leaves them in the lanes, so that the weights go from one product to
// the other in registers.  Bytes past head_dim are never set; queries are zero
// there, and outputs are not written.
#pragma once

#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <string>
#include <vector>

#include "lb_internal.h"
#include "lb_pages.h"

struct lb_cache {
  int device = 0, cus = 0;
  int64_t pages = 0;
  int P = 0, lg = 0, KV = 0, D = 0, Dp = 0;
  uint8_t *k = nullptr, *v = nullptr;   // pages * KV * (P / 16) units
  float *ks = nullptr, *vs = nullptr;   // pages * KV scales
  void *ws = nullptr;                   // partial results of attention
  size_t ws_bytes = 0;
  std::vector<void *> retired;
};

namespace lbi {

typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
// 16 bytes at an element's alignment (global memory takes them as one access).
typedef u32x4_t __attribute__((aligned(2), address_space(1))) loose128_t;
#define LB_LOOSE128(p) ((lbi::loose128_t *)(uintptr_t)(p))

// The sequence of work item `item` (see first_item, whose value `first`
// receives).  All lanes of a wave look together, 64 sequences a step; -1 before
// the first.
__device__ __forceinline__ int find_sequence(const Sequences &S, int64_t item, int mul, int lg, int extra,
                                             int64_t *first) {
  const int lane = threadIdx.x & 63;
  int found = -1;
  for (int base = 0; base < S.n; base += 64) {
    const int b = base + lane;
    int64_t at = INT64_MAX;
    if (b < S.n) at = first_item(S, b, mul, lg, extra);
    const unsigned long long m = __ballot(at <= item);
    if (m == 0) break;  // (starts do not decrease)
    const int last = 63 - __clzll((long long)m);
    found = base + last;
    *first = __shfl(at, last);
    if (last < 63) break;
  }
  return __builtin_amdgcn_readfirstlane(found);
}

__device__ __forceinline__ float h2f(uint16_t v) { return __half2float(__ushort_as_half(v)); }
__device__ __forceinline__ uint32_t f2h(float v) { return __half_as_ushort(__float2half_rn(v)); }
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// The checks of a call's sequences; rows with a value of the call's own.
lb_status check_sequences(const lb_cache *C, const Sequences &S, const char *who);

}  // namespace lbi
