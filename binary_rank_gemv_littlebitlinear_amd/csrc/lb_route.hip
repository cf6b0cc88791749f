// Routing of tokens to the layers of a bank and the way back: lb_route
// chooses every token's experts and sorts the (token, choice) rows by expert
// for lb_bank_grouped; lb_route_combine adds the experts' outputs up.
//
// For token t with logits z_t (NaN counts as -inf) the choices are the k
// largest logits, equal ones by the lowest expert; p_te = exp(z_te - max z_t);
// weight = p_te / sum over the choices (renormalise) or over all experts.
// Experts at -inf are never chosen: a choice that finds none has expert -1,
// row -1 and weight 0.  The rows of expert e are offsets[e] ..
// offsets[e + 1] - 1, in the order of the tokens.
//
// Choosing takes a wave per token: each lane holds its experts' keys (the
// logit's order as an unsigned number) and the wave takes the largest, of the
// lowest expert that has it, k times.  Sorting is counting: rows per expert of every
// block of tokens, then each block places its own rows behind those of the
// blocks before it, 64 rows of a wave at a time (lanes with the same expert
// find one another by ballots over the bits of its number).  Counts are
// integers and every place is computed, so nothing depends on timing.  Up to
// kOneBlock tokens one workgroup does it all in one launch; more take two.
#include <hip/hip_fp16.h>

#include <algorithm>
#include <iterator>
#include <string>

#include "lb_internal.h"

namespace {

using namespace lbi;

constexpr int kWaves = 16, kThreads = kWaves * 64;
constexpr int kMaxE = 1024, kMaxK = 64;
// Tokens that one workgroup routes alone: 6 of 64 experts take 5.7, 7.6 and
// 11.5 us for 16, 32 and 64 tokens so, and 8.0 and 8.6 us for 32 and 64 in two
// launches (2 of 8 experts: 5.0 and 6.8 against 6.2 and 6.9).
constexpr int kOneBlock = 32;
constexpr int kBlockTokens = 16;  // otherwise a block has at least this many,
constexpr int kBlocks = 256;      // and there are at most this many blocks
constexpr int64_t kMaxRows = (int64_t)1 << 30;

struct RouteArgs {
  const void *logits;
  int64_t ld;
  int T, E, k, renorm, f32, tb;  // tb: tokens per block
  int *ids;
  float *weights;
  int *offsets, *token, *row;
  int *hist;  // [block][E]
};

__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }
__device__ __forceinline__ float h2f(uint16_t v) { return __half2float(__ushort_as_half(v)); }

// Reductions over the wave by DPP moves (a few cycles a step; shuffles through
// LDS made choosing 6 of 64 experts for 16384 tokens take 21 us instead of
// 11.8): lane 63 ends up with the result.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, false);
}
constexpr int kShr1 = 0x111, kShr2 = 0x112, kShr4 = 0x114, kShr8 = 0x118, kBcast15 = 0x142, kBcast31 = 0x143;

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max(v, dpp<kShr1, 0xf>(v));
  v = max(v, dpp<kShr2, 0xf>(v));
  v = max(v, dpp<kShr4, 0xf>(v));
  v = max(v, dpp<kShr8, 0xf>(v));
  v = max(v, dpp<kBcast15, 0xa>(v));
  v = max(v, dpp<kBcast31, 0xc>(v));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

__device__ __forceinline__ float wave_sum(float f) {
  auto add = [&](uint32_t o) { f += __uint_as_float(o); };
  add(dpp<kShr1, 0xf>(__float_as_uint(f)));
  add(dpp<kShr2, 0xf>(__float_as_uint(f)));
  add(dpp<kShr4, 0xf>(__float_as_uint(f)));
  add(dpp<kShr8, 0xf>(__float_as_uint(f)));
  add(dpp<kBcast15, 0xa>(__float_as_uint(f)));
  add(dpp<kBcast31, 0xc>(__float_as_uint(f)));
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(f), 63));
}

// exp(z - top), 1 for the top itself (also when it is infinite).
__device__ __forceinline__ float part(float z, float top) { return z == top ? 1.f : expf(z - top); }

// A logit as an unsigned number of the same order, 0 for what cannot be
// chosen (-inf, NaN); and back.
__device__ __forceinline__ uint32_t key_of(float v) {
  if (!(v > -INFINITY)) return 0u;
  const uint32_t u = __float_as_uint(v + 0.f);  // -0 and 0 are equal
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// The lane's keys of token t: expert i * 64 + lane in key[i].
template <int NV>
__device__ __forceinline__ void load_keys(const RouteArgs &A, int t, uint32_t (&key)[NV]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = i * 64 + lane;
    float v = -INFINITY;
    if (e < A.E) {
      const int64_t o = (int64_t)t * A.ld + e;
      v = A.f32 ? ((const float *)A.logits)[o] : h2f(((const uint16_t *)A.logits)[o]);
    }
    key[i] = key_of(v);
  }
}

// One wave: the choices of token t from its keys.
template <int NV>
__device__ __forceinline__ void choose(const RouteArgs &A, int t, uint32_t (&key)[NV]) {
  const int lane = threadIdx.x & 63;
  float mine = 0.f, all = 0.f, top = 0.f;
  int my_id = -1;
  for (int j = 0; j < A.k; ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) best = max(best, key[i]);
    const uint32_t win = wave_max(best);
    if (win == 0u) break;  // nothing left
    if (j == 0) {
      top = logit_of(win);
      if (!A.renorm) {
#pragma unroll
        for (int i = 0; i < NV; ++i) all += key[i] ? part(logit_of(key[i]), top) : 0.f;
      }
    }
    // the lowest expert that has it
    int id = -1;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const unsigned long long m = __ballot(key[i] == win);
      if (id < 0 && m) id = i * 64 + __ffsll(m) - 1;
    }
    if (lane == j) {
      mine = part(logit_of(win), top);
      my_id = id;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (i * 64 + lane == id) key[i] = 0u;
  }
  const float den = wave_sum(A.renorm ? mine : all);
  if (lane < A.k) {
    A.ids[(int64_t)t * A.k + lane] = my_id;
    A.weights[(int64_t)t * A.k + lane] = my_id >= 0 ? mine / den : 0.f;
  }
}

// The wave's tokens: t, t + kWaves, ... below t1, the next one's logits on
// their way meanwhile.
template <int NV>
__device__ __forceinline__ void choose_tokens(const RouteArgs &A, int t, int t1) {
  if (t >= t1) return;
  uint32_t key[NV];
  load_keys<NV>(A, t, key);
  for (; t < t1; t += kWaves) {
    uint32_t next[NV];
    load_keys<NV>(A, min(t + kWaves, t1 - 1), next);
    choose<NV>(A, t, key);
#pragma unroll
    for (int i = 0; i < NV; ++i) key[i] = next[i];
  }
}

__device__ __forceinline__ void choose_all(const RouteArgs &A, int t, int t1) {
  if (A.E <= 64)
    choose_tokens<1>(A, t, t1);
  else if (A.E <= 256)
    choose_tokens<4>(A, t, t1);
  else
    choose_tokens<16>(A, t, t1);
}

// The lanes whose id equals this lane's (id >= 0), by ballots over its bits.
__device__ __forceinline__ unsigned long long same_id(int id, int bits) {
  unsigned long long m = __ballot(id >= 0);
  for (int b = 0; b < bits; ++b) {
    const unsigned long long v = __ballot((id >> b) & 1);
    m &= (id >> b) & 1 ? v : ~v;
  }
  return m;
}

// The workgroup places the rows of tokens [t0, t1).  before[e]: rows of
// expert e in earlier blocks; total[e]: in all blocks; both in LDS and both
// given unless `alone` (then counted here).
__device__ void place(const RouteArgs &A, int t0, int t1, int *cnt, int *start, int *total, bool alone, bool first) {
  const int tid = threadIdx.x, w = wave_id(), lane = tid & 63;
  const int bits = 32 - __clz(A.E - 1 | 1);
  const int64_t n0 = (int64_t)t0 * A.k;
  const int N = (t1 - t0) * A.k;
  const int per = ((N + kWaves - 1) / kWaves + 63) & ~63;
  const int lo = min(N, w * per), hi = min(N, lo + per);
  for (int i = tid; i < kWaves * A.E; i += kThreads) cnt[i] = 0;
  __syncthreads();
  for (int i = lo; i < hi; i += 64) {
    const int id = i + lane < hi ? A.ids[n0 + i + lane] : -1;
    const unsigned long long m = same_id(id, bits);
    if (id >= 0 && (m & ((1ull << lane) - 1)) == 0) cnt[w * A.E + id] += __popcll(m);
  }
  __syncthreads();
  if (alone) {
    for (int e = tid; e < A.E; e += kThreads) {
      int s = 0;
      for (int q = 0; q < kWaves; ++q) s += cnt[q * A.E + e];
      total[e] = s;
      start[e] = 0;
    }
    __syncthreads();
  }
  // offsets: an exclusive scan of the totals by the first wave
  __shared__ int s_sum;
  if (w == 0) {
    int base = 0;
    for (int eb = 0; eb < A.E; eb += 64) {
      const int e = eb + lane;
      const int c = e < A.E ? total[e] : 0;
      int inc = c;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(inc, d);
        if (lane >= d) inc += v;
      }
      if (e < A.E) {
        const int o = base + inc - c;
        if (first) A.offsets[e] = o;
        int at = o + start[e];
        for (int q = 0; q < kWaves; ++q) {  // where each wave's rows begin
          const int v = cnt[q * A.E + e];
          cnt[q * A.E + e] = at;
          at += v;
        }
      }
      base += __shfl(inc, 63);
    }
    if (lane == 0) {
      s_sum = base;
      if (first) A.offsets[A.E] = base;
    }
  }
  __syncthreads();
  const int64_t all = (int64_t)A.T * A.k;
  for (int i = lo; i < hi; i += 64) {
    const int64_t at = n0 + i + lane;
    const bool in = i + lane < hi;
    const int id = in ? A.ids[at] : -1;
    const unsigned long long m = same_id(id, bits), less = m & ((1ull << lane) - 1);
    int r = -1;
    if (id >= 0) {
      r = cnt[w * A.E + id] + __popcll(less);
      // at < 2^30; r < all unless another call uses the workspace meanwhile
      if ((unsigned)r < all) A.token[r] = (int)((unsigned)at / (unsigned)A.k);
    }
    if (in) A.row[at] = r;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (id >= 0 && less == 0) cnt[w * A.E + id] += __popcll(m);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
  // places that no row took
  for (int64_t i = s_sum + (int64_t)blockIdx.x * kThreads + tid; i < all; i += (int64_t)gridDim.x * kThreads)
    A.token[i] = -1;
}

__global__ void __launch_bounds__(kThreads) k_route_one(RouteArgs A) {
  extern __shared__ int sh[];  // cnt [16][E], start [E], total [E]
  choose_all(A, wave_id(), A.T);
  __threadfence_block();
  __syncthreads();
  place(A, 0, A.T, sh, sh + kWaves * A.E, sh + (kWaves + 1) * A.E, true, true);
}

__global__ void __launch_bounds__(kThreads) k_route_choose(RouteArgs A) {
  extern __shared__ int sh[];  // [E]
  const int t0 = blockIdx.x * A.tb, t1 = min(A.T, t0 + A.tb);
  for (int e = threadIdx.x; e < A.E; e += kThreads) sh[e] = 0;
  choose_all(A, t0 + wave_id(), t1);
  __threadfence_block();
  __syncthreads();
  const int64_t n0 = (int64_t)t0 * A.k;
  for (int i = threadIdx.x; i < (t1 - t0) * A.k; i += kThreads) {
    const int id = A.ids[n0 + i];
    if (id >= 0) atomicAdd(&sh[id], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < A.E; e += kThreads) A.hist[(int64_t)blockIdx.x * A.E + e] = sh[e];
}

__global__ void __launch_bounds__(kThreads) k_route_place(RouteArgs A) {
  extern __shared__ int sh[];
  int *start = sh + kWaves * A.E, *total = start + A.E;
  const int b = blockIdx.x, nb = gridDim.x;
  for (int e = threadIdx.x; e < A.E; e += kThreads) start[e] = total[e] = 0;
  __syncthreads();
  const int ng = max(1, kThreads / A.E), e0 = threadIdx.x % A.E, gq = threadIdx.x / A.E;
  if (gq < ng) {
    int before = 0, all = 0;
    for (int q0 = gq; q0 < nb; q0 += 8 * ng) {
      int v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = q0 + u * ng < nb ? A.hist[(int64_t)(q0 + u * ng) * A.E + e0] : 0;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        all += v[u];
        if (q0 + u * ng < b) before += v[u];
      }
    }
    atomicAdd(&start[e0], before);
    atomicAdd(&total[e0], all);
  }
  __syncthreads();
  const int t0 = b * A.tb;
  place(A, t0, min(A.T, t0 + A.tb), sh, start, total, false, b == 0);
}

// ------------------------------------------------------------- combining
// out[t] = residual[t] + sum_j weights[t, j] y[row[t, j]] in the order of j,
// fp32, rounded once.  Bound by reading y and writing out (8192 tokens of 2
// rows of 4096 and a residual: 269 MB in 51 us, 5.3 TB/s; a large copy, which
// writes as much as it reads, reaches 4.9).  A thread takes 8 neighbouring columns (16 bytes of y) of one
// token.
struct CombineArgs {
  const uint16_t *y;
  const int *row;
  const float *weights;
  const void *res;
  void *out;
  int64_t ldy, ldr, ldo, width;
  int y_rows, T, k, f32, nb;  // nb: workgroups per token
};

// 16 bytes at an element's alignment (global memory takes them as one access).
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 __attribute__((aligned(2), address_space(1))) loose128;
#define LB_LOOSE(p) ((loose128 *)(uintptr_t)(p))

__device__ __forceinline__ void add8(float (&acc)[8], u32x4 q, float w) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc[2 * i] = fmaf(w, h2f((uint16_t)(q[i] & 0xffffu)), acc[2 * i]);
    acc[2 * i + 1] = fmaf(w, h2f((uint16_t)(q[i] >> 16)), acc[2 * i + 1]);
  }
}

__global__ void __launch_bounds__(256) k_route_combine(CombineArgs A) {
  const int t = blockIdx.x / A.nb, c = ((blockIdx.x - t * A.nb) * 256 + threadIdx.x) * 8;
  if (c >= A.width) return;
  const int64_t ro = (int64_t)t * A.ldr + c, oo = (int64_t)t * A.ldo + c;
  const int *row = A.row + (int64_t)t * A.k;
  const float *weights = A.weights + (int64_t)t * A.k;
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  if (c + 8 <= A.width) {
    for (int j = 0; j < A.k; ++j) {
      const int r = row[j];
      if (r < 0 || r >= A.y_rows) continue;
      add8(acc, *LB_LOOSE(A.y + (int64_t)r * A.ldy + c), weights[j]);
    }
    if (A.f32) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        u32x4 o;
        if (A.res) {
          const u32x4 r = *LB_LOOSE((const float *)A.res + ro + 4 * h);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[4 * h + i] += __uint_as_float(r[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = __float_as_uint(acc[4 * h + i]);
        *LB_LOOSE((float *)A.out + oo + 4 * h) = o;
      }
    } else {
      if (A.res) add8(acc, *LB_LOOSE((const uint16_t *)A.res + ro), 1.f);
      u32x4 o;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        o[i] = __half_as_ushort(__float2half_rn(acc[2 * i])) |
               ((uint32_t)__half_as_ushort(__float2half_rn(acc[2 * i + 1])) << 16);
      *LB_LOOSE((uint16_t *)A.out + oo) = o;
    }
    return;
  }
  for (int i = 0; c + i < A.width; ++i) {  // the row's last, incomplete piece
    float v = 0.f;
    for (int j = 0; j < A.k; ++j) {
      const int r = row[j];
      if (r >= 0 && r < A.y_rows) v = fmaf(weights[j], h2f(A.y[(int64_t)r * A.ldy + c + i]), v);
    }
    if (A.f32)
      ((float *)A.out)[oo + i] = v + (A.res ? ((const float *)A.res)[ro + i] : 0.f);
    else
      ((uint16_t *)A.out)[oo + i] =
          __half_as_ushort(__float2half_rn(v + (A.res ? h2f(((const uint16_t *)A.res)[ro + i]) : 0.f)));
  }
}

// ------------------------------------------------------------------ host
int tokens_per_block(int64_t T) { return (int)std::max<int64_t>(kBlockTokens, (T + kBlocks - 1) / kBlocks); }

lb_status route_sizes(int64_t tokens, int experts, int k, const char *who) {
  const std::string pre = std::string(who) + ": ";
  if (experts < 1 || experts > kMaxE) return set_error(LB_EINVAL, pre + "need 1 to 1024 experts");
  if (k < 1 || k > kMaxK || k > experts) return set_error(LB_EINVAL, pre + "need 1 <= k <= min(64, experts)");
  if (tokens < 0 || tokens > kMaxRows / k) return set_error(LB_EINVAL, pre + "tokens * k must be in [0, 2^30]");
  return LB_OK;
}

}  // namespace

extern "C" lb_status lb_route_ws_bytes(int64_t tokens, int experts, int k, uint64_t *bytes) {
  if (!bytes) return set_error(LB_EINVAL, "lb_route_ws_bytes: NULL output");
  const lb_status st = route_sizes(tokens, experts, k, "lb_route_ws_bytes");
  if (st != LB_OK) return st;
  // the most blocks that so many tokens or fewer make
  const int64_t blocks = std::min<int64_t>(kBlocks, (tokens + kBlockTokens - 1) / kBlockTokens);
  *bytes = tokens <= kOneBlock ? 0 : (uint64_t)blocks * experts * 4;
  return LB_OK;
}

extern "C" lb_status lb_route(const void *logits, int logits_type, int64_t ld, int64_t tokens, int experts, int k,
                              int renormalise, int32_t *ids, float *weights, int32_t *offsets, int32_t *token,
                              int32_t *row, void *ws, uint64_t ws_bytes, void *stream) {
  uint64_t need = 0;
  lb_status st = route_sizes(tokens, experts, k, "lb_route");
  if (st == LB_OK) st = lb_route_ws_bytes(tokens, experts, k, &need);
  if (st != LB_OK) return st;
  if (logits_type != LB_F16 && logits_type != LB_F32)
    return set_error(LB_EINVAL, "lb_route: logits_type must be LB_F16 or LB_F32");
  if (!offsets || (tokens && (!logits || !ids || !weights || !token || !row)))
    return set_error(LB_EINVAL, "lb_route: NULL argument");
  if (ld < experts || ld > (int64_t)1 << 31) return set_error(LB_EINVAL, "lb_route: the row stride must be in [experts, 2^31]");
  if (ws_bytes < need || (need && !ws))
    return set_error(LB_EINVAL, "lb_route: workspace too small (needs " + std::to_string(need) + " bytes)");
  if ((uintptr_t)logits % (logits_type == LB_F32 ? 4 : 2) ||
      ((uintptr_t)ids | (uintptr_t)weights | (uintptr_t)offsets | (uintptr_t)token | (uintptr_t)row | (uintptr_t)ws) % 4)
    return set_error(LB_EINVAL, "lb_route: misaligned pointer");
  const int ls = logits_type == LB_F32 ? 4 : 2;
  const size_t n = (size_t)tokens * k * 4;
  const int64_t any = tokens > 0;
  const Rows arrays[] = {{logits, tokens, (size_t)ld * ls, (size_t)experts * ls},
                         {offsets, 1, 0, (size_t)(experts + 1) * 4},
                         {ids, any, 0, n}, {weights, any, 0, n}, {token, any, 0, n}, {row, any, 0, n},
                         {ws, need > 0, 0, (size_t)need}};
  for (const Rows &u : arrays)
    for (const Rows *v = &u + 1; v != std::end(arrays); ++v)
      if (meet(u, *v)) return set_error(LB_EINVAL, "lb_route: two arrays overlap");
  RouteArgs A = {};
  A.logits = logits;
  A.ld = ld;
  A.T = (int)tokens; A.E = experts; A.k = k;
  A.renorm = renormalise != 0;
  A.f32 = logits_type == LB_F32;
  A.tb = tokens_per_block(tokens);
  A.ids = ids; A.weights = weights; A.offsets = offsets; A.token = token; A.row = row;
  A.hist = (int *)ws;
  const size_t lds = (size_t)(kWaves + 2) * experts * 4;
  hipStream_t s = (hipStream_t)stream;
  if (lds > 65536) {
    hipError_t e = hipFuncSetAttribute((const void *)k_route_one, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e == hipSuccess)
      e = hipFuncSetAttribute((const void *)k_route_place, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return set_error(LB_EHIP, std::string("lb_route: ") + hipGetErrorString(e));
  }
  if (tokens <= kOneBlock) {
    k_route_one<<<dim3(1), dim3(kThreads), lds, s>>>(A);
  } else {
    const dim3 grid((unsigned)((tokens + A.tb - 1) / A.tb));
    k_route_choose<<<grid, dim3(kThreads), (size_t)experts * 4, s>>>(A);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return set_error(LB_EHIP, std::string("lb_route: ") + hipGetErrorString(e));
    k_route_place<<<grid, dim3(kThreads), lds, s>>>(A);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return set_error(LB_EHIP, std::string("lb_route: ") + hipGetErrorString(e));
  return LB_OK;
}

extern "C" lb_status lb_route_combine(const void *y, int64_t y_rows, int64_t ldy, const int32_t *row,
                                      const float *weights, int64_t tokens, int k, int64_t width,
                                      const void *residual, int64_t ldr, void *out, int64_t ldo, int out_type,
                                      void *stream) {
  if (out_type != LB_F16 && out_type != LB_F32)
    return set_error(LB_EINVAL, "lb_route_combine: out_type must be LB_F16 or LB_F32");
  if (k < 1 || k > kMaxK) return set_error(LB_EINVAL, "lb_route_combine: need 1 <= k <= 64");
  if (tokens < 0 || tokens > kMaxRows / k || y_rows < 0 || y_rows > kMaxRows)
    return set_error(LB_EINVAL, "lb_route_combine: tokens * k and y_rows must be in [0, 2^30]");
  if (width < 1 || width > (1 << 24)) return set_error(LB_EINVAL, "lb_route_combine: need 1 <= width <= 2^24");
  if (tokens == 0) return LB_OK;
  if (!row || !weights || !out || (y_rows && !y)) return set_error(LB_EINVAL, "lb_route_combine: NULL argument");
  if ((y_rows && ldy < width) || ldo < width || (residual && ldr < width))
    return set_error(LB_EINVAL, "lb_route_combine: a row stride is smaller than the row");
  const int64_t most = (int64_t)1 << 31;
  if (ldy > most || ldo > most || ldr > most)
    return set_error(LB_EINVAL, "lb_route_combine: a row stride exceeds 2^31");
  const int os = out_type == LB_F32 ? 4 : 2;
  if ((uintptr_t)y % 2 || ((uintptr_t)row | (uintptr_t)weights) % 4 || ((uintptr_t)out | (uintptr_t)residual) % os)
    return set_error(LB_EINVAL, "lb_route_combine: misaligned pointer");
  const Rows o = {out, tokens, (size_t)ldo * os, (size_t)width * os};
  const size_t choices = (size_t)tokens * k * 4;
  if (meet({y, y_rows, (size_t)ldy * 2, (size_t)width * 2}, o) || meet({row, 1, 0, choices}, o) ||
      meet({weights, 1, 0, choices}, o))
    return set_error(LB_EINVAL, "lb_route_combine: an input and out overlap");
  if (residual && !(residual == out && ldr == ldo) &&
      meet({residual, tokens, (size_t)ldr * os, (size_t)width * os}, o))
    return set_error(LB_EINVAL, "lb_route_combine: residual and out overlap (they may be the same rows)");
  CombineArgs A = {};
  A.y = (const uint16_t *)y;
  A.row = row;
  A.weights = weights;
  A.res = residual;
  A.out = out;
  A.ldy = ldy; A.ldr = ldr; A.ldo = ldo; A.width = width;
  A.y_rows = (int)y_rows; A.k = k;
  A.f32 = out_type == LB_F32;
  A.nb = (int)((width + 2047) / 2048);
  // windows of tokens keep the grid below 2^31 threads
  const int64_t window = std::max<int64_t>(1, (int64_t)0x7fffffff / 256 / A.nb);
  for (int64_t t0 = 0; t0 < tokens; t0 += window) {
    CombineArgs W = A;
    const int64_t n = std::min(window, tokens - t0);
    W.T = (int)n;
    W.row += t0 * k;
    W.weights += t0 * k;
    W.out = (char *)out + (size_t)t0 * ldo * os;
    if (residual) W.res = (const char *)residual + (size_t)t0 * ldr * os;
    k_route_combine<<<dim3((unsigned)(n * A.nb)), dim3(256), 0, (hipStream_t)stream>>>(W);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return set_error(LB_EHIP, std::string("lb_route_combine: ") + hipGetErrorString(e));
  }
  return LB_OK;
}
