// moe_route.cuh — routing to experts from their logits: softmax or sigmoid scores, a
// balancing bias, groups of experts, top-k, gates (dq_moe_route and the layer's
// routing).
//
// Mathematics.  With score s_e and value v_e = s_e + b_e, the experts of the
// `top_groups` groups with the best score (largest v, or sum of the two largest) are
// candidates, and the k largest v among them are taken, the lowest index first among
// equal ones.  The order is that of exact arithmetic:
//  * Without a bias the scores rise with the logits, so logits are compared.
//  * Else v is computed in fp32 (ex2 and rcp approximations) with a known bound on its error, and
//    wherever two values that the selection has to tell apart are closer than the bound allows, they are formed
//    again to 64 bits, and compared so.  (256 experts with normal logits: one token in a few hundred.  A warp's
//    instruction in 64 bits takes some 60 cycles here, and code that runs once is fetched from far: scores
//    come from pairs of fp32, and only those of the experts in doubt.  All 256 in 64 bits took 25 us,
//    longer than all other tokens together.)
//
// A warp takes a token, eight experts a lane.  A group is 32 / n_groups neighbouring
// lanes, so that its score is a few shuffles; lanes hold ascending experts, so
// that of equal values the lowest lane's, and in it the first, is the lowest
// index.  A lane sorts its values as integer keys whose lowest three bits are the
// place in the lane, then k + 1 rounds take the best head (one warp reduction
// and a vote) and advance that lane's list.
//
// What bounds it: instructions, 773 a token (the rounds 170, keys and sort 100, scores and groups 180), with issue in
// 0.6 of the cycles; a warp of its own for every token, so that the GPU evens out what the doubts cost.
// 16384 tokens of 256 experts, 8 of 4 in 8 groups: 16.5 us (bytes alone: 2.7); 8 tokens 3.0 us, a
// launch and one token's chain.  Eight tokens to a warp, four lanes each, took 560 instructions a token but 21 us:
// too few warps to hide their chains.
#pragma once

#include "common.cuh"
#include "moe_route.h"
#include "pair.cuh"

namespace dqmoe {

struct RouteParams {
  const void* logits;
  int64_t stride;              // elements between two tokens' logits
  int64_t part_stride;         // between two partial sums
  int KS, T, E, k;
  int lane_shift;              // log2 of the lanes per group
  int per, each;               // experts per group and per lane (the last lanes of a group may have fewer)
  int groups, top_groups, top2, sigmoid, renorm;
  float scale;
  const float* bias;
  float* sum_out;
  int32_t* idx;
  float* gate;
};

constexpr float kLog2eR = 1.44269504088896341f;
constexpr float kMostLogit = 3.402823466e38f;

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A float's bits as an unsigned key with the float's order, and back.
__device__ __forceinline__ uint32_t route_key(float f) {
  const uint32_t u = __float_as_uint(f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float route_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}

// (no intermediate leaves fp32's range before the score itself does)
__device__ __forceinline__ float sigmoid_of(float x) {
  const float e = expf(-fabsf(x));
  return (x >= 0.f ? 1.f : e) / (1.f + e);
}

// The expert at place j of a lane.
__device__ __forceinline__ int expert_of(const RouteParams& p, int lane, int j) {
  const int in = lane & ((1 << p.lane_shift) - 1);
  return (lane >> p.lane_shift) * p.per + in * p.each + j;
}
// How many experts a lane has.
__device__ __forceinline__ int lane_experts(const RouteParams& p, int lane) {
  const int in = lane & ((1 << p.lane_shift) - 1);
  return max(0, min(p.each, p.per - in * p.each));
}

template <int DT>
__device__ __forceinline__ float logit_at(const RouteParams& p, int64_t at) {
  float x;
  if (DT == DQ_F32) x = ((const float*)p.logits)[at];
  else if (DT == DQ_F16) x = __half2float(((const __half*)p.logits)[at]);
  else x = __bfloat162float(((const __nv_bfloat16*)p.logits)[at]);
  return x;
}

// A logit as it is used: NaN and -inf take an expert out (as -inf), +inf counts as the largest float.
__device__ __forceinline__ float usable(float x) { return x >= -kMostLogit ? fminf(x, kMostLogit) : -INFINITY; }

// e^x for x <= 0: x = k ln 2 + r, the power series of e^r from its 12th term, in pairs from the 7th on.
static __device__ Pair exp_pair(Pair x) {
  if (!(x.h > -87.f)) return {0.f, 0.f};
  const float k = rintf(x.h * 1.44269504f);
  // ln 2 in 16 bits, whose products with k are exact, and the rest as a pair
  Pair r = add({x.h, x.l}, {__fmul_rn(-k, 0x1.62e4p-1f), 0.f});
  r = add(r, mul({-k, 0.f}, {0x1.7f7d1cp-20f, 0x1.ef357ap-45f}));
  const float f = r.h;
  float t = 1.f / 479001600.f;             // 1 / 12!
  t = fmaf(t, f, 1.f / 39916800.f);
  t = fmaf(t, f, 1.f / 3628800.f);
  t = fmaf(t, f, 1.f / 362880.f);
  t = fmaf(t, f, 1.f / 40320.f);
  // 1 / n! as pairs, n = 7 .. 1
  const float ch[7] = {0x1.a01a02p-13f, 0x1.6c16c2p-10f, 0x1.111112p-7f, 0x1.555556p-5f, 0x1.555556p-3f, 0.5f, 1.f};
  const float cl[7] = {-0x1.7f97fap-39f, -0x1.27d27ep-35f, -0x1.dddddep-32f, -0x1.555556p-30f, -0x1.555556p-28f, 0.f, 0.f};
  Pair y = {t, 0.f};
#pragma unroll
  for (int i = 0; i < 7; ++i) y = add(mul(y, r), {ch[i], cl[i]});
  y = add(mul(y, r), {1.f, 0.f});
  const float s = exp2f(k);
  return {y.h * s, y.l * s};
}
// The score of a logit: a sigmoid, or e^(x - top).
static __device__ __noinline__ Pair score_pair(int sigmoid, float x, float top) {
  if (!sigmoid) return exp_pair(sum(x, -top));
  // e = e^-|x| is the small one of both terms: e / (1 + e), or 1 less that
  const Pair e = exp_pair({-fabsf(x), 0.f});
  const Pair q = divide(e, add({1.f, 0.f}, e));
  return x >= 0.f ? add({1.f, 0.f}, {-q.h, -q.l}) : q;
}
// Below 2^-80, where a pair's second part leaves fp32's range, a score is formed in 64 bits: z as in e^(x - top) / z.
constexpr float kLeastPair = 0x1p-80f;
static __device__ __noinline__ double score_tiny(int sigmoid, float x, float top, Pair z) {
  return sigmoid ? 1.0 / (1.0 + exp(-(double)x)) : exp((double)x - (double)top) / ((double)z.h + (double)z.l);
}
// A score next to 1 is 1 / t for t = 1 + e^-x, or the sum of a softmax's e^(x - top) for the largest itself.  64 bits round t to
// a multiple of 2^-52: scores above 1 - 2^-28 are few values that many logits share, which a pair, rounded once, would tell
// apart.  So t is rounded as it is there, and 1 / t = 1 - d + d^2 - d^3 + d^4 for d = t - 1 < 2^-12 once more.
constexpr float kNearOne = 8.5f;
static __device__ __noinline__ double score_near_one(int sigmoid, float x, Pair z) {
  const Pair e = sigmoid ? exp_pair({-x, 0.f}) : z;
  const double t = (double)e.h + (double)e.l, d = sigmoid ? (1.0 + t) - 1.0 : t - 1.0;
  return (1.0 - d) + d * d * (1.0 - d * (1.0 - d));
}
__device__ __forceinline__ Pair shfl_xor_pair(Pair a, int o) {
  return {__shfl_xor_sync(0xffffffffu, a.h, o), __shfl_xor_sync(0xffffffffu, a.l, o)};
}
// 64-bit values as whole numbers of the same order (compared four times as fast), and back.
typedef long long Key64;
constexpr Key64 kNoKey = -0x7ff0000000000000LL;       // below every finite value's
__device__ __forceinline__ Key64 key64(double x) {
  const Key64 b = __double_as_longlong(x);
  return b ^ ((b >> 63) & 0x7fffffffffffffffLL);
}
__device__ __forceinline__ double value64(Key64 k) { return __longlong_as_double(k ^ ((k >> 63) & 0x7fffffffffffffffLL)); }
// The value of logit x, whose score is e.
__device__ __forceinline__ Key64 key64(Pair e, float bias, int sigmoid, float x, float top, Pair z) {
  const bool near = sigmoid ? x > kNearOne : x == top && z.h < 1.f + 0x1p-12f;
  const double s = near ? score_near_one(sigmoid, x, z)
                   : e.h < kLeastPair ? score_tiny(sigmoid, x, top, z) : (double)e.h + (double)e.l;
  return key64(s + (double)bias);
}
__device__ __forceinline__ Key64 sigmoid_key(float x, float bias) {
  return key64(score_pair(1, x, 0.f), bias, 1, x, 0.f, {1.f, 0.f});
}

// The token's selection in 64 bits: lane i < k returns pick i, and in `live` whether it is a candidate.
// `row`: the token's logits, or `summed`.
template <int DT>
static __device__ __noinline__ int route_exact(const RouteParams& p, const float* summed, int64_t row, int lane, bool& live) {
  const int n = lane_experts(p, lane), e0 = expert_of(p, lane, 0);
  float l[8], top = -INFINITY;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    l[j] = j < n ? usable(summed ? summed[e0 + j] : logit_at<DT>(p, row + e0 + j)) : -INFINITY;
    top = fmaxf(top, l[j]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  Pair e[8], z = {0.f, 0.f};
  Key64 v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    e[j] = {0.f, 0.f};
    if (l[j] > -INFINITY) e[j] = score_pair(p.sigmoid, l[j], top);
    z = add(z, e[j]);
  }
  if (!p.sigmoid) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z = add(z, shfl_xor_pair(z, o));
  }
  Key64 g1 = kNoKey, g2 = kNoKey;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (!p.sigmoid && z.h > 0.f) e[j] = divide(e[j], z);
    // (without a bias logits are compared, which differ where scores of 1 or 0 do not; only sums take scores)
    if (!(l[j] > -INFINITY)) v[j] = kNoKey;
    else if (p.bias || p.top2) v[j] = key64(e[j], p.bias ? __ldg(p.bias + e0 + j) : 0.f, p.sigmoid, l[j], top, z);
    else v[j] = key64((double)(l[j] + 0.f));
    g2 = max(g2, min(g1, v[j]));
    g1 = max(g1, v[j]);
  }
  if (p.top_groups < p.groups) {
#pragma unroll 1
    for (int o = 1; o < 1 << p.lane_shift; o <<= 1) {
      const Key64 a1 = __shfl_xor_sync(0xffffffffu, g1, o), a2 = __shfl_xor_sync(0xffffffffu, g2, o);
      g2 = max(min(g1, a1), max(g2, a2));
      g1 = max(g1, a1);
    }
    const Key64 sc = p.top2 && g2 > kNoKey ? key64(value64(g1) + value64(g2)) : g1;
    const int g = lane >> p.lane_shift;
    int better = 0;
#pragma unroll 1
    for (int x = 0; x < p.groups; ++x) {
      const Key64 y = __shfl_sync(0xffffffffu, sc, x << p.lane_shift);
      better += y > sc || (y == sc && x < g) ? 1 : 0;
    }
    if (better >= p.top_groups) {
#pragma unroll
      for (int j = 0; j < 8; ++j) l[j] = -INFINITY;
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (!p.bias) v[j] = key64((double)(l[j] + 0.f));
    if (!(l[j] > -INFINITY)) v[j] = kNoKey;
  }
  uint32_t left = (1u << n) - 1;           // places that are not taken yet
  int pick = 0;
  live = false;
#pragma unroll 1
  for (int r = 0; r < p.k; ++r) {
    Key64 best = kNoKey;
    int at = 0x7fffffff;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if ((left >> j & 1) && (at == 0x7fffffff || v[j] > best)) {
        best = v[j];
        at = e0 + j;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const Key64 b = __shfl_xor_sync(0xffffffffu, best, o);
      const int a = __shfl_xor_sync(0xffffffffu, at, o);
      if (a != 0x7fffffff && (at == 0x7fffffff || b > best || (b == best && a < at))) {
        best = b;
        at = a;
      }
    }
    if (lane == r) {
      pick = at;
      live = best > kNoKey;
    }
    if (at >= e0 && at < e0 + n) left &= ~(1u << (at - e0));
  }
  return pick;
}

__device__ __forceinline__ void cas_keys(uint32_t& a, uint32_t& b) {
  const uint32_t hi = max(a, b), lo = min(a, b);
  a = hi;
  b = lo;
}

// Batcher's odd-even merge sort of 8, descending
__device__ __forceinline__ void sort8(uint32_t (&key)[8]) {
#define DQ_CAS(a, b) cas_keys(key[a], key[b])
  DQ_CAS(0, 1); DQ_CAS(2, 3); DQ_CAS(4, 5); DQ_CAS(6, 7);
  DQ_CAS(0, 2); DQ_CAS(1, 3); DQ_CAS(4, 6); DQ_CAS(5, 7);
  DQ_CAS(1, 2); DQ_CAS(5, 6);
  DQ_CAS(0, 4); DQ_CAS(1, 5); DQ_CAS(2, 6); DQ_CAS(3, 7);
  DQ_CAS(2, 4); DQ_CAS(3, 5);
  DQ_CAS(1, 2); DQ_CAS(3, 4); DQ_CAS(5, 6);
#undef DQ_CAS
}

// The lane's eight logits; FULL: every lane has eight, on a 16-byte boundary.
template <int DT, bool FULL>
__device__ __forceinline__ void load_logits(const RouteParams& p, int64_t at, int n, float (&l)[8]) {
  if (FULL && DT == DQ_F32) {
    const float4* q = (const float4*)((const float*)p.logits + at);
    const float4 a = q[0], b = q[1];
    l[0] = a.x; l[1] = a.y; l[2] = a.z; l[3] = a.w;
    l[4] = b.x; l[5] = b.y; l[6] = b.z; l[7] = b.w;
  } else if (FULL) {
    const uint4 v = *(const uint4*)((const unsigned short*)p.logits + at);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = DT == DQ_F16 ? __half22float2(u32_as_h2(w[j]))
                                    : make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
      l[2 * j] = f.x;
      l[2 * j + 1] = f.y;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) l[j] = j < n ? logit_at<DT>(p, at + j) : -kMostLogit;
  }
}

// How many places the lanes in front have marked in `may`, and all of them.
__device__ __forceinline__ int count_before(uint32_t may, int lane, int& all) {
  int upto = __popc(may);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += u;
  }
  all = __shfl_sync(0xffffffffu, upto, 31);
  return upto - __popc(may);
}
// The marked experts (32 at most) into the warp's list.
__device__ __forceinline__ void list_experts(int* list, int at, int e0, uint32_t may) {
  for (; may; may &= may - 1) list[at++] = e0 + __ffs(may) - 1;
  __syncwarp();
}

// The selection from the lane's logits; lane i < k returns pick i.  ODD: some of them are infinite or NaN.
template <int DT, bool FULL, bool ODD>
__device__ __forceinline__ int route_logits(const RouteParams& p, int t, int lane, float (&l)[8], const float* summed,
                                             int64_t row, int* list);

template <int DT, bool FULL>
__device__ __forceinline__ int route_any(const RouteParams& p, int t, int lane, float (&l)[8], const float* summed,
                                         int64_t row, int* list) {
  // infinite logits and NaN, which few rows have
  uint32_t most = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) most = max(most, __float_as_uint(l[j]) & 0x7FFFFFFFu);
  return __any_sync(0xffffffffu, most >= 0x7F800000u) ? route_logits<DT, FULL, true>(p, t, lane, l, summed, row, list)
                                                      : route_logits<DT, FULL, false>(p, t, lane, l, summed, row, list);
}

// Routes token t by one warp; `list`: the warp's 32 ints of shared memory.
template <int DT, bool FULL>
__device__ __forceinline__ void route_token(const RouteParams& p, int t, int lane, int* list) {
  const int n = FULL ? 8 : lane_experts(p, lane), e0 = expert_of(p, lane, 0);
  const int64_t row = (int64_t)t * p.stride;
  float* summed = p.sum_out ? p.sum_out + (int64_t)t * p.E : nullptr;
  float l[8];
  load_logits<DT, FULL>(p, row + e0, n, l);
  if (summed) {
    // the partial sums in order
    for (int q = 1; q < p.KS; ++q) {
      float a[8];
      load_logits<DT, FULL>(p, q * p.part_stride + row + e0, n, a);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (FULL || j < n) l[j] += a[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (FULL || j < n) summed[e0 + j] = l[j];
    __syncwarp();
  }
  route_any<DT, FULL>(p, t, lane, l, summed, row, list);
}

template <int DT, bool FULL, bool ODD>
__device__ __forceinline__ int route_logits(const RouteParams& p, int t, int lane, float (&l)[8], const float* summed,
                                             int64_t row, int* list) {
  const int n = FULL ? 8 : lane_experts(p, lane), e0 = expert_of(p, lane, 0);
  if (ODD) {
#pragma unroll
    for (int j = 0; j < 8; ++j) l[j] = usable(l[j]);
  }

  // ---- scores, where they are needed to compare
  const bool by_logit = p.bias == nullptr;
  const bool group_sums = p.top2 && p.top_groups < p.groups;
  float v[8], top = 0.f, z = 1.f;
  if (!p.sigmoid) {
    top = fmaxf(fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])), fmaxf(fmaxf(l[4], l[5]), fmaxf(l[6], l[7])));
    top = route_value(__reduce_max_sync(0xffffffffu, route_key(top)));
    z = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = ex2_approx((l[j] - top) * kLog2eR);
      if (ODD) v[j] = l[j] > -INFINITY ? v[j] : 0.f;
      if (!FULL && j >= n) v[j] = 0.f;
      z += v[j];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    const float zi = z > 0.f ? 1.f / z : 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= zi;
  } else if (!by_logit || group_sums) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = rcp_approx(1.f + ex2_approx(l[j] * -kLog2eR));
  }
  if (!by_logit) {
    if (FULL) {
      const float4 a = __ldg((const float4*)(p.bias + e0)), b = __ldg((const float4*)(p.bias + e0) + 1);
      v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
      v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) v[j] += __ldg(p.bias + e0 + j);
    }
  } else {
    // (-0 is 0; a sum is never -0)
#pragma unroll
    for (int j = 0; j < 8; ++j) l[j] += 0.f;
    if (!group_sums) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = l[j];
    }
  }
  if (ODD || !FULL) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j >= n || !(l[j] > -INFINITY) || !(v[j] > -INFINITY)) v[j] = -INFINITY;
  }

  // ---- groups.  A sigmoid is known to 3e-7 (ex2's and the product's error enter times s (1 - s) |l|, at most
  // 0.28 |l| 2^-23), a softmax to 1.2e-6 (of which most is the common sum's), each plus the rounding of the
  // bias' sum; a group's score adds the roundings of both values, which may be far larger than their sum, and its own.
  bool doubtful = false, in = true;
  if (p.top_groups < p.groups) {
    float g1 = v[0], g2 = -INFINITY;
#pragma unroll
    for (int j = 1; j < 8; ++j) {
      g2 = fmaxf(g2, fminf(g1, v[j]));
      g1 = fmaxf(g1, v[j]);
    }
    const int lanes = 1 << p.lane_shift;
    for (int o = 1; o < lanes; o <<= 1) {
      const float a1 = __shfl_xor_sync(0xffffffffu, g1, o), a2 = __shfl_xor_sync(0xffffffffu, g2, o);
      g2 = fmaxf(fminf(g1, a1), fmaxf(g2, a2));
      g1 = fmaxf(g1, a1);
    }
    const bool two = p.top2 && g2 > -INFINITY;
    const float sc = two ? g1 + g2 : g1;
    // the groups that beat this lane's: its lanes take one other group each
    const int g = lane >> p.lane_shift;
    int better = 0;
    for (int x0 = 0; x0 < p.groups; x0 += lanes) {
      const int x = x0 + (lane & (lanes - 1));
      const float y = __shfl_sync(0xffffffffu, sc, x << p.lane_shift);
      const uint32_t m = __ballot_sync(0xffffffffu, x < p.groups && (y > sc || (y == sc && x < g)));
      better += __popc(m >> (g << p.lane_shift) & (uint32_t)((1ULL << lanes) - 1));
    }
    in = better < p.top_groups;
    if (!by_logit || group_sums) {
      // Half of what two scores apart by less may be mistaken for.  (A group without experts is known: its score is
      // -inf.  A sum beyond fp32's range is not: then a bound below is NaN, and the comparisons say so.)
      const float err = g1 > -INFINITY
                            ? (p.sigmoid ? 8e-7f : 2.5e-6f) + 3e-7f * (fabsf(g1) + (two ? fabsf(g2) : 0.f))
                            : 0.f;
      const float worst_in = route_value(__reduce_min_sync(0xffffffffu, in ? route_key(sc - err) : 0xffffffffu));
      const float best_out = route_value(__reduce_max_sync(0xffffffffu, in ? 0u : route_key(sc + err)));
      if (best_out != -INFINITY && !(worst_in > best_out)) {
        // The two largest values of the groups at the border, and what may be one of them, a lane each: the
        // groups are ranked by their sums.
        const bool near = in ? !(sc - err > best_out) : !(sc + err < worst_in);
        // (finite: an expert that is out is below a bias of fp32's lowest value)
        const float low = two ? g2 : g1;
        const float least = fmaxf(low - (8e-7f + 1e-6f * fabsf(low)), -kMostLogit);
        uint32_t may = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) may |= j < n && near && v[j] >= least ? 1u << j : 0u;
        int all = 0;
        const int at = count_before(may, lane, all);
        if (all <= 32 && p.sigmoid) {
          list_experts(list, at, e0, may);
          const int e = list[min(lane, all - 1)];
          const float x = usable(summed ? summed[e] : logit_at<DT>(p, row + e));
          const Key64 y = sigmoid_key(x, p.bias ? __ldg(p.bias + e) : 0.f);
          Key64 k1 = kNoKey, k2 = kNoKey;
#pragma unroll 1
          for (int i = 0; i < all; ++i) {
            const Key64 o = __shfl_sync(0xffffffffu, y, i);
            if (list[i] / p.per != g) continue;
            k2 = max(k2, min(k1, o));
            k1 = max(k1, o);
          }
          const Key64 sum = !near ? key64((double)sc) : p.top2 && k2 > kNoKey ? key64(value64(k1) + value64(k2)) : k1;
          better = 0;
#pragma unroll 1
          for (int x = 0; x < p.groups; ++x) {
            const Key64 o = __shfl_sync(0xffffffffu, sum, x << p.lane_shift);
            better += o > sum || (o == sum && x < g) ? 1 : 0;
          }
          in = better < p.top_groups;
          __syncwarp();
        } else {
          doubtful = true;
        }
      }
    }
  }

  // ---- keys: a value's place in the lane takes the lowest three bits (16-bit logits have none there);
  // an expert that is out 8 and its place, no expert 0
  uint32_t key[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float x = by_logit ? l[j] : v[j];
    key[j] = (in ? route_key(x) & ~7u : 8u) | (7u - j);
    if (ODD) key[j] = x > -INFINITY ? key[j] : 8u | (7u - j);
    if (!FULL && j >= n) key[j] = 0;
  }
  sort8(key);
  uint32_t mine = 0;
  int from = 0;
#pragma unroll
  for (int r = 0; r < 9; ++r) {
    if (r > p.k) break;
    const uint32_t best = __reduce_max_sync(0xffffffffu, key[0] >> 3);
    const int w = __ffs(__ballot_sync(0xffffffffu, key[0] >> 3 == best)) - 1;
    const uint32_t head = __shfl_sync(0xffffffffu, key[0], w);
    if (lane == r) {
      mine = head;
      from = w;
    }
    if (lane == w) {                       // (what the rounds that are left can reach)
#pragma unroll
      for (int j = 0; j < 8 - r; ++j) key[j] = j < 7 ? key[j + 1] : 0;
    }
  }
  // ---- two picks in a row, or the last one and the best that is left, too close to tell
  // (fp32 logits lose three bits to the place; a value has its own error too)
  auto tolerance = [&](float a) {
    return by_logit ? (DT == DQ_F32 ? 2e-6f * fabsf(a) + 1e-37f : -1.f)
                    : (p.sigmoid ? 8e-7f : 2.5e-6f) + 2.5e-6f * fabsf(a);
  };
  const float mine_v = route_value(mine & ~7u);
  bool close = false;
  {
    const uint32_t next = __shfl_down_sync(0xffffffffu, mine, 1);
    close = lane < p.k && next >= 16u && mine_v - route_value(next & ~7u) <= tolerance(mine_v);
  }
  int pick = expert_of(p, from, 7 - (int)(mine & 7u));
  // the pick's score, down to what fp32 holds at least
  auto score = [&]() {
    const float x = usable(summed ? summed[pick] : logit_at<DT>(p, row + pick));
    return p.sigmoid ? sigmoid_of(x) : expf(x - top) / z;
  };
  float s = 0.f;
  if (lane < p.k && mine >= 16u) s = score();
  if (__any_sync(0xffffffffu, doubtful || close)) {
    // The experts that may be among the picks, a lane each, where they are so few that they find room and a value
    // can be had of a logit alone: they are ranked.
    const float last = __shfl_sync(0xffffffffu, mine_v, p.k - 1);
    // (finite, as above)
    const float least = fmaxf(last - fmaxf(tolerance(last), 0.f), -kMostLogit);
    uint32_t may = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) may |= j < n && in && (by_logit ? l[j] : v[j]) >= least ? 1u << j : 0u;
    int all = 0;
    const int at = count_before(may, lane, all);
    const bool few = !__any_sync(0xffffffffu, doubtful) && all <= 32 && all >= p.k && (by_logit || p.sigmoid) &&
                     __shfl_sync(0xffffffffu, mine, p.k - 1) >= 16u;
    if (few) {
      list_experts(list, at, e0, may);
      const int e = list[min(lane, all - 1)];
      const float x = usable(summed ? summed[e] : logit_at<DT>(p, row + e));
      const Key64 y = by_logit ? key64((double)(x + 0.f)) : sigmoid_key(x, __ldg(p.bias + e));
      int rank = 0;
#pragma unroll 1
      for (int i = 0; i < all; ++i) {
        const Key64 o = __shfl_sync(0xffffffffu, y, i);
        rank += o > y || (o == y && i < lane) ? 1 : 0;        // (the list is in the order of experts)
      }
      __syncwarp();
      if (lane < all && rank < p.k) list[rank] = e;
      __syncwarp();
      if (lane < p.k) {
        pick = list[lane];
        s = score();
      }
      __syncwarp();
    } else {
      bool live;
      pick = route_exact<DT>(p, summed, row, lane, live);
      s = lane < p.k && live ? score() : 0.f;
    }
  }
  float sum = lane < p.k ? s : 0.f;
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane < p.k) {
    p.idx[(int64_t)t * p.k + lane] = pick;
    p.gate[(int64_t)t * p.k + lane] = p.renorm ? s / (sum + 1e-20f) * p.scale : s * p.scale;
  }
  return pick;
}

// Token t of one warp from its logits in memory (E of them), as a part of a larger kernel: lane i < k returns pick i.
__device__ __forceinline__ int route_one(const RouteParams& p, int t, int lane, const float* logits, int* list) {
  const int n = lane_experts(p, lane), e0 = expert_of(p, lane, 0);
  float l[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) l[j] = j < n ? logits[e0 + j] : -kMostLogit;
  return route_any<DQ_F32, false>(p, t, lane, l, logits, 0, list);
}

// What a routing says of E experts and k picks; the tokens' pointers are left open.
inline RouteParams route_params(const dq_moe_routing& r, int E, int k) {
  RouteParams p = {};
  p.E = E;
  p.k = k;
  p.groups = r.n_groups;
  p.lane_shift = 5;
  for (int g = r.n_groups; g > 1; g >>= 1) --p.lane_shift;
  p.per = E / r.n_groups;
  p.each = (p.per + (1 << p.lane_shift) - 1) >> p.lane_shift;
  p.top_groups = r.top_groups;
  p.top2 = r.group_score == DQ_ROUTE_GROUP_TOP2;
  p.sigmoid = r.scores == DQ_ROUTE_SIGMOID;
  p.renorm = r.renormalize;
  p.scale = r.scale;
  p.bias = r.bias;
  return p;
}

}  // namespace dqmoe
