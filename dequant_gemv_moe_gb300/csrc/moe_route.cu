// moe_route.cu — routing to experts from their logits: softmax or sigmoid scores, a
// balancing bias, groups of experts, top-k, gates (dq_moe_route and the layer's
// routing).
//
// Mathematics.  With score s_e and value v_e = s_e + b_e, the experts of the
// `top_groups` groups with the best score (largest v, or sum of the two largest) are
// candidates, and the k largest v among them are taken, the lowest index first among
// equal ones.  The order is that of exact arithmetic:
//  * Without a bias the scores rise with the logits, so logits are compared.
//  * Else v is computed in fp32 (ex2 and rcp approximations) with a known bound on its error, and
//    wherever two values that the selection has to tell apart are closer than the bound allows, the token's
//    warp does it again in 64 bits.  (256 experts with normal logits: one token in a few hundred.)
//
// A warp takes a token, eight experts a lane.  A group is 32 / n_groups neighbouring
// lanes, so that its score is a few shuffles; lanes hold ascending experts, so
// that of equal values the lowest lane's, and in it the first, is the lowest
// index.  A lane sorts its values as integer keys whose lowest three bits are the
// place in the lane, then k + 1 rounds take the best head (one warp reduction
// and a vote) and advance that lane's list.
#include <algorithm>

#include "common.cuh"
#include "moe_route.h"

namespace dqmoe {

namespace {

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

__device__ __forceinline__ double shfl_xor_d(double x, int o) {
  return __longlong_as_double(__shfl_xor_sync(0xffffffffu, __double_as_longlong(x), o));
}

// The token's selection in 64 bits: lane i < k gets pick i and its score.
// `row`: the token's logits, `fp32` if they are.
template <int DT>
__device__ __noinline__ void route_exact(const RouteParams& p, const float* summed, int64_t row, int lane, int& pick,
                                         double& score) {
  const int n = lane_experts(p, lane);
  float l[8];
  double s[8], v[8];
  double top = -INFINITY;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int e = expert_of(p, lane, j);
    l[j] = -INFINITY;
    if (j < n) l[j] = usable(summed ? summed[e] : logit_at<DT>(p, row + e));
    s[j] = l[j];
    top = fmax(top, s[j]);
  }
  if (!p.sigmoid) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmax(top, shfl_xor_d(top, o));
  }
  double z = 0.;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const bool on = l[j] > -INFINITY;
    s[j] = !on ? 0. : p.sigmoid ? 1. / (1. + exp(-s[j])) : exp(s[j] - top);
    z += s[j];
  }
  if (!p.sigmoid) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += shfl_xor_d(z, o);
  }
  double g1 = -INFINITY, g2 = -INFINITY;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (!p.sigmoid) s[j] = z > 0. ? s[j] / z : 0.;
    // (without a bias logits are compared, which differ where scores of 1 or 0 do not; only sums take scores)
    v[j] = !(l[j] > -INFINITY) ? -INFINITY
           : p.bias            ? s[j] + (double)__ldg(p.bias + expert_of(p, lane, j))
           : p.top2            ? s[j]
                               : (double)l[j];
    if (!(v[j] > -INFINITY)) v[j] = -INFINITY;
    g2 = fmax(g2, fmin(g1, v[j]));
    g1 = fmax(g1, v[j]);
  }
  if (p.top_groups < p.groups) {
    for (int o = 1; o < 1 << p.lane_shift; o <<= 1) {
      const double a1 = shfl_xor_d(g1, o), a2 = shfl_xor_d(g2, o);
      g2 = fmax(fmin(g1, a1), fmax(g2, a2));
      g1 = fmax(g1, a1);
    }
    const double sc = p.top2 && g2 > -INFINITY ? g1 + g2 : g1;
    const int g = lane >> p.lane_shift;
    int better = 0;
    for (int x = 0; x < p.groups; ++x) {
      const double y = __longlong_as_double(__shfl_sync(0xffffffffu, __double_as_longlong(sc), x << p.lane_shift));
      better += y > sc || (y == sc && x < g) ? 1 : 0;
    }
    if (better >= p.top_groups) {
#pragma unroll
      for (int j = 0; j < 8; ++j) l[j] = -INFINITY;
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (!p.bias || !(l[j] > -INFINITY)) v[j] = l[j];
  }
  uint32_t left = (1u << n) - 1;           // places that are not taken yet
  pick = 0;
  score = 0.;
  for (int r = 0; r < p.k; ++r) {
    double best = -INFINITY, bs = 0.;
    int at = 0x7fffffff;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (!(left >> j & 1)) continue;
      const int e = expert_of(p, lane, j);
      if (v[j] > best || at == 0x7fffffff) {
        best = v[j];
        bs = v[j] > -INFINITY ? s[j] : 0.;
        at = e;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double b = shfl_xor_d(best, o), c = shfl_xor_d(bs, o);
      const int a = __shfl_xor_sync(0xffffffffu, at, o);
      if (a != 0x7fffffff && (at == 0x7fffffff || b > best || (b == best && a < at))) {
        best = b;
        bs = c;
        at = a;
      }
    }
    if (lane == r) {
      pick = at;
      score = bs;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (expert_of(p, lane, j) == at && (left >> j & 1)) left &= ~(1u << j);
  }
}

__device__ __forceinline__ void cas_keys(uint32_t& a, uint32_t& b) {
  const uint32_t hi = max(a, b), lo = min(a, b);
  a = hi;
  b = lo;
}

// Routes token t by one warp.
template <int DT>
__device__ __forceinline__ void route_token(const RouteParams& p, int t, int lane) {
  const int n = lane_experts(p, lane), e0 = expert_of(p, lane, 0);
  const int64_t row = (int64_t)t * p.stride;
  float* summed = p.sum_out ? p.sum_out + (int64_t)t * p.E : nullptr;
  float l[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) l[j] = j < n ? logit_at<DT>(p, row + e0 + j) : -INFINITY;
  if (summed) {
    // the partial sums in order
    for (int q = 1; q < p.KS; ++q)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) l[j] += logit_at<DT>(p, q * p.part_stride + row + e0 + j);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) summed[e0 + j] = l[j];
    __syncwarp();
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) l[j] = usable(l[j]);

  // ---- scores, where they are needed to compare
  const bool by_logit = p.bias == nullptr;
  const bool group_sums = p.top2 && p.top_groups < p.groups;
  float v[8], top = 0.f, z = 1.f;
  if (!p.sigmoid) {
    top = fmaxf(fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])), fmaxf(fmaxf(l[4], l[5]), fmaxf(l[6], l[7])));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    z = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = l[j] > -INFINITY ? ex2_approx((l[j] - top) * kLog2eR) : 0.f;
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
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < n ? v[j] + __ldg(p.bias + e0 + j) : 0.f;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (by_logit && !group_sums) v[j] = l[j];
    if (!(l[j] > -INFINITY) || !(v[j] > -INFINITY)) v[j] = -INFINITY;
  }

  // ---- groups.  A sigmoid is known to 3e-7 (ex2's and the product's error enter times s (1 - s) |l|, at most
  // 0.28 |l| 2^-23), a softmax to 1.2e-6 (of which most is the common sum's), each plus the rounding of the
  // bias' sum.
  bool doubtful = false, in = true;
  if (p.top_groups < p.groups) {
    float g1 = -INFINITY, g2 = -INFINITY;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      g2 = fmaxf(g2, fminf(g1, v[j]));
      g1 = fmaxf(g1, v[j]);
    }
    for (int o = 1; o < 1 << p.lane_shift; o <<= 1) {
      const float a1 = __shfl_xor_sync(0xffffffffu, g1, o), a2 = __shfl_xor_sync(0xffffffffu, g2, o);
      g2 = fmaxf(fminf(g1, a1), fmaxf(g2, a2));
      g1 = fmaxf(g1, a1);
    }
    const float sc = p.top2 && g2 > -INFINITY ? g1 + g2 : g1;
    const int g = lane >> p.lane_shift;
    int better = 0;
    for (int x = 0; x < p.groups; ++x) {
      const float y = __shfl_sync(0xffffffffu, sc, x << p.lane_shift);
      better += y > sc || (y == sc && x < g) ? 1 : 0;
    }
    in = better < p.top_groups;
    if (!by_logit || group_sums) {
      const uint32_t key = route_key(sc);
      const float worst_in = route_value(__reduce_min_sync(0xffffffffu, in ? key : 0xffffffffu));
      const float best_out = route_value(__reduce_max_sync(0xffffffffu, in ? 0u : key));
      doubtful = worst_in > -INFINITY && best_out > -INFINITY &&
                 worst_in - best_out <= (p.sigmoid ? 1.6e-6f : 5e-6f) + 6e-7f * (fabsf(worst_in) + fabsf(best_out));
    }
  }

  // ---- keys: a value's place in the lane takes the lowest three bits (16-bit logits have none there);
  // an expert that is out 8 and its place, no expert 0
  uint32_t key[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float x = by_logit ? l[j] : v[j];
    key[j] = j >= n ? 0u : (!in || !(x > -INFINITY) ? 8u : route_key(x) & ~7u) | (7u - j);
  }
  // Batcher's odd-even merge sort of 8
#define DQ_CAS(a, b) cas_keys(key[a], key[b])
  DQ_CAS(0, 1); DQ_CAS(2, 3); DQ_CAS(4, 5); DQ_CAS(6, 7);
  DQ_CAS(0, 2); DQ_CAS(1, 3); DQ_CAS(4, 6); DQ_CAS(5, 7);
  DQ_CAS(1, 2); DQ_CAS(5, 6);
  DQ_CAS(0, 4); DQ_CAS(1, 5); DQ_CAS(2, 6); DQ_CAS(3, 7);
  DQ_CAS(2, 4); DQ_CAS(3, 5);
  DQ_CAS(1, 2); DQ_CAS(3, 4); DQ_CAS(5, 6);
#undef DQ_CAS
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
    if (lane == w) {
#pragma unroll
      for (int j = 0; j < 7; ++j) key[j] = key[j + 1];
      key[7] = 0;
    }
  }
  // ---- two picks in a row, or the last one and the best that is left, too close to tell
  {
    const uint32_t next = __shfl_down_sync(0xffffffffu, mine, 1);
    const float a = route_value(mine & ~7u), b = route_value(next & ~7u);
    // fp32 logits lose three bits to the place; a value has its own error too
    const float tol = by_logit ? (DT == DQ_F32 ? 2e-6f * fabsf(a) + 1e-37f : -1.f)
                               : (p.sigmoid ? 8e-7f : 2.5e-6f) + 2.5e-6f * fabsf(a);
    if (lane < p.k && next >= 16u && a - b <= tol) doubtful = true;
  }
  int pick = expert_of(p, from, 7 - (int)(mine & 7u));
  float s;
  if (__any_sync(0xffffffffu, doubtful)) {
    int pick64;
    double s64;
    route_exact<DT>(p, summed, row, lane, pick64, s64);
    pick = pick64;
    s = (float)s64;
  } else {
    s = 0.f;
    if (lane < p.k && mine >= 16u) {
      const float x = usable(summed ? summed[pick] : logit_at<DT>(p, row + pick));
      s = p.sigmoid ? 1.f / (1.f + expf(-x)) : expf(x - top) / z;
    }
  }
  float sum = lane < p.k ? s : 0.f;
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane < p.k) {
    p.idx[(int64_t)t * p.k + lane] = pick;
    p.gate[(int64_t)t * p.k + lane] = p.renorm ? s / (sum + 1e-20f) * p.scale : s * p.scale;
  }
}

constexpr int kRouteWarps = 4;

template <int DT>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(const __grid_constant__ RouteParams p) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  for (int64_t t = (int64_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5); t < p.T; t += (int64_t)gridDim.x * kRouteWarps)
    route_token<DT>(p, (int)t, lane);
}

}  // namespace

int check_routing(const dq_moe_routing* r, int E, int top_k) {
  if (!r || (r->scores != DQ_ROUTE_SOFTMAX && r->scores != DQ_ROUTE_SIGMOID) ||
      (r->group_score != DQ_ROUTE_GROUP_MAX && r->group_score != DQ_ROUTE_GROUP_TOP2) ||
      (r->renormalize != 0 && r->renormalize != 1) || !(r->scale > 0.f) || !(r->scale <= 3.4e38f))
    return DQ_ERR_ARG;
  if (r->n_groups <= 0 || E % r->n_groups || r->top_groups <= 0 || r->top_groups > r->n_groups ||
      (int64_t)r->top_groups * (E / r->n_groups) < top_k)
    return DQ_ERR_ARG;
  if (r->n_groups > 32 || (r->n_groups & (r->n_groups - 1))) return DQ_ERR_UNSUPPORTED;
  if ((uintptr_t)r->bias & 3) return DQ_ERR_ALIGN;
  return DQ_OK;
}

int launch_route(const void* logits, int dtype, int64_t stride, int KS, int T, int E, int k,
                 const dq_moe_routing& r, float* sum_out, int32_t* idx, float* gate, cudaStream_t s) {
  RouteParams p;
  p.logits = logits;
  p.stride = stride;
  p.part_stride = (int64_t)T * E;
  p.KS = KS;
  p.T = T;
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
  p.sum_out = sum_out;
  p.idx = idx;
  p.gate = gate;
  const int ctas = std::min((T + kRouteWarps - 1) / kRouteWarps, 152 * 12);
  cudaError_t e;
  if (dtype == DQ_F32) e = launch_pdl(route_kernel<DQ_F32>, dim3(ctas), dim3(kRouteWarps * 32), 0, s, 0, p);
  else if (dtype == DQ_F16) e = launch_pdl(route_kernel<DQ_F16>, dim3(ctas), dim3(kRouteWarps * 32), 0, s, 0, p);
  else e = launch_pdl(route_kernel<DQ_BF16>, dim3(ctas), dim3(kRouteWarps * 32), 0, s, 0, p);
  if (e != cudaSuccess) return DQ_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? DQ_OK : DQ_ERR_CUDA;
}

}  // namespace dqmoe

using namespace dqmoe;

extern "C" int dq_moe_route(const void* logits, int dtype, int64_t stride, int T, int E, int top_k,
                            const dq_moe_routing* routing, int32_t* topk_idx, float* topk_gate,
                            void* stream) {
  if (!logits || !topk_idx || !topk_gate || (dtype != DQ_F32 && dtype != DQ_F16 && dtype != DQ_BF16))
    return DQ_ERR_ARG;
  if (T <= 0 || E <= 0 || top_k <= 0 || top_k > E || stride < E || stride > (1LL << 31)) return DQ_ERR_ARG;
  if (E > 256 || top_k > 8) return DQ_ERR_UNSUPPORTED;
  const int rc = check_routing(routing, E, top_k);
  if (rc != DQ_OK) return rc;
  if ((uintptr_t)logits & (dtype == DQ_F32 ? 3 : 1) || (uintptr_t)topk_idx & 3 || (uintptr_t)topk_gate & 3)
    return DQ_ERR_ALIGN;
  return launch_route(logits, dtype, stride, 1, T, E, top_k, *routing, nullptr, topk_idx, topk_gate,
                      (cudaStream_t)stream);
}
