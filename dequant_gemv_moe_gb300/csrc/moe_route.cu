// moe_route.cu — dq_moe_route and the layer's routing of more than a few tokens
// (moe_route.cuh).
#include "moe_route.cuh"

namespace dqmoe {

namespace {

constexpr int kRouteWarps = 4;

template <int DT, bool FULL>
__global__ void __launch_bounds__(kRouteWarps * 32, 8) route_kernel(const __grid_constant__ RouteParams p) {
  __shared__ int list[kRouteWarps][32];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp;
  if (t < p.T) route_token<DT, FULL>(p, (int)t, lane, list[warp]);
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
  RouteParams p = route_params(r, E, k);
  p.logits = logits;
  p.stride = stride;
  p.part_stride = (int64_t)T * E;
  p.KS = KS;
  p.T = T;
  p.sum_out = sum_out;
  p.idx = idx;
  p.gate = gate;
  const int ctas = (int)(((int64_t)T + kRouteWarps - 1) / kRouteWarps);
  // Rows and bias that the lanes take in 16-byte words, eight experts each and none without: 256 experts on a boundary (16384
  // tokens, fp32 16.5 us, one logit at a time 20.0; bf16 20.8 and 24.1; 8 tokens 3.0 and 3.3).  Fewer experts leave lanes that have
  // fewer than eight and are loaded one at a time: 64, 128 or 160 take 18.1 to 18.3.
  const int el = dtype == DQ_F32 ? 4 : 2;
  const bool full = E == 256 && (uintptr_t)logits % 16 == 0 && stride * el % 16 == 0 && (uintptr_t)r.bias % 16 == 0;
  cudaError_t e = cudaSuccess;
#define DQ_ROUTE(DT, FULL)        \
  if (dtype == DT && full == FULL) \
    e = launch_pdl(route_kernel<DT, FULL>, dim3(ctas), dim3(kRouteWarps * 32), 0, s, 0, p);
  DQ_ROUTE(DQ_F32, true)
  DQ_ROUTE(DQ_F16, true)
  DQ_ROUTE(DQ_BF16, true)
  DQ_ROUTE(DQ_F32, false)
  DQ_ROUTE(DQ_F16, false)
  DQ_ROUTE(DQ_BF16, false)
#undef DQ_ROUTE
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
