// moe_route.h — routing from logits (include/dqmoe.h: dq_moe_routing), shared by
// its own entry point and the layer's.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/dqmoe.h"

namespace dqmoe {

// Argument checks of a routing for E experts and top_k picks.
int check_routing(const dq_moe_routing* r, int E, int top_k);

// logits: [KS][T][E] partial sums in fp32 (KS > 1, or `sum_out`: their sums go there too),
// or rows of `dtype`, `stride` elements apart.
int launch_route(const void* logits, int dtype, int64_t stride, int KS, int T, int E, int k,
                 const dq_moe_routing& r, float* sum_out, int32_t* idx, float* gate, cudaStream_t s);

}  // namespace dqmoe
