// kv_attn_tc_ext.cu — the same with capped or biased scores, prefixes and first positions.
#include "kv_attn_tc.cuh"

namespace dqmoe {

int launch_kv_tc_ext(const AttnParams& p, int head_dim, cudaStream_t s) {
  return launch_tc_any<true>(p, head_dim, s);
}

}  // namespace dqmoe
