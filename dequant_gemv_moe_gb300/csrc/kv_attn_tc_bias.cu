// kv_attn_tc_bias.cu — attention of many query rows: a distance bias (kv_attn_tc.cuh).
#include "kv_attn_tc.cuh"

namespace dqmoe {

int launch_kv_tc_bias(const AttnParams& p, int head_dim, cudaStream_t s) {
  return launch_tc_any<kBias>(p, head_dim, s);
}

}  // namespace dqmoe
