// kv_attn_tc_caps.cu — attention of many query rows: capped scores (kv_attn_tc.cuh).
#include "kv_attn_tc.cuh"

namespace dqmoe {

int launch_kv_tc_caps(const AttnParams& p, int head_dim, cudaStream_t s) {
  return launch_tc_any<kCaps>(p, head_dim, s);
}

}  // namespace dqmoe
