// kv_attn_tc_scores.cu — attention of many query rows: any cap with any bias (kv_attn_tc.cuh).
#include "kv_attn_tc.cuh"

namespace dqmoe {

int launch_kv_tc_scores(const AttnParams& p, int head_dim, cudaStream_t s) {
  return launch_tc_any<kAnyScores>(p, head_dim, s);
}

}  // namespace dqmoe
