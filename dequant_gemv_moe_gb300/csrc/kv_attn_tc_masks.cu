// kv_attn_tc_masks.cu — attention of many query rows: prefixes and first positions (kv_attn_tc.cuh).
#include "kv_attn_tc.cuh"

namespace dqmoe {

int launch_kv_tc_masks(const AttnParams& p, int head_dim, cudaStream_t s) {
  return launch_tc_any<kMasks>(p, head_dim, s);
}

}  // namespace dqmoe
