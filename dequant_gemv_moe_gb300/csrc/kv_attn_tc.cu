// kv_attn_tc.cu — attention of many query rows over the 4-bit paged cache, plain scores
// (kv_attn_tc.cuh).
#include "kv_attn_tc.cuh"

namespace dqmoe {

int launch_kv_tc_ext(const AttnParams& p, int head_dim, cudaStream_t s);       // kv_attn_tc_ext.cu

size_t kv_tc_workspace() { return kTcO + kTcMl + kTcDesc; }

int launch_kv_tc(const AttnParams& p, int head_dim, bool ext, cudaStream_t s) {
  return ext ? launch_kv_tc_ext(p, head_dim, s) : launch_tc_any<false>(p, head_dim, s);
}

}  // namespace dqmoe
