// kv_attn_stream_ext.cu — the same with capped or biased scores, prefixes and first positions.
#include "kv_attn_stream.cuh"

namespace dqmoe {

int launch_kv_stream_ext(const AttnParams& p, int head_dim, cudaStream_t s) {
  return launch_stream_any<true>(p, head_dim, s);
}

}  // namespace dqmoe
