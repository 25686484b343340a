// kv_attn_stream_caps.cu — attention of few query rows: capped scores (kv_attn_stream.cuh).
#include "kv_attn_stream.cuh"

namespace dqmoe {

int launch_kv_stream_caps(const AttnParams& p, int head_dim, cudaStream_t s) {
  return launch_stream_any<kCaps>(p, head_dim, s);
}

}  // namespace dqmoe
