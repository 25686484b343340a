// kv_attn_stream_bias.cu — attention of few query rows: a distance bias (kv_attn_stream.cuh).
#include "kv_attn_stream.cuh"

namespace dqmoe {

int launch_kv_stream_bias(const AttnParams& p, int head_dim, cudaStream_t s) {
  return launch_stream_any<kBias>(p, head_dim, s);
}

}  // namespace dqmoe
