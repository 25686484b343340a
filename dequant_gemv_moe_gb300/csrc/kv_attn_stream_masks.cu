// kv_attn_stream_masks.cu — attention of few query rows: prefixes and first positions (kv_attn_stream.cuh).
#include "kv_attn_stream.cuh"

namespace dqmoe {

int launch_kv_stream_masks(const AttnParams& p, int head_dim, cudaStream_t s) {
  return launch_stream_any<kMasks>(p, head_dim, s);
}

}  // namespace dqmoe
