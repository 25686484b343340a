// kv_attn_stream.cu — attention of few query rows over the 4-bit paged cache, plain
// scores (kv_attn_stream.cuh).
#include "kv_attn_stream.cuh"

namespace dqmoe {

int launch_kv_stream_ext(const AttnParams& p, int head_dim, cudaStream_t s);   // kv_attn_stream_ext.cu

size_t kv_stream_workspace() { return kStreamO + kStreamMl + kStreamDesc; }

int launch_kv_stream(const AttnParams& p, int head_dim, bool ext, cudaStream_t s) {
  return ext ? launch_kv_stream_ext(p, head_dim, s) : launch_stream_any<false>(p, head_dim, s);
}

}  // namespace dqmoe
