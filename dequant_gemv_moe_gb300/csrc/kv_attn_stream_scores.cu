// kv_attn_stream_scores.cu — attention of few query rows: a cap and a bias (kv_attn_stream.cuh).
#include "kv_attn_stream.cuh"

namespace dqmoe {

int launch_kv_stream_scores(const AttnParams& p, int head_dim, cudaStream_t s) {
  return launch_stream_any<kAnyScores>(p, head_dim, s);
}

}  // namespace dqmoe
