// kv_attn_stream.cu — attention of few query rows over the 4-bit paged cache: the choice of
// the kernel's mode, and plain scores (kv_attn_stream.cuh).
#include "kv_attn_stream.cuh"

namespace dqmoe {

int launch_kv_stream_masks(const AttnParams& p, int head_dim, cudaStream_t s);  // kv_attn_stream_masks.cu
int launch_kv_stream_caps(const AttnParams& p, int head_dim, cudaStream_t s);   // kv_attn_stream_caps.cu
int launch_kv_stream_bias(const AttnParams& p, int head_dim, cudaStream_t s);   // kv_attn_stream_bias.cu
int launch_kv_stream_scores(const AttnParams& p, int head_dim, cudaStream_t s); // kv_attn_stream_scores.cu

size_t kv_stream_workspace() { return kStreamO + kStreamMl + kStreamDesc; }

int launch_kv_stream(const AttnParams& p, int head_dim, bool ext, cudaStream_t s) {
  if (!ext) return launch_stream_any<kPlain>(p, head_dim, s);
  if (p.cap == 0.f) return p.slopes ? launch_kv_stream_bias(p, head_dim, s) : launch_kv_stream_masks(p, head_dim, s);
  return p.slopes ? launch_kv_stream_scores(p, head_dim, s) : launch_kv_stream_caps(p, head_dim, s);
}

}  // namespace dqmoe
