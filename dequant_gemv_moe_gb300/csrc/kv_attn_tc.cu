// kv_attn_tc.cu — attention of many query rows over the 4-bit paged cache: the choice of
// the kernel's mode, and plain scores (kv_attn_tc.cuh).
#include "kv_attn_tc.cuh"

namespace dqmoe {

int launch_kv_tc_masks(const AttnParams& p, int head_dim, cudaStream_t s);      // kv_attn_tc_masks.cu
int launch_kv_tc_caps(const AttnParams& p, int head_dim, cudaStream_t s);       // kv_attn_tc_caps.cu
int launch_kv_tc_bias(const AttnParams& p, int head_dim, cudaStream_t s);       // kv_attn_tc_bias.cu
int launch_kv_tc_scores(const AttnParams& p, int head_dim, cudaStream_t s);     // kv_attn_tc_scores.cu

size_t kv_tc_workspace() { return kTcO + kTcMl + kTcDesc; }

int launch_kv_tc(const AttnParams& p, int head_dim, bool ext, cudaStream_t s) {
  if (!ext) return launch_tc_any<kPlain>(p, head_dim, s);
  if (p.cap == 0.f && !p.slopes) return launch_kv_tc_masks(p, head_dim, s);
  if (p.cap_small && !p.slopes) return launch_kv_tc_caps(p, head_dim, s);
  if (p.cap == 0.f) return launch_kv_tc_bias(p, head_dim, s);
  return launch_kv_tc_scores(p, head_dim, s);
}

}  // namespace dqmoe
