// kv_attn.h — what the attention kernels over the 4-bit cache share: the call's
// parameters and the workspace plan.
#pragma once

#include "kv.cuh"

namespace dqmoe {

struct AttnParams {
  KvGeom g;
  const void* q;
  int64_t q_stride;
  int q_dtype, n_q_heads, group, T, B;
  const int32_t* q_start;
  const int32_t* kv_len;
  const int32_t* table;
  int max_pages, max_q_len;
  float scale;
  int causal, window;
  void* out;
  int out_dtype;
  int64_t out_stride;
  float* lse;
  uint8_t* ws;
};

// streaming kernel (kv_attn_stream.cu): few rows per K/V head
size_t kv_stream_workspace(int head_dim);
int launch_kv_stream(const AttnParams& p, int head_dim, cudaStream_t s);

// the length of request r as the kernels read it
__device__ __forceinline__ int kv_length(const AttnParams& p, int r) {
  const int64_t cap = (int64_t)p.max_pages << p.g.page_shift;
  return (int)min((int64_t)max(__ldg(p.kv_len + r), 0), cap);
}
__device__ __forceinline__ int q_rows(const AttnParams& p, int r, int* first) {
  const int a = __ldg(p.q_start + r);
  *first = a;
  // memory-safe whatever q_start holds
  return a < 0 ? 0 : max(0, min(min(__ldg(p.q_start + r + 1), p.T) - a, p.max_q_len));
}

}  // namespace dqmoe
