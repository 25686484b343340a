// kv_attn.cu — attention over the 4-bit paged cache: the plain kernel, one CTA
// per (row, query head), every product in fp32.
#include <algorithm>

#include "kv_attn.h"

namespace dqmoe {

namespace {

__device__ __forceinline__ float q_at(const AttnParams& p, int64_t i) {
  return p.q_dtype == DQ_BF16 ? __bfloat162float(((const __nv_bfloat16*)p.q)[i])
                              : __half2float(((const __half*)p.q)[i]);
}

__device__ __forceinline__ const uint8_t* kv_block(const AttnParams& p, int r, int h, int tok) {
  int page = __ldg(p.table + (int64_t)r * p.max_pages + (tok >> p.g.page_shift));
  if (page < 0 || page >= p.g.n_pages) page = 0;
  return p.g.pages + page * p.g.page_bytes + h * p.g.head_bytes;
}

constexpr int kPlainThreads = 128;

template <int D>
__global__ void __launch_bounds__(kPlainThreads) kv_attn_plain_kernel(const __grid_constant__ AttnParams p) {
  using B = KvBlk<D>;
  pdl_wait();
  pdl_trigger();
  __shared__ float qs[D], ps[kPlainThreads], red[4];
  __shared__ int req;
  const int row = blockIdx.x, hq = blockIdx.y, h = hq / p.group, tid = threadIdx.x;
  if (tid == 0) {
    int lo = 0, hi = p.B;                     // the last request that starts at or before the row
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(p.q_start + mid) <= row) lo = mid;
      else hi = mid;
    }
    req = lo;
  }
  __syncthreads();
  const int r = req;
  const int r0 = __ldg(p.q_start + r), n = __ldg(p.q_start + r + 1) - r0;
  if (row >= __ldg(p.q_start + p.B) || row - r0 >= p.max_q_len) return;
  const int len = (int)min((int64_t)max(__ldg(p.kv_len + r), 0),
                           (int64_t)p.max_pages << p.g.page_shift);
  const int pos = len - n + (row - r0);
  const int end = p.causal ? min(len, pos + 1) : len;
  const int begin = p.window > 0 ? max(0, pos - p.window + 1) : 0;
  for (int i = tid; i < D; i += kPlainThreads)
    qs[i] = q_at(p, (int64_t)row * p.q_stride + (int64_t)hq * D + i) * p.scale;
  __syncthreads();
  float m = -INFINITY, l = 0.f, o[(D + kPlainThreads - 1) / kPlainThreads] = {};
  for (int j0 = begin; j0 < end; j0 += kPlainThreads) {
    const int j = j0 + tid;
    float s = -INFINITY;
    if (j < end) {
      const int off = j & (p.g.page_size - 1), i = off % kKvBlk;
      const uint8_t* blk = kv_block(p, r, h, j) + (off / kKvBlk) * B::BYTES;
      s = 0.f;
      for (int g = 0; g < B::G; ++g) {
        float a = 0.f;
        for (int t = 0; t < 4; ++t) {
          const uint32_t w = *(const uint32_t*)(blk + B::k_word(i, g, t));
#pragma unroll
          for (int e = 0; e < 8; ++e)
            a += qs[g * 32 + 8 * t + e] *
                 (float)((int)(w >> (4 * (e >> 1) + 16 * (e & 1)) & 15u) - 8);
        }
        s += a * __half2float(*(const __half*)(blk + B::k_scale(i, g)));
      }
    }
    float mx = s;
    for (int o2 = 16; o2 > 0; o2 >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o2));
    __syncthreads();
    if ((tid & 31) == 0) red[tid >> 5] = mx;
    __syncthreads();
    const float mn = fmaxf(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), m);
    const float corr = expf(m - mn), e = j < end ? expf(s - mn) : 0.f;
    m = mn;
    ps[tid] = e;
    __syncthreads();
    float sum = 0.f;
    for (int t = 0; t < kPlainThreads; ++t) sum += ps[t];
    l = l * corr + sum;
    const int cnt = min(kPlainThreads, end - j0);
#pragma unroll
    for (int k = 0; k < (D + kPlainThreads - 1) / kPlainThreads; ++k) {
      const int d = tid + k * kPlainThreads;
      o[k] *= corr;
      if (d >= D) continue;
      for (int t = 0; t < cnt; ++t) {
        const int jj = j0 + t, off = jj & (p.g.page_size - 1), i = off % kKvBlk;
        const uint8_t* blk = kv_block(p, r, h, jj) + (off / kKvBlk) * B::BYTES;
        const uint32_t w = *(const uint16_t*)(blk + B::v_unit(i, d / 32, d % 32 / 4));
        o[k] += ps[t] * (__half2float(*(const __half*)(blk + B::v_scale(i, d / 32))) *
                         (float)((int)(w >> (4 * (d & 3)) & 15u) - 8));
      }
    }
  }
  for (int k = 0; k < (D + kPlainThreads - 1) / kPlainThreads; ++k) {
    const int d = tid + k * kPlainThreads;
    if (d >= D) continue;
    const float v = l > 0.f ? o[k] / l : 0.f;
    const int64_t at = (int64_t)row * p.out_stride + (int64_t)hq * D + d;
    if (p.out_dtype == DQ_F32) ((float*)p.out)[at] = v;
    else if (p.out_dtype == DQ_F16) ((__half*)p.out)[at] = __float2half_rn(v);
    else ((__nv_bfloat16*)p.out)[at] = __float2bfloat16_rn(v);
  }
  if (tid == 0 && p.lse) p.lse[(int64_t)row * p.n_q_heads + hq] = l > 0.f ? m + logf(l) : -INFINITY;
}

int attn_sizes_ok(const dq_kv_cache* cache, int n_q_heads, int T, int B, int max_q_len) {
  if (n_q_heads <= 0 || T <= 0 || B <= 0 || max_q_len <= 0 || max_q_len > T) return DQ_ERR_ARG;
  if (n_q_heads % cache->n_kv_heads) return DQ_ERR_ARG;
  if (n_q_heads > 4096 || B > DQ_KV_MAX_REQUESTS || T > (1 << 24)) return DQ_ERR_UNSUPPORTED;
  return DQ_OK;
}

}  // namespace
}  // namespace dqmoe

using namespace dqmoe;

extern "C" {

int dq_kv_attention_workspace_size(const dq_kv_cache* cache, int n_q_heads, int T, int B,
                                   int max_q_len, size_t* bytes) {
  if (!bytes) return DQ_ERR_ARG;
  KvGeom g;
  int rc = kv_check(cache, &g, false);
  if (rc != DQ_OK) return rc;
  rc = attn_sizes_ok(cache, n_q_heads, T, B, max_q_len);
  if (rc != DQ_OK) return rc;
  *bytes = kv_stream_workspace(cache->head_dim);
  return DQ_OK;
}

int dq_kv_attention(const dq_kv_cache* cache, const dq_kv_attn* a, void* ws, size_t ws_bytes,
                    void* stream) {
  AttnParams p;
  int rc = kv_check(cache, &p.g, true);
  if (rc != DQ_OK) return rc;
  if (!a || !a->q || !a->q_start || !a->kv_len || !a->block_table || !a->out) return DQ_ERR_ARG;
  rc = attn_sizes_ok(cache, a->n_q_heads, a->T, a->B, a->max_q_len);
  if (rc != DQ_OK) return rc;
  const int64_t row = (int64_t)a->n_q_heads * cache->head_dim;
  if (a->q_dtype < DQ_F32 || a->q_dtype > DQ_BF16 || a->out_dtype < DQ_F32 ||
      a->out_dtype > DQ_BF16)
    return DQ_ERR_ARG;
  if (a->max_pages <= 0 || (int64_t)a->max_pages * cache->page_size > 2147483647LL ||
      a->q_stride < row || a->out_stride < row || a->q_stride > (1LL << 31) ||
      a->out_stride > (1LL << 31) || !(a->scale > 0.f) || !(a->scale <= 3.4e38f) ||
      (a->causal != 0 && a->causal != 1) || a->window < 0)
    return DQ_ERR_ARG;
  // fp32 queries would be held to a bar that 16-bit operands cannot meet
  if (a->q_dtype == DQ_F32) return DQ_ERR_UNSUPPORTED;
  if (!kv_aligned(a->q, 16) || !kv_aligned(a->out, 16) || a->q_stride % 8 || a->out_stride % 8 ||
      !kv_aligned(a->q_start, 4) || !kv_aligned(a->kv_len, 4) || !kv_aligned(a->block_table, 4) ||
      !kv_aligned(a->lse, 4))
    return DQ_ERR_ALIGN;
  size_t need = 0;
  rc = dq_kv_attention_workspace_size(cache, a->n_q_heads, a->T, a->B, a->max_q_len, &need);
  if (rc != DQ_OK) return rc;
  if (!ws) return DQ_ERR_WORKSPACE;
  if (!kv_aligned(ws, 256)) return DQ_ERR_ALIGN;
  if (ws_bytes < need) return DQ_ERR_WORKSPACE;
  p.q = a->q;
  p.q_stride = a->q_stride;
  p.q_dtype = a->q_dtype;
  p.n_q_heads = a->n_q_heads;
  p.group = a->n_q_heads / cache->n_kv_heads;
  p.T = a->T;
  p.B = a->B;
  p.q_start = a->q_start;
  p.kv_len = a->kv_len;
  p.table = a->block_table;
  p.max_pages = a->max_pages;
  p.max_q_len = a->max_q_len;
  p.scale = a->scale;
  p.causal = a->causal;
  p.window = a->window;
  p.out = a->out;
  p.out_dtype = a->out_dtype;
  p.out_stride = a->out_stride;
  p.lse = a->lse;
  p.ws = (uint8_t*)ws;
  if ((int64_t)a->max_q_len * p.group <= 64)
    return launch_kv_stream(p, cache->head_dim, (cudaStream_t)stream);
  const dim3 grid((unsigned)a->T, (unsigned)a->n_q_heads), block(kPlainThreads);
  cudaError_t e;
  cudaStream_t s = (cudaStream_t)stream;
  if (cache->head_dim == 64) e = launch_pdl(kv_attn_plain_kernel<64>, grid, block, 0, s, 0, p);
  else if (cache->head_dim == 128) e = launch_pdl(kv_attn_plain_kernel<128>, grid, block, 0, s, 0, p);
  else e = launch_pdl(kv_attn_plain_kernel<256>, grid, block, 0, s, 0, p);
  if (e != cudaSuccess) return DQ_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? DQ_OK : DQ_ERR_CUDA;
}

}  // extern "C"
