// kv_attn.cu — dq_kv_attention: argument checks and the choice of kernels.
#include "kv_attn.h"

namespace dqmoe {

namespace {

// The streaming kernel decodes a page once for every 8 rows, the tensor-core kernel once for 256, at the
// price of a tile of 128 rows whatever their number.  32 requests of up to 32 rows (8 K/V heads of 128,
// 16000 tokens): 134 us streaming, 257 us on the tensor core; they meet at about 64 rows.
constexpr int kStreamRows = 64;

// Many rows: up to this cap tanh comes from the exponential's unit, c - 2c / (1 + e^2u), above it from the polynomial,
// which is off by 2.5e-7 of itself.  The first is off by that of the cap, whatever the score: of c, at most 7e-7 (e^2u two
// units, the sum, the product of two, its inverse to one unit, and two more products), 3.6e-7 measured.  For this cap that
// is 7e-5 in a score, a third of what rounding its weight to fp16 (2^-12) moves the output by; the lse takes it as it is:
// rows of one to four tokens with scores about 6, 7e-6 off in the mean square at a cap of 100, 3.9e-6 at 50, 2.8e-6 at 101.
// What it saves: chunks of 2048 over 16384, 32 heads of 128 on 8, 1435 us, with the polynomial 1936.
constexpr float kSmallCap = 100.f;

// tanh(u) / u in powers of u^2: interpolated at the Chebyshev points of [0, 1]
constexpr double kTanh[7] = {0.9999999486455697,  -0.333328279786008,    0.13325076146118553, -0.053451646370382085,
                             0.02027970828675751, -0.006194324834556632, 0.0010380250969887872};

int attn_sizes_ok(const dq_kv_cache* cache, int n_q_heads, int T, int B, int max_q_len) {
  if (n_q_heads <= 0 || T <= 0 || B <= 0 || max_q_len <= 0 || max_q_len > T) return DQ_ERR_ARG;
  if (n_q_heads % cache->n_kv_heads) return DQ_ERR_ARG;
  if (n_q_heads > 4096 || B > DQ_KV_MAX_REQUESTS || T > (1 << 24) ||
      (int64_t)T * (n_q_heads / cache->n_kv_heads) > (1LL << 30))
    return DQ_ERR_UNSUPPORTED;
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
  *bytes = kv_stream_workspace() +
           ((int64_t)max_q_len * (n_q_heads / cache->n_kv_heads) > kStreamRows ? kv_tc_workspace() : 0);
  return DQ_OK;
}

int dq_kv_attention(const dq_kv_cache* cache, const dq_kv_attn* a, void* ws, size_t ws_bytes,
                    void* stream) {
  return dq_kv_attention_ex(cache, a, nullptr, ws, ws_bytes, stream);
}

int dq_kv_attention_ex(const dq_kv_cache* cache, const dq_kv_attn* a, const dq_kv_scores* x, void* ws,
                       size_t ws_bytes, void* stream) {
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
  if (x && x->softcap != 0.f && !(x->softcap >= 0.01f && x->softcap <= 1e6f)) return DQ_ERR_ARG;
  // fp32 queries would be held to a bar that 16-bit operands cannot meet
  if (a->q_dtype == DQ_F32) return DQ_ERR_UNSUPPORTED;
  if (!kv_aligned(a->q, 16) || !kv_aligned(a->out, 16) || a->q_stride % 8 || a->out_stride % 8 ||
      !kv_aligned(a->q_start, 4) || !kv_aligned(a->kv_len, 4) || !kv_aligned(a->block_table, 4) ||
      !kv_aligned(a->lse, 4))
    return DQ_ERR_ALIGN;
  if (x && (!kv_aligned(x->slopes, 4) || !kv_aligned(x->prefix_len, 4) || !kv_aligned(x->first_pos, 4)))
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
  p.group_inv = group_inverse(p.group);
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
  const bool ext = x && (x->softcap != 0.f || x->slopes || x->prefix_len || x->first_pos);
  p.cap = ext ? (float)(x->softcap * 1.4426950408889634) : 0.f;
  p.cap_inv = p.cap > 0.f ? 1.f / p.cap : 1.f;
  p.cap_small = p.cap > 0.f && x->softcap <= kSmallCap;
  for (int k = 0; k < 7; ++k) p.cap_c[k].x = p.cap_c[k].y = (float)(kTanh[k] * p.cap);
  p.slopes = ext ? x->slopes : nullptr;
  p.prefix = ext && a->causal ? x->prefix_len : nullptr;
  p.first_pos = ext ? x->first_pos : nullptr;
  // Requests with at most kStreamRows rows per K/V head stream.  If one may have more, so that the
  // tensor-core kernel is launched anyway, those with more than half as many go there: what streams is
  // then a launch of its own beside it (one request of 45 rows among prompts: 11 us more as a stream).
  const bool many = (int64_t)a->max_q_len * p.group > kStreamRows;
  p.rows_above = 0;
  p.alone = 0;
  p.rows_upto = many ? kStreamRows / 2 : kStreamRows;
  p.ws = (uint8_t*)ws;
  rc = launch_kv_stream(p, cache->head_dim, ext, (cudaStream_t)stream);
  if (rc != DQ_OK || !many) return rc;
  p.rows_above = p.rows_upto;
  p.rows_upto = 1 << 30;
  p.ws = (uint8_t*)ws + kv_stream_workspace();
  return launch_kv_tc(p, cache->head_dim, ext, (cudaStream_t)stream);
}

}  // extern "C"
