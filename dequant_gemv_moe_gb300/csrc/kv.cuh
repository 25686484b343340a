// kv.cuh — the 4-bit paged K/V cache's layout (include/dqmoe.h) in device code,
// and the argument checks its entry points share.
#pragma once

#include "common.cuh"

namespace dqmoe {

constexpr int kKvBlk = 16;                       // tokens per block

// byte offsets inside one token block of a head of D values
template <int D>
struct KvBlk {
  static constexpr int G = D / 32;               // scale groups
  static constexpr int W = G < 4 ? G : 4;        // groups a lane takes at a time
  static constexpr int OFF_V = 8 * D;            // V codes
  static constexpr int OFF_KD = 16 * D;          // K scales
  static constexpr int OFF_VD = 17 * D;          // V scales
  static constexpr int BYTES = 18 * D;
  // K code word of (token, group g, values 8t..8t+7)
  __device__ __forceinline__ static int k_word(int tok, int g, int t) {
    return 4 * ((((g / W) * kKvBlk + tok) * 4 + t) * W + g % W);
  }
  // V code unit (16 bits) of (token, group g, values 4a..4a+3)
  __device__ __forceinline__ static int v_unit(int tok, int g, int a) {
    return OFF_V +
           2 * ((((((tok >> 3) * (G / W) + g / W) * 8 + a) * 4 + ((tok & 7) >> 1)) * 2 + (tok & 1)) * W +
                g % W);
  }
  __device__ __forceinline__ static int k_scale(int tok, int g) {
    return OFF_KD + 2 * (tok * G + g);
  }
  __device__ __forceinline__ static int v_scale(int tok, int g) {
    return OFF_VD + 2 * ((((tok & 7) >> 1) * G + g) * 4 + (tok >> 3) * 2 + (tok & 1));
  }
};

struct KvGeom {
  uint8_t* pages;
  int heads, page_size, page_shift, n_pages;
  int64_t head_bytes;                            // one head's blocks of one page
  int64_t page_bytes;
};

inline bool kv_page_size_ok(int ps) { return ps >= 16 && ps <= 256 && (ps & (ps - 1)) == 0; }

// The checks every cache entry point makes; fills `g`.
inline int kv_check(const dq_kv_cache* c, KvGeom* g, bool need_pages) {
  if (!c || c->n_kv_heads <= 0 || c->head_dim <= 0 || c->n_pages <= 0 ||
      !kv_page_size_ok(c->page_size) || c->fmt < DQ_Q4_K || c->fmt > DQ_Q3_K)
    return DQ_ERR_ARG;
  if (c->fmt != DQ_Q4_0 || c->n_kv_heads > 1024 ||
      (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256))
    return DQ_ERR_UNSUPPORTED;
  if (need_pages) {
    if (!c->pages) return DQ_ERR_ARG;
    if ((uintptr_t)c->pages & 127) return DQ_ERR_ALIGN;
  }
  g->pages = (uint8_t*)c->pages;
  g->heads = c->n_kv_heads;
  g->page_size = c->page_size;
  g->page_shift = 0;
  while ((1 << g->page_shift) < c->page_size) ++g->page_shift;
  g->n_pages = c->n_pages;
  g->head_bytes = (int64_t)(c->page_size / kKvBlk) * 18 * c->head_dim;
  g->page_bytes = g->head_bytes * c->n_kv_heads;
  return DQ_OK;
}

inline bool kv_aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

}  // namespace dqmoe
