// kv_cache.cu — the 4-bit paged K/V cache: a step's block tables and slots
// (dq_kv_plan), K/V rows into it as Q4_0 blocks (dq_kv_append) and back out
// (dq_kv_read).
#include <algorithm>

#include "kv_rows.cuh"

namespace dqmoe {

namespace {

struct KvRows {
  KvGeom g;
  const void* k;
  const void* v;
  void* ko;
  void* vo;
  int64_t k_stride, v_stride;
  const int64_t* slots;
  int64_t n_slots;
  int64_t items;               // of one head's K or V: T * D / 8
};

constexpr int kRowsThreads = 256;
constexpr int kRowsUnroll = 2;   // chunks per thread, their loads all in flight

// Eight values per thread, a head's (token, chunk of 8) in one line, the chunks
// fastest: a group of 32 values is four lanes.  K's eight values are a word of its
// layout; for V two lanes whose groups are neighbours exchange halves of their
// units, so that each stores one word too.
//
// Bound by latency for a step (64 tokens, 8 heads of 128: 2.7 us).  A prompt (8191
// tokens, bf16: 13 us, 43 MB at 3.3 TB/s) is near no single limit: range, quotient, clamp and packing of
// each value keep issue and the ALU pipe busy in 69 % of the cycles, beside HBM at half.  fp32 rows
// with one true division each, appended and read back: 38 us for 8191 tokens, 4.1 TB/s.  1, 2
// and 4 chunks a thread take 25.4, 23.1 and 22.5 us with the reading back, and four leave a
// step on too few CTAs.  K and V are different CTAs: with both in one thread it was 31 us.
template <int D, int DT, bool V>
__device__ __forceinline__ void append_rows(const KvRows& p) {
  using B = KvBlk<D>;
  constexpr int C = D / 8;
  const int lane = threadIdx.x & 31, h = blockIdx.y;
  const void* src = V ? p.v : p.k;
  const int64_t stride = V ? p.v_stride : p.k_stride;
  const int64_t base = (int64_t)blockIdx.x * (kRowsThreads * kRowsUnroll) + threadIdx.x;
  const int c = threadIdx.x % C, g = c / 4, t = c & 3;   // kRowsThreads is a multiple of C
  float x[kRowsUnroll][8];
  int64_t slot[kRowsUnroll];
#pragma unroll
  for (int j = 0; j < kRowsUnroll; ++j) {
    const int64_t id = base + j * kRowsThreads;
    const bool in = id < p.items;          // (the shuffles below take whole warps)
    const int64_t tok = in ? id / C : 0;
    slot[j] = in ? __ldg(p.slots + tok) : -1;
    if (slot[j] >= p.n_slots) slot[j] = -1;
    load8<DT>(src, tok * stride + h * D + 8 * c, x[j]);
  }
#pragma unroll
  for (int j = 0; j < kRowsUnroll; ++j) {
    const __half d = __float2half_rn(first_largest(x[j], lane) * -0.125f);
    uint32_t word = q4_word<DT, V>(x[j], d);
    if (V) {
      // units 2t and 2t + 1 of group g are the halves of `word`; the even group stores both groups' first
      // units, the odd one their second
      const uint32_t other = __shfl_xor_sync(0xffffffffu, word, 4);
      word = (g & 1) ? __byte_perm(other, word, 0x7632) : __byte_perm(word, other, 0x5410);
    }
    if (slot[j] < 0) continue;
    const int off = (int)(slot[j] & (p.g.page_size - 1)), i = off % kKvBlk;
    uint8_t* blk = p.g.pages + (slot[j] >> p.g.page_shift) * p.g.page_bytes + h * p.g.head_bytes +
                   (off / kKvBlk) * B::BYTES;
    *(uint32_t*)(blk + (V ? B::v_unit(i, g & ~1, 2 * t + (g & 1)) : B::k_word(i, g, t))) = word;
    if (t == 0) *(__half*)(blk + (V ? B::v_scale(i, g) : B::k_scale(i, g))) = d;
  }
}

template <int D, int DT>
__global__ void __launch_bounds__(kRowsThreads) kv_append_kernel(const __grid_constant__ KvRows p) {
  pdl_wait();
  pdl_trigger();
  if (blockIdx.z) append_rows<D, DT, true>(p);
  else append_rows<D, DT, false>(p);
}

// The way back, by the same chunks: the codes' words are gathered, whole rows are written.
// (8191 tokens, 8 heads of 128, bf16: 10.5 us, 43 MB at 4.1 TB/s: below HBM's rate because V's units, two tokens
// side by side, are gathered by 2-byte loads, two a lane.)
template <int D, int DT, bool V>
__device__ __forceinline__ void read_rows(const KvRows& p) {
  using B = KvBlk<D>;
  constexpr int C = D / 8;
  const int h = blockIdx.y;
  const int64_t base = (int64_t)blockIdx.x * (kRowsThreads * kRowsUnroll) + threadIdx.x;
  const int c = threadIdx.x % C, g = c / 4, t = c & 3;
  uint32_t word[kRowsUnroll];
  float d[kRowsUnroll];
#pragma unroll
  for (int j = 0; j < kRowsUnroll; ++j) {
    const int64_t id = base + j * kRowsThreads;
    const int64_t slot = __ldg(p.slots + (id < p.items ? id / C : 0));
    const bool in = slot >= 0 && slot < p.n_slots;
    const int off = in ? (int)(slot & (p.g.page_size - 1)) : 0, i = off % kKvBlk;
    const uint8_t* blk = p.g.pages + (in ? slot >> p.g.page_shift : 0) * p.g.page_bytes +
                         h * p.g.head_bytes + (off / kKvBlk) * B::BYTES;
    if (V)
      word[j] = *(const uint16_t*)(blk + B::v_unit(i, g, 2 * t)) |
                (uint32_t)*(const uint16_t*)(blk + B::v_unit(i, g, 2 * t + 1)) << 16;
    else
      word[j] = *(const uint32_t*)(blk + B::k_word(i, g, t));
    d[j] = __half2float(*(const __half*)(blk + (V ? B::v_scale(i, g) : B::k_scale(i, g))));
    if (!in) {                             // zeros, whatever the block in front holds
      d[j] = 0.f;
      word[j] = 0x88888888u;
    }
  }
#pragma unroll
  for (int j = 0; j < kRowsUnroll; ++j) {
    const int64_t id = base + j * kRowsThreads;
    if (id >= p.items) continue;
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      // nibble n, read where it stands: 2^23 + c 2^s is a float for s <= 19, and loses its 2^23 and 8 2^s exactly
      const int n = V ? e : (e >> 1) + 4 * (e & 1);
      const int s = n < 5 ? 4 * n : 4 * n - 20;
      const float y = __uint_as_float(lop3_and_or(n < 5 ? word[j] : word[j] >> 20, 15u << s, 0x4B000000u));
      x[e] = (y - (8388608.f + 8.f * (float)(1 << s))) * (d[j] * (1.f / (float)(1 << s)));
    }
    store8<DT>(V ? p.vo : p.ko, (id / C * p.g.heads + h) * D + 8 * c, x);
  }
}

template <int D, int DT>
__global__ void __launch_bounds__(kRowsThreads) kv_read_kernel(const __grid_constant__ KvRows p) {
  pdl_wait();
  pdl_trigger();
  if (blockIdx.z) read_rows<D, DT, true>(p);
  else read_rows<D, DT, false>(p);
}

// ---------------------------------------------------------------------------
// plan
// ---------------------------------------------------------------------------
struct PlanParams {
  const int32_t* ctx;
  const int32_t* add;
  int B, page_size, page_shift, max_pages, n_pages, T;
  int32_t* table;
  int32_t* stack;
  const int32_t* count;
  int32_t* kv_len;
  int32_t* q_start;
  int64_t* slots;
  int32_t* pos;
  int32_t* count_out;
  int32_t* unserved;
};

constexpr int kPlanThreads = 1024;

// exclusive block sums of three counts at once; `tot` gets their sums
__device__ __forceinline__ void block_scan3(int (&v)[3], int (&tot)[3], int (*part)[3]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    inc[k] = v[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc[k], o);
      if (lane >= o) inc[k] += u;
    }
  }
  __syncthreads();
  if (lane == 31)
    for (int k = 0; k < 3; ++k) part[warp][k] = inc[k];
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      int s = lane < kPlanThreads / 32 ? part[lane][k] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += u;
      }
      part[lane][k] = s;
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    tot[k] = part[kPlanThreads / 32 - 1][k];
    v[k] = inc[k] - v[k] + (warp > 0 ? part[warp - 1][k] : 0);
  }
}

// the last i in [0, n) with first[i] <= x, for ascending first with first[0] <= x
__device__ __forceinline__ int find_last(const int* first, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Every CTA sums all requests' tokens, needs and returned pages (B is at most a
// few thousand lengths, read from L2), so that none waits for another; they
// then share the tokens, the popped and the pushed pages among them.  A page
// that is pushed and popped by one call is found through the request that
// returns it, never through the stack: no CTA reads what another writes.
//
// Bound by the latency of one launch and a few dependent loads: 48 requests of one token
// each 3.9 us in a graph, 1000 requests with prompts and finished ones 7.0 us.
__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(const __grid_constant__ PlanParams p) {
  extern __shared__ int sm[];
  __shared__ int part[32][3];
  __shared__ int taken_s, unserved_s;
  pdl_wait();
  pdl_trigger();
  int* tok0 = sm;                          // [B + 1] new tokens before r
  int* need0 = tok0 + p.B + 1;             // [B + 1] pages needed before r
  int* back0 = need0 + p.B + 1;            // [B + 1] pages returned before r
  uint8_t* state = (uint8_t*)(back0 + p.B + 1);   // 0 not served, 1 served, 2 finished
  const int tid = threadIdx.x;
  const int cap = p.max_pages;
  const int mask = p.page_size - 1;
  if (tid == 0) taken_s = unserved_s = 0;

  int run[3] = {0, 0, 0};
  for (int r0 = 0; r0 < p.B; r0 += kPlanThreads) {
    const int r = r0 + tid;
    int v[3] = {0, 0, 0}, tot[3];
    if (r < p.B) {
      const int ctx = max(__ldg(p.ctx + r), 0), add = __ldg(p.add + r);
      const int have = (int)(((int64_t)ctx + mask) >> p.page_shift);
      const int64_t want = ((int64_t)ctx + max(add, 0) + mask) >> p.page_shift;
      const bool fits = add >= 0 && want <= cap;
      v[0] = max(add, 0);
      v[1] = fits ? (int)want - have : 0;
      v[2] = add < 0 ? min(have, cap) : 0;
      state[r] = add < 0 ? 2 : fits ? 1 : 0;
    }
    block_scan3(v, tot, part);
    if (r < p.B) {
      tok0[r] = run[0] + v[0];
      need0[r] = run[1] + v[1];
      back0[r] = run[2] + v[2];
    }
    for (int k = 0; k < 3; ++k) run[k] += tot[k];
  }
  if (tid == 0) {
    tok0[p.B] = run[0];
    need0[p.B] = run[1];
    back0[p.B] = run[2];
  }
  __syncthreads();
  const int count = min(max(__ldg(p.count), 0), p.n_pages);
  const int returned = run[2];
  const int top = count + returned;
  int taken = 0, miss = 0;
  for (int r = tid; r < p.B; r += kPlanThreads) {
    if (state[r] == 1) {
      if (need0[r + 1] > need0[r]) {
        if (need0[r + 1] <= top) taken = max(taken, need0[r + 1]);
        else state[r] = 0;
      }
    }
    miss += state[r] == 0;
  }
  atomicMax(&taken_s, taken);
  if (miss) atomicAdd(&unserved_s, miss);
  __syncthreads();
  taken = taken_s;

  const int64_t gt = (int64_t)blockIdx.x * kPlanThreads + tid;
  const int64_t gn = (int64_t)gridDim.x * kPlanThreads;
  // page at height x of the stack as it stands after the pushes
  auto page_at = [&](int x) -> int {
    if (x < count) return __ldg(p.stack + x);
    const int r = find_last(back0, p.B, x - count);
    return p.table[(int64_t)r * cap + (x - count - back0[r])];
  };
  for (int64_t r = gt; r < p.B; r += gn) {
    const int ctx = max(__ldg(p.ctx + r), 0), st = state[r];
    p.kv_len[r] = st == 2 ? 0 : st == 1 ? ctx + (tok0[r + 1] - tok0[r]) : ctx;
    p.q_start[r] = tok0[r];
  }
  if (gt == 0) {
    p.q_start[p.B] = run[0];
    *p.count_out = top - taken;
    *p.unserved = unserved_s;
  }
  for (int64_t e = gt; e < returned; e += gn) {
    const int r = find_last(back0, p.B, (int)e);
    if (count + e < p.n_pages)
      p.stack[count + e] = p.table[(int64_t)r * cap + ((int)e - back0[r])];
  }
  for (int64_t e = gt; e < taken; e += gn) {
    const int r = find_last(need0, p.B, (int)e);
    const int have = (int)(((int64_t)max(__ldg(p.ctx + r), 0) + mask) >> p.page_shift);
    const int at = have + ((int)e - need0[r]);
    if (at < cap) p.table[(int64_t)r * cap + at] = page_at(top - 1 - (int)e);
  }
  for (int64_t j = gt; j < p.T; j += gn) {
    int64_t slot = -1;
    int pos = -1;
    if (j < run[0]) {
      const int r = find_last(tok0, p.B, (int)j);
      const int ctx = max(__ldg(p.ctx + r), 0);
      pos = ctx + ((int)j - tok0[r]);
      const int at = pos >> p.page_shift;
      if (state[r] == 1 && at >= 0 && at < cap) {
        const int have = (int)(((int64_t)ctx + mask) >> p.page_shift);
        const int page = at < have ? p.table[(int64_t)r * cap + at]
                                   : page_at(top - 1 - (need0[r] + at - have));
        slot = ((int64_t)page << p.page_shift) + (pos & mask);
      }
    }
    p.slots[j] = slot;
    p.pos[j] = pos;
  }
}

template <int D>
int launch_rows(KvRows p, int T, int dtype, bool append, cudaStream_t s) {
  p.items = (int64_t)T * (D / 8);
  const int64_t ctas = (p.items + kRowsThreads * kRowsUnroll - 1) / (kRowsThreads * kRowsUnroll);
  if (ctas > 2147483647) return DQ_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)ctas, (unsigned)p.g.heads, 2), block(kRowsThreads);
#define DQ_KV_ROWS(DT)                                                                        \
  if (dtype == DT)                                                                            \
    return launched(append ? launch_pdl(kv_append_kernel<D, DT>, grid, block, 0, s, 0, p)     \
                           : launch_pdl(kv_read_kernel<D, DT>, grid, block, 0, s, 0, p));
  DQ_KV_ROWS(DQ_F32)
  DQ_KV_ROWS(DQ_F16)
  DQ_KV_ROWS(DQ_BF16)
#undef DQ_KV_ROWS
  return DQ_ERR_ARG;
}

}  // namespace
}  // namespace dqmoe

using namespace dqmoe;

extern "C" {

int dq_kv_cache_size(const dq_kv_cache* cache, size_t* bytes) {
  if (!bytes) return DQ_ERR_ARG;
  KvGeom g;
  const int rc = kv_check(cache, &g, false);
  if (rc != DQ_OK) return rc;
  *bytes = (size_t)g.page_bytes * (size_t)g.n_pages;
  return DQ_OK;
}

int dq_kv_plan(const int32_t* ctx_len, const int32_t* new_len, int B, int page_size,
               int32_t* block_table, int max_pages, int32_t* free_pages, int n_pages,
               const int32_t* free_count, int T, int32_t* kv_len, int32_t* q_start,
               int64_t* slots, int32_t* positions, int32_t* free_count_out, int32_t* unserved,
               void* stream) {
  if (!ctx_len || !new_len || !block_table || !free_pages || !free_count || !kv_len || !q_start ||
      !free_count_out || !unserved || (T > 0 && (!slots || !positions)))
    return DQ_ERR_ARG;
  if (B <= 0 || T < 0 || max_pages <= 0 || n_pages <= 0 || !kv_page_size_ok(page_size))
    return DQ_ERR_ARG;
  if ((int64_t)max_pages * page_size > 2147483647LL) return DQ_ERR_ARG;
  // (every CTA reads the lengths and the count, whenever it runs)
  if (free_count_out == free_count || kv_len == ctx_len || kv_len == new_len) return DQ_ERR_ARG;
  if (B > DQ_KV_MAX_REQUESTS) return DQ_ERR_UNSUPPORTED;
  const void* p4[] = {ctx_len, new_len, block_table, free_pages, free_count,
                      kv_len, q_start, positions, free_count_out, unserved};
  for (const void* q : p4)
    if (!kv_aligned(q, 4)) return DQ_ERR_ALIGN;
  if (!kv_aligned(slots, 8)) return DQ_ERR_ALIGN;
  PlanParams p;
  p.ctx = ctx_len;
  p.add = new_len;
  p.B = B;
  p.page_size = page_size;
  p.page_shift = 0;
  while ((1 << p.page_shift) < page_size) ++p.page_shift;
  p.max_pages = max_pages;
  p.n_pages = n_pages;
  p.T = T;
  p.table = block_table;
  p.stack = free_pages;
  p.count = free_count;
  p.kv_len = kv_len;
  p.q_start = q_start;
  p.slots = slots;
  p.pos = positions;
  p.count_out = free_count_out;
  p.unserved = unserved;
  const size_t smem = (size_t)(B + 1) * 12 + (size_t)B;
  constexpr size_t kMost = (size_t)(DQ_KV_MAX_REQUESTS + 1) * 12 + DQ_KV_MAX_REQUESTS;
  static bool attr[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DQ_ERR_CUDA;
  if (dev >= 64 || !attr[dev]) {
    if (cudaFuncSetAttribute(kv_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)kMost) != cudaSuccess)
      return DQ_ERR_CUDA;
    if (dev < 64) attr[dev] = true;
  }
  const int grid = (int)std::min<int64_t>(64, std::max<int64_t>(1, ((int64_t)T + 1023) / 1024));
  return launched(launch_pdl(kv_plan_kernel, dim3(grid), dim3(kPlanThreads), smem,
                             (cudaStream_t)stream, 0, p));
}

int dq_kv_append(const dq_kv_cache* cache, const void* k, int64_t k_stride, const void* v,
                 int64_t v_stride, int dtype, const int64_t* slots, int T, void* stream) {
  KvRows p;
  const int rc = kv_check(cache, &p.g, true);
  if (rc != DQ_OK) return rc;
  if (!k || !v || !slots || T <= 0 || (dtype != DQ_F32 && dtype != DQ_F16 && dtype != DQ_BF16))
    return DQ_ERR_ARG;
  const int64_t row = (int64_t)cache->n_kv_heads * cache->head_dim;
  if (k_stride < row || v_stride < row || k_stride > (1LL << 31) || v_stride > (1LL << 31))
    return DQ_ERR_ARG;
  const int el = dtype == DQ_F32 ? 4 : 2;
  if (!kv_aligned(k, 16) || !kv_aligned(v, 16) || k_stride * el % 16 || v_stride * el % 16 ||
      !kv_aligned(slots, 8))
    return DQ_ERR_ALIGN;
  p.k = k;
  p.v = v;
  p.ko = p.vo = nullptr;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.slots = slots;
  p.n_slots = (int64_t)cache->n_pages * cache->page_size;
  return by_dim(cache->head_dim, [&](auto d) {
    return launch_rows<decltype(d)::value>(p, T, dtype, true, (cudaStream_t)stream);
  });
}

int dq_kv_read(const dq_kv_cache* cache, const int64_t* slots, int T, void* k, void* v, int dtype,
               void* stream) {
  KvRows p;
  const int rc = kv_check(cache, &p.g, true);
  if (rc != DQ_OK) return rc;
  if (!k || !v || !slots || T <= 0 || (dtype != DQ_F32 && dtype != DQ_F16 && dtype != DQ_BF16))
    return DQ_ERR_ARG;
  if (!kv_aligned(k, 16) || !kv_aligned(v, 16) || !kv_aligned(slots, 8)) return DQ_ERR_ALIGN;
  p.k = p.v = nullptr;
  p.ko = k;
  p.vo = v;
  p.k_stride = p.v_stride = 0;
  p.slots = slots;
  p.n_slots = (int64_t)cache->n_pages * cache->page_size;
  return by_dim(cache->head_dim, [&](auto d) {
    return launch_rows<decltype(d)::value>(p, T, dtype, false, (cudaStream_t)stream);
  });
}

}  // extern "C"
