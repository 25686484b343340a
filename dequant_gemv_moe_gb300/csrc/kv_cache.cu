// kv_cache.cu — the 4-bit paged K/V cache: a step's block tables and slots
// (dq_kv_plan), K/V rows into it as Q4_0 blocks (dq_kv_append) and back out
// (dq_kv_read).
#include <algorithm>

#include "kv.cuh"

namespace dqmoe {

namespace {

template <int DT>
struct Elem;
template <> struct Elem<DQ_F32> { using T = float; };
template <> struct Elem<DQ_F16> { using T = __half; };
template <> struct Elem<DQ_BF16> { using T = __nv_bfloat16; };

// four consecutive values as fp32
template <int DT>
__device__ __forceinline__ void load4(const void* p, int64_t i, float (&x)[4]) {
  if (DT == DQ_F32) {
    const float4 v = __ldg((const float4*)((const float*)p + i));
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  } else {
    const uint2 v = __ldg((const uint2*)((const unsigned short*)p + i));
    if (DT == DQ_BF16) {
      x[0] = __uint_as_float(v.x << 16);
      x[1] = __uint_as_float(v.x & 0xFFFF0000u);
      x[2] = __uint_as_float(v.y << 16);
      x[3] = __uint_as_float(v.y & 0xFFFF0000u);
    } else {
      const float2 a = __half22float2(u32_as_h2(v.x)), b = __half22float2(u32_as_h2(v.y));
      x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
    }
  }
}

template <int DT>
__device__ __forceinline__ void store4(void* p, int64_t i, const float (&x)[4]) {
  if (DT == DQ_F32) {
    *(float4*)((float*)p + i) = make_float4(x[0], x[1], x[2], x[3]);
  } else if (DT == DQ_BF16) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    *(uint2*)((__nv_bfloat16*)p + i) = make_uint2(*(const uint32_t*)&a, *(const uint32_t*)&b);
  } else {
    const __half2 a = __floats2half2_rn(x[0], x[1]), b = __floats2half2_rn(x[2], x[3]);
    *(uint2*)((__half*)p + i) = make_uint2(h2_as_u32(a), h2_as_u32(b));
  }
}

// The Q4_0 codes and scale of the 32 values that 8 consecutive lanes hold four
// of each.  The scale takes the first value of the largest magnitude, so a tie
// between lanes goes to the lower one.  x / d is the correctly rounded
// quotient: for 16-bit x the code then equals that of exact arithmetic (x and d
// have at most 11 bits, so a quotient that is not itself half-way between two
// codes differs from half-way by at least 2^-14, and the sum with 8.5 rounds by
// less than 2^-20).
__device__ __forceinline__ __half quantise4(const float (&xin)[4], int lane, uint32_t (&c)[4]) {
  float x[4], m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = fminf(fmaxf(xin[i], -65504.f), 65504.f);
    if (fabsf(x[i]) > fabsf(m)) m = x[i];
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    const float p = __shfl_xor_sync(0xffffffffu, m, o);
    const bool mine = fabsf(m) > fabsf(p) || (fabsf(m) == fabsf(p) && (lane & o) == 0);
    m = mine ? m : p;
  }
  const __half d = __float2half_rn(m * -0.125f);
  const float df = __half2float(d);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float q = floorf(__fadd_rn(__fdiv_rn(x[i], df), 8.5f));
    c[i] = df == 0.f ? 8u : (uint32_t)fminf(fmaxf(q, 0.f), 15.f);
  }
  return d;
}

struct KvRows {
  KvGeom g;
  const void* k;
  const void* v;
  void* ko;
  void* vo;
  int64_t k_stride, v_stride;
  const int64_t* slots;
  int64_t n_slots;
  int T;
};

// One warp per (token, head); a lane holds four consecutive values of each 128.
template <int D, int DT>
__global__ void __launch_bounds__(256) kv_append_kernel(const __grid_constant__ KvRows p) {
  using B = KvBlk<D>;
  pdl_wait();
  pdl_trigger();
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int64_t tok = w / p.g.heads;
  const int h = (int)(w - tok * p.g.heads);
  if (tok >= p.T) return;
  const int64_t slot = __ldg(p.slots + tok);
  if (slot < 0 || slot >= p.n_slots) return;
  const int off = (int)(slot & (p.g.page_size - 1));
  uint8_t* blk = p.g.pages + (slot >> p.g.page_shift) * p.g.page_bytes + h * p.g.head_bytes +
                 (off / kKvBlk) * B::BYTES;
  const int i = off % kKvBlk;
  constexpr int LANES = D < 128 ? D / 4 : 32;
#pragma unroll
  for (int r = 0; r < (D + 127) / 128; ++r) {
    // lanes without values of their own (D = 64) repeat the last ones and store nothing
    const int l = lane < LANES ? lane : LANES - 8 + (lane & 7);
    const int grp = r * 4 + l / 8, a = l & 7;
    float x[4], y[4];
    load4<DT>(p.k, tok * p.k_stride + (int64_t)h * D + grp * 32 + 4 * a, x);
    load4<DT>(p.v, tok * p.v_stride + (int64_t)h * D + grp * 32 + 4 * a, y);
    uint32_t c[4], e[4];
    const __half dk = quantise4(x, lane, c), dv = quantise4(y, lane, e);
    uint32_t kw = (c[0] | c[1] << 16 | c[2] << 4 | c[3] << 20) << (8 * (a & 1));
    kw |= __shfl_xor_sync(0xffffffffu, kw, 1);
    if (lane < LANES) {
      if (!(a & 1)) *(uint32_t*)(blk + B::k_word(i, grp, a >> 1)) = kw;
      *(uint16_t*)(blk + B::v_unit(i, grp, a)) =
          (uint16_t)(e[0] | e[1] << 4 | e[2] << 8 | e[3] << 12);
      if (a == 0) {
        *(__half*)(blk + B::k_scale(i, grp)) = dk;
        *(__half*)(blk + B::v_scale(i, grp)) = dv;
      }
    }
  }
}

template <int D, int DT>
__global__ void __launch_bounds__(256) kv_read_kernel(const __grid_constant__ KvRows p) {
  using B = KvBlk<D>;
  pdl_wait();
  pdl_trigger();
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int64_t tok = w / p.g.heads;
  const int h = (int)(w - tok * p.g.heads);
  if (tok >= p.T) return;
  const int64_t slot = __ldg(p.slots + tok);
  const bool in = slot >= 0 && slot < p.n_slots;
  const int off = in ? (int)(slot & (p.g.page_size - 1)) : 0;
  const uint8_t* blk = p.g.pages + (in ? slot >> p.g.page_shift : 0) * p.g.page_bytes +
                       h * p.g.head_bytes + (off / kKvBlk) * B::BYTES;
  const int i = off % kKvBlk;
#pragma unroll
  for (int r = 0; r < (D + 127) / 128; ++r) {
    const int grp = r * 4 + lane / 8, a = lane & 7;
    if (grp >= B::G) return;
    float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
    if (in) {
      const uint32_t kw = *(const uint32_t*)(blk + B::k_word(i, grp, a >> 1)) >> (8 * (a & 1));
      const uint32_t vw = *(const uint16_t*)(blk + B::v_unit(i, grp, a));
      const float dk = __half2float(*(const __half*)(blk + B::k_scale(i, grp)));
      const float dv = __half2float(*(const __half*)(blk + B::v_scale(i, grp)));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // value e sits in nibble (e >> 1) + 4 * (e & 1) of the half of the word
        x[e] = dk * (float)((int)(kw >> (4 * (e >> 1) + 16 * (e & 1)) & 15u) - 8);
        y[e] = dv * (float)((int)(vw >> (4 * e) & 15u) - 8);
      }
    }
    const int64_t at = (tok * p.g.heads + h) * D + grp * 32 + 4 * a;
    store4<DT>(p.ko, at, x);
    store4<DT>(p.vo, at, y);
  }
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

template <typename F>
int by_dim(int dim, F f) {
  switch (dim) {
    case 64: return f(std::integral_constant<int, 64>());
    case 128: return f(std::integral_constant<int, 128>());
    default: return f(std::integral_constant<int, 256>());
  }
}

int launched(cudaError_t e) {
  if (e != cudaSuccess) return DQ_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? DQ_OK : DQ_ERR_CUDA;
}

template <int D>
int launch_rows(const KvRows& p, int dtype, bool append, cudaStream_t s) {
  const int64_t ctas = ((int64_t)p.T * p.g.heads + 7) / 8;
  if (ctas > 2147483647) return DQ_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)ctas), block(256);
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
  if (free_count_out == free_count || kv_len == ctx_len) return DQ_ERR_ARG;
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
  p.T = T;
  return by_dim(cache->head_dim, [&](auto d) {
    return launch_rows<decltype(d)::value>(p, dtype, true, (cudaStream_t)stream);
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
  p.T = T;
  return by_dim(cache->head_dim, [&](auto d) {
    return launch_rows<decltype(d)::value>(p, dtype, false, (cudaStream_t)stream);
  });
}

}  // extern "C"
