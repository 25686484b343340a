// kv_rope.cu — dq_kv_append_rope: a step's q and k rows rotated by their positions, q
// written to its rows, k and v into the cache as Q4_0 blocks.
//
// Mathematics.  The pair (a, b) of frequency i turns by angle = position * inv_freq[i]:
//   a' = f (a cos - b sin),  b' = f (b cos + a sin).
// * Angles.  A position times a frequency reaches 10^6 and more, where fp32 holds no fraction of a turn.
//   With inv_freq / 2 pi as two floats (from one product in 64 bits) the turns are a product and its
//   exact error (FMA) and the low part's; the whole turns are taken off exactly, and what the last
//   addition rounds off comes back as a first-order term: cos and sin within 2e-7, for positions below
//   2^24.  Beyond, the turns are formed in 64 bits.
// * K's codes are those of the rotated row in 64 bits, not of its rounding: a code or a scale next to a
//   border would otherwise depend on how the rotation was rounded, and an equal pair of largest magnitudes
//   decides the sign of a scale.  The fp32 rotation knows its error (kErr of |a| + |b|), and where a group has
//   a value that close to a border, that value is formed in 64 bits.  (bf16 rows, heads of 128: a
//   warp's 256 values in about 250.)
#include <algorithm>

#include "kv_rows.cuh"

namespace dqmoe {

namespace {

struct RopeParams {
  KvGeom g;
  const void* q;
  const void* k;
  const void* v;
  int64_t q_stride, k_stride, v_stride;
  const int64_t* slots;
  int64_t n_slots;
  const int32_t* pos;
  const float* freq;
  int half;                    // frequencies: half of the values that turn
  int interleaved;
  float factor;
  int T, q_heads;
  void* out;
  int64_t out_stride;
  int out_dtype;
  int tile;                    // tokens a CTA takes
};

constexpr int kRopeThreads = 256;
constexpr int kMostTile = 4;
// of |a| + |b|: cos and sin 2e-7, their product with the factor, the product and the sum 2^-24 each
constexpr float kErr = 4.5e-7f;
constexpr int kFarPosition = 1 << 24;
constexpr float kErrFar = 2e-6f;           // (positions above it, whose turns are known to 2^-52 of themselves)

// cos and sin of pos * freq, times the factor
__device__ __forceinline__ float2 turn(int pos, float freq, float factor) {
  const double g = (double)freq * 0.15915494309189533577;        // 1 / 2 pi
  float r, rest;
  if (pos < kFarPosition) {
    const float gh = (float)g, gl = (float)(g - (double)gh), p = (float)pos;
    const float hi = p * gh, lo = fmaf(p, gl, fmaf(p, gh, -hi));
    const float part = hi - rintf(hi);
    r = part + lo;
    rest = lo - (r - part);
  } else {
    const double t = (double)pos * g;
    r = (float)(t - rint(t));
    rest = 0.f;
  }
  float s, c;
  sincospif(2.f * r, &s, &c);
  rest *= 6.2831853f;
  return make_float2(fmaf(-rest, s, c) * factor, fmaf(rest, c, s) * factor);
}

// eight values that this thread may overwrite later
template <int DT>
__device__ __forceinline__ void load8_rw(const void* p, int64_t i, float (&x)[8]) {
  if (DT == DQ_F32) {
    const float4* s = (const float4*)((const float*)p + i);
    const float4 a = s[0], b = s[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
    const uint4 v = *(const uint4*)((const unsigned short*)p + i);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (DT == DQ_BF16) {
        x[2 * k] = __uint_as_float(w[k] << 16);
        x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
      } else {
        const float2 f = __half22float2(u32_as_h2(w[k]));
        x[2 * k] = f.x;
        x[2 * k + 1] = f.y;
      }
    }
  }
}

__device__ __forceinline__ void store8_any(int dtype, void* p, int64_t i, const float (&x)[8]) {
  if (dtype == DQ_BF16) store8<DQ_BF16>(p, i, x);
  else if (dtype == DQ_F16) store8<DQ_F16>(p, i, x);
  else store8<DQ_F32>(p, i, x);
}

// ---------------------------------------------------------------- q
// A thread takes the sixteen values of eight pairs: two chunks of eight that stand `half` apart, or
// next to one another; the values that do not turn go through in sixteens.
template <int D, int DT>
__device__ __forceinline__ void rope_q(const RopeParams& p, const float2* cs, int t0, int n) {
  constexpr int U = D / 16, ROWS = kRopeThreads / U;
  const int u = threadIdx.x % U;
  const bool turns = 8 * u < p.half;
  const int c0 = p.interleaved || !turns ? 2 * u : u, c1 = p.interleaved || !turns ? 2 * u + 1 : u + p.half / 8;
  for (int r = threadIdx.x / U; r < n * p.q_heads; r += ROWS) {
    const int tt = r / p.q_heads, h = r - tt * p.q_heads, t = t0 + tt;
    if (__ldg(p.pos + t) < 0) continue;
    const int64_t at = (int64_t)t * p.q_stride + (int64_t)h * D, to = (int64_t)t * p.out_stride + (int64_t)h * D;
    float x[8], y[8];
    load8_rw<DT>(p.q, at + 8 * c0, x);
    load8_rw<DT>(p.q, at + 8 * c1, y);
    if (turns) {
      const float2* w = cs + tt * p.half + 8 * u;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float& a = p.interleaved ? (i < 4 ? x[2 * (i & 3)] : y[2 * (i & 3)]) : x[i];
        float& b = p.interleaved ? (i < 4 ? x[2 * (i & 3) + 1] : y[2 * (i & 3) + 1]) : y[i];
        const float2 z = w[i];
        const float na = fmaf(a, z.x, -(b * z.y)), nb = fmaf(b, z.x, a * z.y);
        a = na;
        b = nb;
      }
    }
    store8_any(p.out_dtype, p.out, to + 8 * c0, x);
    store8_any(p.out_dtype, p.out, to + 8 * c1, y);
  }
}

// ---------------------------------------------------------------- k
// A value in 64 bits: own cos + sign other sin.
__device__ __noinline__ double turned64(float own, float other, float sign, int pos, float freq, float factor) {
  double s, c;
  sincos((double)pos * (double)freq, &s, &c);
  const double x = ((double)own * c + (double)sign * (double)other * s) * (double)factor;
  return fmin(fmax(x, -65504.), 65504.);
}

// The four lanes of a group hold eight values x each, known to `err`; `exact(e)` gives value e in 64 bits.  Returns
// the word of codes and the scale.  Every lane of the warp calls it.
template <typename F>
__device__ __forceinline__ uint32_t k_word_known(const float (&x)[8], float err, int lane, __half& d, F exact) {
  float hi = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
  float lo = fminf(fminf(fminf(x[0], x[1]), fminf(x[2], x[3])), fminf(fminf(x[4], x[5]), fminf(x[6], x[7])));
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    err = fmaxf(err, __shfl_xor_sync(0xffffffffu, err, o));
  }
  const float top = fmaxf(hi, -lo);
  float m = hi > -lo ? hi : lo;
  d = __float2half_rn(m * -0.125f);
  // which sign the largest has, and which scale its eighth rounds to
  const bool unsure = fabsf(hi + lo) <= 2.f * err || top + err >= 65504.f ||
                      __half_as_ushort(__float2half_rn((top - err) * 0.125f)) !=
                          __half_as_ushort(__float2half_rn((top + err) * 0.125f));
  if (__any_sync(0xffffffffu, unsure)) {
    double best = -1., val = 0.;
    if (unsure) {
#pragma unroll 1
      for (int e = 0; e < 8; ++e) {
        float xe = x[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) xe = e == i ? x[i] : xe;
        if (fabsf(xe) >= top - 2.f * err) {
          const double y = exact(e);
          if (fabs(y) > best) {
            best = fabs(y);
            val = y;
          }
        }
      }
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      const double ob = __longlong_as_double(__shfl_xor_sync(0xffffffffu, __double_as_longlong(best), o));
      const double ov = __longlong_as_double(__shfl_xor_sync(0xffffffffu, __double_as_longlong(val), o));
      if (ob > best || (ob == best && (lane & o) != 0)) {
        best = ob;
        val = ov;
      }
    }
    if (unsure) d = __double2half(val * -0.125);
  }
  const float df = __half2float(d), inv = df == 0.f ? 0.f : __frcp_rn(df);
  // the quotient's own error: the reciprocal, the product and the sum
  const float room = err * fabsf(inv) + 1.5e-6f;
  uint32_t word = 0, near = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float y = fmaf(x[e], inv, 8.5f);
    const float c = fminf(fmaxf(floorf(y), 0.f), 15.f);
    const float k = rintf(y);
    near |= fabsf(y - k) <= room && k >= 1.f && k <= 15.f && df != 0.f ? 1u << e : 0u;
    word |= (uint32_t)c << (4 * (e >> 1) + 16 * (e & 1));
  }
  if (__any_sync(0xffffffffu, near != 0)) {
#pragma unroll 1
    for (; near; near &= near - 1) {
      const int e = __ffs(near) - 1, at = 4 * (e >> 1) + 16 * (e & 1);
      const double c = fmin(fmax(floor(exact(e) / (double)df + 8.5), 0.), 15.);
      word = (word & ~(15u << at)) | (uint32_t)c << at;
    }
  }
  return word;
}

// Eight values per thread, a group of 32 four lanes, as in dq_kv_append; the other halves of the pairs are
// loaded too (from L1: their own threads load them).
template <int D, int DT>
__device__ __forceinline__ void rope_k(const RopeParams& p, const float2* cs, int t0, int n) {
  using B = KvBlk<D>;
  constexpr int C = D / 8, ROWS = kRopeThreads / C;
  const int lane = threadIdx.x & 31, c = threadIdx.x % C, g = c / 4, t4 = c & 3;
  const int rows = n * p.g.heads;
  const bool turns = 4 * c < p.half;
  const bool second = !p.interleaved && 8 * c >= p.half;      // of its pairs (half apart)
  const int i0 = p.interleaved ? 4 * c : second ? 8 * c - p.half : 8 * c;
  const int other = p.interleaved || !turns ? c : second ? c - p.half / 8 : c + p.half / 8;
  for (int r0 = 0; r0 < rows; r0 += ROWS) {
    const int r = r0 + (int)threadIdx.x / C;
    const bool in = r < rows;                                  // (the shuffles below take whole warps)
    const int tt = in ? r / p.g.heads : 0, h = in ? r - tt * p.g.heads : 0, t = t0 + tt;
    const int pos = __ldg(p.pos + t);
    int64_t slot = in && pos >= 0 ? __ldg(p.slots + t) : -1;
    if (slot >= p.n_slots) slot = -1;
    const int64_t at = (int64_t)t * p.k_stride + (int64_t)h * D;
    float raw[8], oth[8], x[8], err = 0.f;
    load8<DT>(p.k, at + 8 * c, raw);
    load8<DT>(p.k, at + 8 * other, oth);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = raw[e];
    if (turns && pos >= 0) {
      const float2* w = cs + tt * p.half + i0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 z = p.interleaved ? w[e >> 1] : w[e];
        const float b = p.interleaved ? raw[e ^ 1] : oth[e];
        const float s = p.interleaved ? ((e & 1) ? z.y : -z.y) : second ? z.y : -z.y;
        x[e] = fmaf(raw[e], z.x, b * s);
        err = fmaxf(err, fabsf(raw[e]) + fabsf(b));
      }
      err *= p.factor * (pos < kFarPosition ? kErr : kErrFar);
    }
    __half d;
    uint32_t word;
    const bool all = __all_sync(0xffffffffu, !turns);          // (values as they are need no bounds)
    if (DT != DQ_F32 && all) {
      d = __float2half_rn(first_largest(x, lane) * -0.125f);
      word = q4_word<DT, false>(x, d);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = fminf(fmaxf(x[e], -65504.f), 65504.f);
      word = k_word_known(x, err, lane, d, [&](int e) -> double {
        float own = raw[0], b = p.interleaved ? raw[1] : oth[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) {
          own = e == i ? raw[i] : own;
          b = e == i ? (p.interleaved ? raw[i ^ 1] : oth[i]) : b;
        }
        if (!turns) return fmin(fmax((double)own, -65504.), 65504.);
        const bool minus = p.interleaved ? (e & 1) == 0 : !second;
        return turned64(own, b, minus ? -1.f : 1.f, pos, __ldg(p.freq + i0 + (p.interleaved ? e >> 1 : e)), p.factor);
      });
    }
    if (slot < 0) continue;
    const int off = (int)(slot & (p.g.page_size - 1)), i = off % kKvBlk;
    uint8_t* blk = p.g.pages + (slot >> p.g.page_shift) * p.g.page_bytes + h * p.g.head_bytes + (off / kKvBlk) * B::BYTES;
    *(uint32_t*)(blk + B::k_word(i, g, t4)) = word;
    if (t4 == 0) *(__half*)(blk + B::k_scale(i, g)) = d;
  }
}

// ---------------------------------------------------------------- v, as dq_kv_append writes it
template <int D, int DT>
__device__ __forceinline__ void rope_v(const RopeParams& p, int t0, int n) {
  using B = KvBlk<D>;
  constexpr int C = D / 8, ROWS = kRopeThreads / C;
  const int lane = threadIdx.x & 31, c = threadIdx.x % C, g = c / 4, t4 = c & 3;
  const int rows = n * p.g.heads;
  for (int r0 = 0; r0 < rows; r0 += ROWS) {
    const int r = r0 + (int)threadIdx.x / C;
    const bool in = r < rows;
    const int tt = in ? r / p.g.heads : 0, h = in ? r - tt * p.g.heads : 0, t = t0 + tt;
    int64_t slot = in && __ldg(p.pos + t) >= 0 ? __ldg(p.slots + t) : -1;
    if (slot >= p.n_slots) slot = -1;
    float x[8];
    load8<DT>(p.v, (int64_t)t * p.v_stride + (int64_t)h * D + 8 * c, x);
    const __half d = __float2half_rn(first_largest(x, lane) * -0.125f);
    uint32_t word = q4_word<DT, true>(x, d);
    const uint32_t other = __shfl_xor_sync(0xffffffffu, word, 4);
    word = (g & 1) ? __byte_perm(other, word, 0x7632) : __byte_perm(word, other, 0x5410);
    if (slot < 0) continue;
    const int off = (int)(slot & (p.g.page_size - 1)), i = off % kKvBlk;
    uint8_t* blk = p.g.pages + (slot >> p.g.page_shift) * p.g.page_bytes + h * p.g.head_bytes + (off / kKvBlk) * B::BYTES;
    *(uint32_t*)(blk + B::v_unit(i, g & ~1, 2 * t4 + (g & 1))) = word;
    if (t4 == 0) *(__half*)(blk + B::v_scale(i, g)) = d;
  }
}

// blockIdx.y: 0 K, 1 V, 2 q (what takes longest to start first); blockIdx.x: `tile` tokens.
template <int D, int DT>
__global__ void __launch_bounds__(kRopeThreads) kv_rope_kernel(const __grid_constant__ RopeParams p) {
  __shared__ float2 cs[kMostTile * D / 2];
  pdl_wait();
  pdl_trigger();
  const int t0 = blockIdx.x * p.tile, n = min(p.tile, p.T - t0);
  if (blockIdx.y == 1) {
    rope_v<D, DT>(p, t0, n);
    return;
  }
  for (int i = threadIdx.x; i < n * p.half; i += kRopeThreads) {
    const int tt = i / p.half;
    cs[i] = turn(max(0, __ldg(p.pos + t0 + tt)), __ldg(p.freq + i - tt * p.half), p.factor);
  }
  __syncthreads();
  if (blockIdx.y == 0) rope_k<D, DT>(p, cs, t0, n);
  else rope_q<D, DT>(p, cs, t0, n);
}

template <int D>
int launch_rope(const RopeParams& p, int dtype, cudaStream_t s) {
  const dim3 grid((unsigned)((p.T + p.tile - 1) / p.tile), p.q ? 3 : 2), block(kRopeThreads);
#define DQ_KV_ROPE(DT) \
  if (dtype == DT) return launched(launch_pdl(kv_rope_kernel<D, DT>, grid, block, 0, s, 0, p));
  DQ_KV_ROPE(DQ_F32)
  DQ_KV_ROPE(DQ_F16)
  DQ_KV_ROPE(DQ_BF16)
#undef DQ_KV_ROPE
  return DQ_ERR_ARG;
}

}  // namespace
}  // namespace dqmoe

using namespace dqmoe;

extern "C" int dq_kv_append_rope(const dq_kv_cache* cache, const dq_kv_rope* a, void* stream) {
  RopeParams p;
  const int rc = kv_check(cache, &p.g, true);
  if (rc != DQ_OK) return rc;
  if (!a || !a->k || !a->v || !a->slots || !a->positions || !a->inv_freq || a->T <= 0 ||
      (a->q && !a->q_out) || (a->dtype != DQ_F32 && a->dtype != DQ_F16 && a->dtype != DQ_BF16))
    return DQ_ERR_ARG;
  const int64_t D = cache->head_dim, row = cache->n_kv_heads * D;
  if (a->k_stride < row || a->v_stride < row || a->k_stride > (1LL << 31) || a->v_stride > (1LL << 31) ||
      a->rotary_dim <= 0 || a->rotary_dim > D || (a->interleaved != 0 && a->interleaved != 1) ||
      !(a->factor > 0.f) || !(a->factor <= 1e4f))
    return DQ_ERR_ARG;
  if (a->q) {
    if (a->n_q_heads <= 0 || a->q_stride < a->n_q_heads * D || a->out_stride < a->n_q_heads * D ||
        a->q_stride > (1LL << 31) || a->out_stride > (1LL << 31) || a->out_dtype < DQ_F32 ||
        a->out_dtype > DQ_BF16)
      return DQ_ERR_ARG;
    // a row is written while others are read: only where each of its values is read first
    if (a->q_out == a->q && (a->out_dtype != a->dtype || a->out_stride != a->q_stride)) return DQ_ERR_ARG;
  }
  if (a->rotary_dim % 16 || a->T > (1 << 24) || (a->q && a->n_q_heads > 4096)) return DQ_ERR_UNSUPPORTED;
  const int el = a->dtype == DQ_F32 ? 4 : 2, oel = a->out_dtype == DQ_F32 ? 4 : 2;
  if (!kv_aligned(a->k, 16) || !kv_aligned(a->v, 16) || a->k_stride * el % 16 || a->v_stride * el % 16 ||
      !kv_aligned(a->slots, 8) || !kv_aligned(a->positions, 4) || !kv_aligned(a->inv_freq, 4))
    return DQ_ERR_ALIGN;
  if (a->q && (!kv_aligned(a->q, 16) || !kv_aligned(a->q_out, 16) || a->q_stride * el % 16 || a->out_stride * oel % 16))
    return DQ_ERR_ALIGN;
  p.q = a->q;
  p.k = a->k;
  p.v = a->v;
  p.q_stride = a->q_stride;
  p.k_stride = a->k_stride;
  p.v_stride = a->v_stride;
  p.slots = a->slots;
  p.n_slots = (int64_t)cache->n_pages * cache->page_size;
  p.pos = a->positions;
  p.freq = a->inv_freq;
  p.half = a->rotary_dim / 2;
  p.interleaved = a->interleaved;
  p.factor = a->factor;
  p.T = a->T;
  p.q_heads = a->q ? a->n_q_heads : 0;
  p.out = a->q_out;
  p.out_stride = a->out_stride;
  p.out_dtype = a->out_dtype;
  p.tile = a->T >= 1024 ? kMostTile : 1;
  return by_dim(cache->head_dim,
                [&](auto d) { return launch_rope<decltype(d)::value>(p, a->dtype, (cudaStream_t)stream); });
}
