// kv_rope.cu — dq_kv_append_rope: a step's q and k rows rotated by their positions, q
// written to its rows, k and v into the cache as Q4_0 blocks.
//
// Mathematics.  The pair (a, b) of frequency i turns by angle = position * inv_freq[i]:
//   a' = f (a cos - b sin),  b' = f (b cos + a sin).
// * Angles.  A position times a frequency reaches 10^6 and more, where fp32 holds no fraction of a turn.
//   With inv_freq / 2 pi as two floats the turns are a product and its exact error (FMA) and the low part's;
//   the whole turns are taken off exactly, and what the last addition rounds off comes back as a first-order
//   term: cos and sin within 2.3e-7, for positions below 2^24.  Beyond, the turns are formed in 64 bits.
// * A group's scale is the fp16 nearest to -1/8 of its largest value's fp32, as of rows that come in fp32: the rotation in
//   64 bits, rounded to fp32 and then to fp16 (rounded to fp16 at once, one scale in 25000 is its neighbour).  K's codes are
//   those of the rotated row in 64 bits for that scale.  Neither may depend on how a kernel rounds its rotation next to a
//   border, and of an equal pair of largest magnitudes the first decides the sign of the scale.  The fp32 rotation knows its error (kErr of |a| + |b|), and where a group has
//   a value that close to a border, that value is formed again, to 2^-44 (pair.cuh).  (bf16 rows, heads of 128: a
//   warp's 256 values in about 250.)
//
// What bounds it.  A prompt of 8191 tokens (32 query heads, 8 K/V heads of 128, bf16: 177 MB) takes 44.7 us, 4.0
// TB/s: K and V by themselves 23.4 us, which are instructions (a K value's range, bounds, quotient, clamp and
// packing; issue in 0.58 of the cycles), q the rest, which waits for its loads (two heads' worth a lane in flight).
// With an angle per head and thread from shared memory, and K's doubts in 64 bits, it was 96 us.  64 tokens
// 4.1 us (left out for a measurement, K's doubts, one warp's or two's, were 1.6 of 4.7).
#include "kv_rows.cuh"
#include "pair.cuh"

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
  int q_each, q_splits;        // heads of a warp, warps of a token
  uint32_t k_inv;              // of the K/V heads, for row_of
  void* out;
  int64_t out_stride;
  int out_dtype;
  int tile;                    // tokens a CTA takes
};

constexpr int kRopeThreads = 256;
constexpr int kMostTile = 8;             // tokens of a CTA in a long call
constexpr int kTileCtas = 300;
constexpr int kLongCall = 1024;
// of |a| + |b|: cos and sin 2.3e-7 with the factor's product, a product and a sum of 2^-24 each
constexpr float kErr = 4.5e-7f;
constexpr int kFarPosition = 1 << 24;
constexpr float kErrFar = 2e-6f;           // (positions above it, whose turns are known to 2^-52 of themselves)

// (of its own, so that nothing of it is worked out for nearer positions)
__device__ __noinline__ float far_turns(int pos, float freq) {
  const double t = (double)pos * ((double)freq * 0.15915494309189533577);      // 1 / 2 pi
  return (float)(t - rint(t));
}

// cos and sin of pos * freq, times the factor
__device__ __forceinline__ float2 turn(int pos, float freq, float factor) {
  // freq / 2 pi
  const float ch = 0x1.45f306p-3f, cl = 0x1.b9391p-28f;
  const float gh = __fmul_rn(freq, ch), gl = fmaf(freq, cl, __fmaf_rn(freq, ch, -gh)), p = (float)pos;
  const float hi = __fmul_rn(p, gh), lo = fmaf(p, gl, __fmaf_rn(p, gh, -hi));
  const float part = hi - rintf(hi);
  float r = __fadd_rn(part, lo), rest = (lo - (r - part)) * 6.2831853f;
  if (pos >= kFarPosition) {
    r = far_turns(pos, freq);
    rest = 0.f;
  }
  float s, c;
  sincospif(2.f * r, &s, &c);
  return make_float2(fmaf(-rest, s, c) * factor, fmaf(rest, c, s) * factor);
}

// a row of `tile` tokens' heads as (token, head): floor(r / heads) by its inverse, floor(2^32 / heads) + 1
__device__ __forceinline__ int row_of(int r, int heads, uint32_t inv, int& head) {
  const int t = heads == 1 ? r : (int)__umulhi((uint32_t)r, inv);
  head = r - t * heads;
  return t;
}

// eight values as they stand, which this thread may overwrite later
template <int DT>
struct Raw8 {
  uint4 v[DT == DQ_F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    if (DT == DQ_F32) {
      v[0] = ((const uint4*)((const float*)p + i))[0];
      v[DT == DQ_F32] = ((const uint4*)((const float*)p + i))[1];
    } else {
      v[0] = *(const uint4*)((const unsigned short*)p + i);
    }
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
    if (DT == DQ_F32) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint4 w = v[DT == DQ_F32 ? k : 0];
        x[4 * k] = __uint_as_float(w.x);
        x[4 * k + 1] = __uint_as_float(w.y);
        x[4 * k + 2] = __uint_as_float(w.z);
        x[4 * k + 3] = __uint_as_float(w.w);
      }
    } else {
      const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = DT == DQ_F16 ? __half22float2(u32_as_h2(w[k]))
                                      : make_float2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u));
        x[2 * k] = f.x;
        x[2 * k + 1] = f.y;
      }
    }
  }
};

__device__ __forceinline__ void store8_any(int dtype, void* p, int64_t i, const float (&x)[8]) {
  if (dtype == DQ_BF16) store8<DQ_BF16>(p, i, x);
  else if (dtype == DQ_F16) store8<DQ_F16>(p, i, x);
  else store8<DQ_F32>(p, i, x);
}

// What a CTA keeps of its tokens: cosines and sines apart, so that neighbouring pairs' are packed operands.
template <int D>
struct Angles {
  float c[kMostTile * D / 2], s[kMostTile * D / 2];
  int pos[kMostTile];
  int64_t slot[kMostTile];
};

// ---------------------------------------------------------------- q
// A warp takes a token and up to `q_each` of its heads, by itself: 32 / U heads at a time, of which a lane
// takes sixteen values, eight pairs: two chunks of eight that stand `half` apart, or next to one another (the
// values that do not turn go through in sixteens).  A lane's eight angles are those of all its heads; the lanes of
// one unit work out a share of them each.  The first heads' loads are under way meanwhile.
template <int D, int DT>
__device__ __forceinline__ void rope_q(const RopeParams& p, int item) {
  constexpr int U = D / 16, HL = 32 / U, PER = 8 / HL;       // units, heads at a time, angles a lane works out
  constexpr int N = DT == DQ_F32 ? 1 : 2;                    // such steps whose loads are in flight together
  const int lane = threadIdx.x & 31, u = lane % U, hl = lane / U;
  const int t = item / p.q_splits, h0 = (item - t * p.q_splits) * p.q_each, h1 = min(h0 + p.q_each, p.q_heads);
  if (t >= p.T) return;
  const int pos = __ldg(p.pos + t);
  if (pos < 0) return;
  const bool turns = 8 * u < p.half, near = p.interleaved || !turns;
  const int c0 = near ? 2 * u : u, c1 = near ? 2 * u + 1 : u + p.half / 8;
  const int64_t at = (int64_t)t * p.q_stride, to = (int64_t)t * p.out_stride;
  Raw8<DT> a[N], b[N];
  auto load = [&](int h) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (h + j * HL >= h1) continue;
      a[j].load(p.q, at + (int64_t)(h + j * HL) * D + 8 * c0);
      b[j].load(p.q, at + (int64_t)(h + j * HL) * D + 8 * c1);
    }
  };
  int h = h0 + hl;
  load(h);
  float2 c[4], z[4];                                         // cosines and sines, two pairs' together
  {
    float2 mine[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k)
      mine[k] = turns ? turn(pos, __ldg(p.freq + 8 * u + hl * PER + k), p.factor) : make_float2(1.f, 0.f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = __shfl_sync(0xffffffffu, mine[i % PER].x, u + U * (i / PER));
      const float y = __shfl_sync(0xffffffffu, mine[i % PER].y, u + U * (i / PER));
      if (i & 1) {
        c[i / 2].y = x;
        z[i / 2].y = y;
      } else {
        c[i / 2].x = x;
        z[i / 2].x = y;
      }
    }
  }
  while (true) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (h + j * HL >= h1) continue;
      float x[8], y[8];
      a[j].values(x);
      b[j].values(y);
      if (turns) {
        auto pair = [&](int i, float& v0, float& v1) {
          const float ci = i & 1 ? c[i / 2].y : c[i / 2].x, zi = i & 1 ? z[i / 2].y : z[i / 2].x;
          const float w = fmaf(v0, ci, -(v1 * zi));
          v1 = fmaf(v1, ci, v0 * zi);
          v0 = w;
        };
        if (p.interleaved) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            pair(i, x[2 * i], x[2 * i + 1]);
            pair(i + 4, y[2 * i], y[2 * i + 1]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) pair(i, x[i], y[i]);
        }
      }
      store8_any(p.out_dtype, p.out, to + (int64_t)(h + j * HL) * D + 8 * c0, x);
      store8_any(p.out_dtype, p.out, to + (int64_t)(h + j * HL) * D + 8 * c1, y);
    }
    h += N * HL;
    if (h >= h1) break;                                      // (lanes of the last heads alone may go on)
    load(h);
  }
}

// ---------------------------------------------------------------- k
// A value to 2^-44 of |own| + |other|: (own cos + sign other sin) factor, the angle as 64 bits round it.
__device__ __noinline__ Pair turned_pair(float own, float other, float sign, int pos, float freq, float factor) {
  const double a = (double)pos * (double)freq;
  const double k = rint(a * 0.63661977236758134308);   // 2 / pi
  const double r = fma(-k, 0x1.1a62633145c07p-54, fma(-k, 0x1.921fb54442d18p+0, a));
  const Pair x = {(float)r, (float)(r - (double)(float)r)};
  const int quarter = (int)((long long)k & 3);
  // the power series of both, in pairs up to x^9 and x^10
  const Pair y = mul(x, x);
  Pair s = {fmaf(fmaf(-1.f / 1307674368000.f, y.h, 1.f / 6227020800.f), y.h, -1.f / 39916800.f), 0.f};
  Pair c = {fmaf(fmaf(1.f / 20922789888000.f, y.h, -1.f / 87178291200.f), y.h, 1.f / 479001600.f), 0.f};
  const float sh[5] = {0x1.71de3ap-19f, -0x1.a01a02p-13f, 0x1.111112p-7f, -0x1.555556p-3f, 1.f};
  const float sl[5] = {0x1.55b1ccp-45f, 0x1.7f97fap-39f, -0x1.dddddep-32f, 0x1.555556p-28f, 0.f};
  const float ch[6] = {-0x1.27e4fcp-22f, 0x1.a01a02p-16f, -0x1.6c16c2p-10f, 0x1.555556p-5f, -0.5f, 1.f};
  const float cl[6] = {0x1.10ec14p-47f, -0x1.7f97fap-42f, 0x1.27d27ep-35f, -0x1.555556p-30f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 5; ++i) s = add(mul(s, y), {sh[i], sl[i]});
#pragma unroll
  for (int i = 0; i < 6; ++i) c = add(mul(c, y), {ch[i], cl[i]});
  s = mul(s, x);
  // the quarter turns
  Pair cs = quarter & 1 ? s : c, sn = quarter & 1 ? c : s;
  if (quarter == 1 || quarter == 2) cs = {-cs.h, -cs.l};
  if (quarter >= 2) sn = {-sn.h, -sn.l};
  const Pair v = add(mul({own, 0.f}, cs), mul({sign * other, 0.f}, sn));
  return factor == 1.f ? v : mul(v, {factor, 0.f});
}

// |a| against |b|
__device__ __forceinline__ bool larger(Pair a, Pair b) {
  const float la = a.h < 0.f ? -a.l : a.l, lb = b.h < 0.f ? -b.l : b.l;
  return fabsf(a.h) > fabsf(b.h) || (fabsf(a.h) == fabsf(b.h) && la > lb);
}
// The scale: the fp16 nearest to -1/8 of the fp32 nearest to x (rows of dq_kv_append are fp32 at most).
__device__ __forceinline__ __half scale_of(Pair x) { return __float2half_rn(x.h * -0.125f); }
__device__ __forceinline__ Pair within_fp16(Pair x) {
  return fabsf(x.h) > 65504.f || (fabsf(x.h) == 65504.f && (x.l < 0.f) == (x.h < 0.f)) ? Pair{copysignf(65504.f, x.h), 0.f} : x;
}

// The four lanes of a group hold eight values x each, known to `err`; `exact(e)` forms value e again.  Returns
// the word of codes and the scale.  Every lane of the warp calls it.
template <typename F>
__device__ __forceinline__ uint32_t k_word_known(const float (&x)[8], float err, int lane, __half& d, F exact) {
  float hi = max_of8(x), lo = min_of8(x);
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    err = fmaxf(err, __shfl_xor_sync(0xffffffffu, err, o));
  }
  const float top = fmaxf(hi, -lo);
  d = __float2half_rn((hi > -lo ? hi : lo) * -0.125f);
  // which sign the largest has, and which scale its eighth rounds to
  const __half2 around = __floats2half2_rn((top - err) * 0.125f, (top + err) * 0.125f);
  const bool unsure = fabsf(hi + lo) <= 2.f * err || top + err >= 65504.f ||
                      __half_as_ushort(__low2half(around)) != __half_as_ushort(__high2half(around));
  if (__any_sync(0xffffffffu, unsure)) {
    Pair best = {0.f, 0.f};
    if (unsure) {
#pragma unroll 1
      for (int e = 0; e < 8; ++e) {
        float xe = x[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) xe = e == i ? x[i] : xe;
        if (fabsf(xe) >= fminf(top, 65504.f) - 2.f * err) {       // (beyond fp16 all are equal)
          const Pair y = within_fp16(exact(e));
          if (larger(y, best)) best = y;
        }
      }
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      const Pair y = {__shfl_xor_sync(0xffffffffu, best.h, o), __shfl_xor_sync(0xffffffffu, best.l, o)};
      if (larger(y, best) || ((lane & o) != 0 && !larger(best, y))) best = y;
    }
    if (unsure) d = scale_of(best);
  }
  const float df = __half2float(d), inv = df == 0.f ? 0.f : __frcp_rn(df);
  // the quotient's own error: the reciprocal, the product and the sum
  // (taken in units of 15.5, where the saturating FMA clamps it; no value is below the largest's code 0)
  const float room = 0.5f - (err * fabsf(inv) + 3e-6f), scaled = inv * (1.f / 15.5f);
  uint32_t word = 0;
  float most = 0.f;                        // the distance from the middle of the code
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t unit = 1u << (4 * (e >> 1) + 16 * (e & 1));
    const float y = __saturatef(fmaf(x[e], scaled, 8.5f / 15.5f));
    const float t = __fmaf_rz(y, 15.5f, 8388608.f);
    most = fmaxf(most, fabsf(fmaf(y, 15.5f, 8388607.5f - t)));
    word += __float_as_uint(t) * unit;
  }
  word -= 0x4B000000u * 0x11111111u;
  if (__any_sync(0xffffffffu, most > room && df != 0.f)) {
#pragma unroll 1
    for (int e = 0; e < 8; ++e) {
      float xe = x[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) xe = e == i ? x[i] : xe;
      const float near = 0.5f - room, y = fmaf(xe, inv, 8.5f), k = rintf(y);
      if (df == 0.f || (near < 0.4f && (fabsf(y - k) >= near || k < 1.f || k > 15.f))) continue;
      const Pair v = exact(e);
      const float z = fmaf(v.h, inv, 8.5f), b = rintf(z);
      uint32_t code = (uint32_t)fminf(fmaxf(floorf(z), 0.f), 15.f);
      if (fabsf(z - b) < 2e-6f && b >= 1.f && b <= 15.f) {
        // against the border (b - 8.5) d, which is exact
        const float past = (v.h - (b - 8.5f) * df) + v.l;
        code = (uint32_t)b - ((df > 0.f ? past >= 0.f : past <= 0.f) ? 0u : 1u);
      }
      const int at = 4 * (e >> 1) + 16 * (e & 1);
      word = (word & ~(15u << at)) | code << at;
    }
  }
  return word;
}

// Eight values per thread, a group of 32 four lanes, as in dq_kv_append; the other halves of the pairs are
// loaded too (from L1: their own threads load them).
template <int D, int DT>
__device__ __forceinline__ void rope_k(const RopeParams& p, const Angles<D>& A, int t0, int n) {
  using B = KvBlk<D>;
  constexpr int C = D / 8, ROWS = kRopeThreads / C;
  const int lane = threadIdx.x & 31, c = threadIdx.x % C, g = c / 4, t4 = c & 3;
  const int rows = n * p.g.heads;
  const bool turns = 8 * c < 2 * p.half;
  const bool second = !p.interleaved && 8 * c >= p.half;      // of its pairs (half apart)
  const int i0 = p.interleaved ? 4 * c : second ? 8 * c - p.half : 8 * c;
  const int other = p.interleaved || !turns ? c : second ? c - p.half / 8 : c + p.half / 8;
  for (int r0 = 0; r0 < rows; r0 += ROWS) {
    const int r = r0 + (int)threadIdx.x / C;
    const bool in = r < rows;                                  // (the shuffles below take whole warps)
    int h;
    const int tt = row_of(in ? r : 0, p.g.heads, p.k_inv, h), t = t0 + tt;
    const int pos = A.pos[tt];
    const int64_t slot = in ? A.slot[tt] : -1;
    const int64_t at = (int64_t)t * p.k_stride + (int64_t)h * D;
    float raw[8], oth[8], x[8], err = 0.f;
    load8<DT>(p.k, at + 8 * c, raw);
    load8<DT>(p.k, at + 8 * other, oth);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = raw[e];
    if (turns && pos >= 0) {
      const float* cc = A.c + tt * p.half + i0;
      const float* ss = A.s + tt * p.half + i0;
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        float2 z, s;
        if (p.interleaved) {
          z = make_float2(cc[e >> 1], cc[e >> 1]);
          s = make_float2(-ss[e >> 1], ss[e >> 1]);
        } else {
          z = *(const float2*)(cc + e);
          s = *(const float2*)(ss + e);
          if (!second) s = make_float2(-s.x, -s.y);
        }
        const float2 b = p.interleaved ? make_float2(raw[e + 1], raw[e]) : make_float2(oth[e], oth[e + 1]);
        const float2 v = ffma2(make_float2(raw[e], raw[e + 1]), z, fmul2(b, s));
        x[e] = v.x;
        x[e + 1] = v.y;
        err = max_of3(err, fabsf(raw[e]) + fabsf(b.x), fabsf(raw[e + 1]) + fabsf(b.y));
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
      word = k_word_known(x, err, lane, d, [&](int e) -> Pair {
        float own = raw[0], b = p.interleaved ? raw[1] : oth[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) {
          own = e == i ? raw[i] : own;
          b = e == i ? (p.interleaved ? raw[i ^ 1] : oth[i]) : b;
        }
        if (!turns) return {own, 0.f};
        const bool minus = p.interleaved ? (e & 1) == 0 : !second;
        return turned_pair(own, b, minus ? -1.f : 1.f, pos, __ldg(p.freq + i0 + (p.interleaved ? e >> 1 : e)), p.factor);
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
__device__ __forceinline__ void rope_v(const RopeParams& p, const Angles<D>& A, int t0, int n) {
  using B = KvBlk<D>;
  constexpr int C = D / 8, ROWS = kRopeThreads / C;
  const int lane = threadIdx.x & 31, c = threadIdx.x % C, g = c / 4, t4 = c & 3;
  const int rows = n * p.g.heads;
  for (int r0 = 0; r0 < rows; r0 += ROWS) {
    const int r = r0 + (int)threadIdx.x / C;
    const bool in = r < rows;
    int h;
    const int tt = row_of(in ? r : 0, p.g.heads, p.k_inv, h), t = t0 + tt;
    const int64_t slot = in ? A.slot[tt] : -1;
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

// The angles of the CTA's tokens, their positions and slots.
template <int D>
__device__ __forceinline__ void find_angles(const RopeParams& p, Angles<D>& A, int t0, int n, bool turns) {
  if ((int)threadIdx.x < n) {
    const int pos = __ldg(p.pos + t0 + threadIdx.x);
    int64_t slot = pos >= 0 ? __ldg(p.slots + t0 + threadIdx.x) : -1;
    A.pos[threadIdx.x] = pos;
    A.slot[threadIdx.x] = slot < p.n_slots ? slot : -1;
  }
  if (turns) {
    // a thread keeps to one frequency
    const int at_once = kRopeThreads / p.half, t = (int)threadIdx.x / p.half, i = (int)threadIdx.x - t * p.half;
    const float freq = __ldg(p.freq + i);
    for (int tt = t; t < at_once && tt < n; tt += at_once) {
      const float2 z = turn(max(0, __ldg(p.pos + t0 + tt)), freq, p.factor);
      A.c[tt * p.half + i] = z.x;
      A.s[tt * p.half + i] = z.y;
    }
  }
  __syncthreads();
}

// blockIdx.x: K's CTAs of `tile` tokens, as many for V, and q's.
template <int D, int DT>
__global__ void __launch_bounds__(kRopeThreads, 4) kv_rope_kernel(const __grid_constant__ RopeParams p) {
  __shared__ __align__(16) Angles<D> A;
  pdl_wait();
  pdl_trigger();
  const int kv_ctas = (p.T + p.tile - 1) / p.tile, cta = (int)blockIdx.x;
  if (cta >= 2 * kv_ctas) {
    rope_q<D, DT>(p, (cta - 2 * kv_ctas) * (kRopeThreads / 32) + (int)threadIdx.x / 32);
    return;
  }
  const bool k = cta < kv_ctas;
  const int t0 = (k ? cta : cta - kv_ctas) * p.tile, n = min(p.tile, p.T - t0);
  find_angles<D>(p, A, t0, n, k);
  if (k) rope_k<D, DT>(p, A, t0, n);
  else rope_v<D, DT>(p, A, t0, n);
}

template <int D>
int launch_rope(RopeParams p, int dtype, cudaStream_t s) {
  constexpr int HL = 32 / (D / 16);
  // long calls spread an angle's price over more heads, short ones and rows of twice the bytes the work over more warps
  // (32 heads of 128 and 8: 4096 bf16 tokens 21.7 us with two turns, 20.9 with eight; 1023 7.7 and 8.1; 2047 fp32 tokens
  // 16.6, 16.4, 25.4 with one, two, eight, 1023 with 15 heads of 64 and 5 6.2, 7.4, 7.5)
  p.q_each = HL * (dtype == DQ_F32 ? 1 : p.T >= kLongCall ? 8 : 2);
  p.q_splits = (p.q_heads + p.q_each - 1) / p.q_each;
  const int64_t ctas = 2 * (((int64_t)p.T + p.tile - 1) / p.tile) +
                       ((int64_t)p.T * p.q_splits + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  if (ctas > 2147483647 || (int64_t)p.T * p.q_splits > 2147483647) return DQ_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)ctas), block(kRopeThreads);
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
  p.k_inv = (uint32_t)((1ULL << 32) / (uint32_t)p.g.heads) + 1;
  p.out = a->q_out;
  p.out_stride = a->out_stride;
  p.out_dtype = a->out_dtype;
  // about kTileCtas CTAs of K, of two tokens at least (64 tokens: 4.1 us with one, 4.1, 4.8, 6.7 with two, four, eight;
  // 1023: 11.2, 7.8, 7.4, 9.4; 4096: 39.9, 25.8, 22.3, 20.7)
  p.tile = 2;
  while (p.tile < kMostTile && p.tile * kTileCtas < a->T) p.tile *= 2;
  return by_dim(cache->head_dim,
                [&](auto d) { return launch_rope<decltype(d)::value>(p, a->dtype, (cudaStream_t)stream); });
}
