// kv_attn_stream.cu — attention of few query rows over the 4-bit paged cache:
// a decode step, or a handful of drafted tokens per request.
//
// Mathematics.  For one K/V head and up to 8 NT query rows (the query heads that
// share it, and the step's tokens) a warp walks tiles of 32 tokens and keeps
// the running maximum, sum and weighted V sum of the softmax.  Both products
// run on the tensor core with the tokens' codes as the A operand and the rows
// as the 8-wide B operand:
//   S^T[16 tokens x 8]  = K[16 x D] Q^T,   O^T[16 dims x 8] += V^T[16 x 16 tokens] P^T.
// * A code c masked out of its word is the fp16 subnormal c 2^-24 (low nibble of
//   each half) or c 2^-20 (second nibble): one AND per operand register, exact.
//   K: the rows' values are scaled by a power of two into fp16 (exact for the 16-bit
//   inputs but for values 2^-28 below the row's largest), those that meet the second
//   nibble by 2^-4 less; each 32-value group sums in its own accumulator, which starts
//   at -8 sum(q) (the codes' offset) and is scaled by the group's d in fp32.
//   V: d is a factor of the token, so it goes into the weights: per group
//   P' = fp16(p) * d (one HMUL2 for two tokens), and the offset is one more product, of
//   a constant -8 with P'.  O's even and odd values carry 2^-24 and 2^-20 to the end.
// * fp16 weights: p = 2^(s - M) with M = max - b, renewed only when a score passes
//   M + b + 4, so p <= 2^(b + 4).  b = 10 while every V scale is below 2 (p' < 2^15), and
//   -2 for good once one is not (p' <= 2^2 * 8188): no overflow, and weights down to
//   2^-24 of the largest keep at least one bit.  Rounding p and p' to fp16 (2^-11 each)
//   is the price of 16-bit operands; s, M, the sum of p and O stay fp32.
//
// Work.  All (request, K/V head, row tile, 32-token tile) units of the call in
// one line, cut into equal contiguous shares, one per warp: any mix of lengths
// fills the GPU, and no warp waits for another.  The host never sees a length:
// every CTA sums the requests' units itself.  A warp that holds a whole item
// writes its rows; otherwise it leaves a partial (at most two per warp), which
// kv_stream_join_kernel adds up in order, so that results do not depend on timing.
//
// Each warp has a ring of three tiles filled by its own bulk copies (a tile of a page
// is one contiguous run), two in flight while one is computed.
#include <algorithm>

#include "kv_attn.h"

namespace dqmoe {

namespace {

constexpr int kTile = 32;                 // tokens per unit
constexpr int kBlks = kTile / kKvBlk;
constexpr int kStages = 3;
constexpr int kMaxCtas = 160;

template <int D, int NT>
struct StreamCfg {
  // O (D NT / 4 registers), the offsets, Q and the scores: 16 warps of 128 registers, 12 of 168 or 8 of 255
  static constexpr int NW = D * NT <= 64 ? 16 : D * NT <= 128 ? 12 : 8;
  static constexpr int ROWS = 8 * NT;
  static constexpr int STG = kBlks * KvBlk<D>::BYTES;
  static constexpr int OFF_PRE = 1024;                              // int64 [513]
  static constexpr int OFF_RING = OFF_PRE + 4352;                   // (NTH + 1 + NTH / 32) * 8 at most
  static constexpr int SMEM = OFF_RING + NW * kStages * STG;
  static_assert(SMEM <= 232448, "shared memory");
};

// workspace: partial O [warps][2][ROWS][D] fp32, (M, l) [warps][2][ROWS], descriptors [warps]
struct StreamWs {
  float* o;
  float2* ml;
  int4* desc;
};
constexpr size_t kStreamO = (size_t)kMaxCtas * 16 * 2 * 8 * 128 * 4;   // NW * ROWS * D is the same for every D >= 128
constexpr size_t kStreamMl = (size_t)kMaxCtas * 16 * 2 * 16 * 8;
constexpr size_t kStreamDesc = (size_t)kMaxCtas * 16 * 16;

__device__ __forceinline__ StreamWs stream_ws(uint8_t* ws) {
  StreamWs w;
  w.o = (float*)ws;
  w.ml = (float2*)(ws + kStreamO);
  w.desc = (int4*)(ws + kStreamO + kStreamMl);
  return w;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// W consecutive words (2 or 4) from shared memory
template <int W>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t* v) {
  if (W == 4) {
    const uint4 x = lds_u128(addr);
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
  } else {
    const uint2 x = lds_u64(addr);
    v[0] = x.x; v[1] = x.y;
  }
}

template <int D, int NT>
__global__ void __launch_bounds__(StreamCfg<D, NT>::NW * 32, 1)
kv_stream_kernel(const __grid_constant__ AttnParams p) {
  using B = KvBlk<D>;
  using C = StreamCfg<D, NT>;
  constexpr int G = B::G, W = B::W, GH = G / W;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lr = lane >> 2, lt = lane & 3;
  uint64_t* bars = (uint64_t*)smem + warp * kStages;
  int64_t* pre = (int64_t*)(smem + C::OFF_PRE);
  uint8_t* ring = smem + C::OFF_RING + warp * kStages * C::STG;
  if (lane < kStages) mbar_init(&bars[lane], 1);
  fence_barrier_init();
  pdl_wait();
  pdl_trigger();

  constexpr int NTH = C::NW * 32;
  using Wk = Walk<C::ROWS, kTile>;
  Wk::template sum_units<NTH>(p, pre);
  const int64_t U = pre[NTH];
  // at least one unit per warp of the CTAs that take part
  const int ctas = (int)min((int64_t)gridDim.x, (U + C::NW - 1) / C::NW);
  const int gw = blockIdx.x * C::NW + warp;
  const StreamWs ws = stream_ws(p.ws);
  if (blockIdx.x >= ctas) {
    if (lane == 0) ws.desc[gw] = make_int4(0, 0, 0, 0);
    return;
  }
  const int64_t N = min((int64_t)ctas * C::NW, U);      // every one of the N shares holds a unit
  const int64_t u0 = U * gw / N, u1 = U * (gw + 1) / N;
  if (lane == 0) ws.desc[gw] = make_int4(0, 0, 0, 0);
  if (gw >= N) return;

  Item it;
  int64_t iu = Wk::template seek<NTH>(p, pre, u0, it);   // the unit at which the item starts

  // ---- producer state: the next unit to copy, its item, and 32 entries of its table row
  Item pi = it;
  int64_t pu = u0, piu = iu;
  int tbase = -1, tent = 0;
  const uint64_t pol = l2_evict_first_policy();
  const int tshift = p.g.page_shift;
  auto produce = [&](int stage) {
    if (pu >= u1) return;
    const int tile = pi.t0 + (int)(pu - piu);
    uint8_t* dst = ring + stage * C::STG;
    const int tok = tile * kTile;
    if (lane == 0) mbar_arrive_expect_tx(&bars[stage], C::STG);
    __syncwarp();
    int run = 0;
    while (run < kTile) {
      const int pg = (tok + run) >> tshift;
      if (tbase < 0 || pg < tbase || pg >= tbase + 32) {
        tbase = pg;
        const int e = pg + lane;
        tent = e < p.max_pages ? __ldg(p.table + (int64_t)pi.r * p.max_pages + e) : 0;
        if (tent < 0 || tent >= p.g.n_pages) tent = 0;
      }
      const int page = __shfl_sync(0xffffffffu, tent, pg - tbase);
      const int cnt = min(p.g.page_size, kTile - run);
      const int off = (tok + run) & (p.g.page_size - 1);
      if (lane == 0)
        bulk_g2s(dst + run / kKvBlk * B::BYTES,
                 p.g.pages + (int64_t)page * p.g.page_bytes + pi.h * p.g.head_bytes +
                     off / kKvBlk * B::BYTES,
                 cnt / kKvBlk * B::BYTES, &bars[stage], pol);
      run += cnt;
    }
    if (++pu == piu + pi.tiles && pu < u1) {
      piu += pi.tiles;
      Wk::next(p, pi);
      tbase = -1;
    }
  };
  __syncwarp();
#pragma unroll
  for (int s = 0; s < kStages; ++s) produce(s);

  // ---- consumer state
  uint32_t qf[G][4][NT];
  float qi[G][NT][2], cf[NT][2];
  float o[G][2][NT][4], ofs[G][NT][4];
  float M[NT][2], l[NT][2];
  float b = 10.f;
  bool ok = true;

  int64_t u = u0;
  int slot = 0;
  int stage = 0, phase = 0;
  while (u < u1) {
    // ---- rows of the item: column lr of each 8-row tile, values 8 lt.. of every group
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = it.row0 + nt * 8 + lr;
      const bool live = nt * 8 + lr < it.rows;
      const int tokq = row / p.group, uq = row - tokq * p.group;
      const uint16_t* src = (const uint16_t*)p.q + (int64_t)(it.first + tokq) * p.q_stride +
                            ((int64_t)it.h * p.group + uq) * D + 8 * lt;
      uint4 raw[G];
#pragma unroll
      for (int g = 0; g < G; ++g)
        raw[g] = live ? __ldg((const uint4*)(src + 32 * g)) : make_uint4(0, 0, 0, 0);
      float x[G][8], mx = 0.f;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const uint32_t w4[4] = {raw[g].x, raw[g].y, raw[g].z, raw[g].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (p.q_dtype == DQ_BF16) {
            x[g][2 * i] = __uint_as_float(w4[i] << 16);
            x[g][2 * i + 1] = __uint_as_float(w4[i] & 0xFFFF0000u);
          } else {
            const float2 f = __half22float2(u32_as_h2(w4[i]));
            x[g][2 * i] = f.x;
            x[g][2 * i + 1] = f.y;
          }
          mx = fmaxf(mx, fmaxf(fabsf(x[g][2 * i]), fabsf(x[g][2 * i + 1])));
        }
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      // 2^e with 2^14 <= max * 2^e < 2^15
      const int ex = (int)((__float_as_uint(mx) >> 23) & 255) - 127;
      const int e = mx > 0.f ? min(14 - ex, 100) : 0;
      const float up = __uint_as_float((uint32_t)(127 + e) << 23);
      const float c = p.scale * kLog2e * 16777216.f *
                      __uint_as_float((uint32_t)(127 - e) << 23);
      float sum[G];
#pragma unroll
      for (int g = 0; g < G; ++g) {
        sum[g] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float f = (i & 1) ? up * 0.0625f : up;
          const __half2 hv = __floats2half2_rn(x[g][2 * i] * f, x[g][2 * i + 1] * f);
          qf[g][i][nt] = h2_as_u32(hv);
          const float2 back = __half22float2(hv);
          sum[g] += (back.x + back.y) * ((i & 1) ? 16.f : 1.f);
        }
        sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 1);
        sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 2);
        const float s8 = sum[g] * (-8.f / 16777216.f);
        qi[g][nt][0] = __shfl_sync(0xffffffffu, s8, 8 * lt);
        qi[g][nt][1] = __shfl_sync(0xffffffffu, s8, 8 * lt + 4);
      }
      cf[nt][0] = __shfl_sync(0xffffffffu, c, 8 * lt);
      cf[nt][1] = __shfl_sync(0xffffffffu, c, 8 * lt + 4);
      M[nt][0] = M[nt][1] = kNone;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[g][0][nt][k] = o[g][1][nt][k] = ofs[g][nt][k] = 0.f;
    }
    b = 10.f;
    // the positions that every row of the item sees, and each column's own limits
    int lo_c[NT][2], hi_c[NT][2];
    int lo_all, hi_all;
    {
      const int lo_pos = it.len - it.qlen + it.row0 / p.group;
      const int hi_pos = it.len - it.qlen + (it.row0 + it.rows - 1) / p.group;
      hi_all = p.causal ? min(it.len, lo_pos + 1) : it.len;
      lo_all = p.window > 0 ? max(0, hi_pos - p.window + 1) : 0;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int pos = it.len - it.qlen + (it.row0 + nt * 8 + 2 * lt + k) / p.group;
          hi_c[nt][k] = p.causal ? min(it.len, pos + 1) : it.len;
          lo_c[nt][k] = p.window > 0 ? pos - p.window + 1 : 0;
        }
    }

    const int64_t ue = min(u1, iu + it.tiles);
    const bool from_start = u == iu, to_end = ue == iu + it.tiles;
    for (; u < ue; ++u) {
      const int tok0 = (it.t0 + (int)(u - iu)) * kTile;
      ok = ok && mbar_wait(&bars[stage], phase);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint32_t base = smem_u32(ring + stage * C::STG);
      const bool inner = tok0 >= lo_all && tok0 + kTile <= hi_all;

      // ---- scores
      float s[kBlks][NT][4];
#pragma unroll
      for (int k = 0; k < kBlks; ++k) {
        const uint32_t kb = base + k * B::BYTES;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[k][nt][i] = 0.f;
#pragma unroll
        for (int gh = 0; gh < GH; ++gh) {
          uint32_t wa[W], wb[W];
          lds_words<W>(kb + (((gh * 16 + lr) * 4 + lt) * W) * 4, wa);
          lds_words<W>(kb + (((gh * 16 + lr + 8) * 4 + lt) * W) * 4, wb);
          uint32_t da[W / 2], db[W / 2];
          if (W == 4) {
            const uint2 x = lds_u64(kb + B::OFF_KD + 2 * (lr * G + gh * W));
            const uint2 y = lds_u64(kb + B::OFF_KD + 2 * ((lr + 8) * G + gh * W));
            da[0] = x.x; da[W / 2 - 1] = x.y;
            db[0] = y.x; db[W / 2 - 1] = y.y;
          } else {
            da[0] = lds_u32(kb + B::OFF_KD + 2 * (lr * G));
            db[0] = lds_u32(kb + B::OFF_KD + 2 * ((lr + 8) * G));
          }
#pragma unroll
          for (int gw2 = 0; gw2 < W; ++gw2) {
            const int g = gh * W + gw2;
            const uint32_t x = wa[gw2], y = wb[gw2], x8 = x >> 8, y8 = y >> 8;
            const float2 fa = __half22float2(u32_as_h2(da[gw2 / 2])),
                         fb = __half22float2(u32_as_h2(db[gw2 / 2]));
            const float sa = (gw2 & 1) ? fa.y : fa.x, sb = (gw2 & 1) ? fb.y : fb.x;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float acc[4] = {qi[g][nt][0], qi[g][nt][1], qi[g][nt][0], qi[g][nt][1]};
              mma_16816_nv(acc, x & 0x000F000Fu, y & 0x000F000Fu, x & 0x00F000F0u, y & 0x00F000F0u,
                           qf[g][0][nt], qf[g][1][nt]);
              mma_16816_nv(acc, x8 & 0x000F000Fu, y8 & 0x000F000Fu, x8 & 0x00F000F0u,
                           y8 & 0x00F000F0u, qf[g][2][nt], qf[g][3][nt]);
              s[k][nt][0] = fmaf(sa, acc[0], s[k][nt][0]);
              s[k][nt][1] = fmaf(sa, acc[1], s[k][nt][1]);
              s[k][nt][2] = fmaf(sb, acc[2], s[k][nt][2]);
              s[k][nt][3] = fmaf(sb, acc[3], s[k][nt][3]);
            }
          }
        }
      }
      // ---- V scales (and their exponents' top bit)
      uint32_t dv[kBlks][G][2], big = 0;
#pragma unroll
      for (int k = 0; k < kBlks; ++k) {
        const uint32_t va = base + k * B::BYTES + B::OFF_VD + 8 * lt * G;
#pragma unroll
        for (int g = 0; g < G; g += 2) {
          const uint4 x = lds_u128(va + 8 * g);
          dv[k][g][0] = x.x; dv[k][g][1] = x.y;
          dv[k][g + 1][0] = x.z; dv[k][g + 1][1] = x.w;
        }
        if (!inner) {
          // tokens that no row sees may hold anything: their scales become 0
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int a = tok0 + k * 16 + 8 * j + 2 * lt;
            const uint32_t keep = ((a >= it.begin && a < it.end) ? 0x0000FFFFu : 0u) |
                                  ((a + 1 >= it.begin && a + 1 < it.end) ? 0xFFFF0000u : 0u);
#pragma unroll
            for (int g = 0; g < G; ++g) dv[k][g][j] &= keep;
          }
        }
#pragma unroll
        for (int g = 0; g < G; ++g) big |= dv[k][g][0] | dv[k][g][1];
      }
      // ---- weights
      float top[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float m = -INFINITY;
#pragma unroll
          for (int k = 0; k < kBlks; ++k)
#pragma unroll
            for (int hrow = 0; hrow < 2; ++hrow) {
              float v = s[k][nt][2 * hrow + i] * cf[nt][i];
              if (!inner) {
                const int a = tok0 + k * 16 + 8 * hrow + lr;
                v = a >= lo_c[nt][i] && a < hi_c[nt][i] ? v : -INFINITY;
              }
              s[k][nt][2 * hrow + i] = v;
              m = fmaxf(m, v);
            }
          top[nt][i] = m;
        }
      }
      const float lim = b + 4.f;
      bool over = b > 0.f && (big & 0x40004000u) != 0;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        over = over || top[nt][0] > M[nt][0] + lim || top[nt][1] > M[nt][1] + lim;
      if (__any_sync(0xffffffffu, over)) {
        const float bn = __any_sync(0xffffffffu, (big & 0x40004000u) != 0) ? -2.f : b;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float m = top[nt][i];
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
            const float mo = M[nt][i], mn = fmaxf(mo + (b - bn), m - bn), corr = ex2(mo - mn);
            M[nt][i] = mn;
            l[nt][i] *= corr;
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
              for (int k = i; k < 4; k += 2) {
                o[g][0][nt][k] *= corr;
                o[g][1][nt][k] *= corr;
                ofs[g][nt][k] *= corr;
              }
          }
        b = bn;
      }
      // ---- p and P V
#pragma unroll
      for (int k = 0; k < kBlks; ++k) {
        uint32_t pt[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int hrow = 0; hrow < 2; ++hrow) {
            const float p0 = ex2(s[k][nt][2 * hrow] - M[nt][0]);
            const float p1 = ex2(s[k][nt][2 * hrow + 1] - M[nt][1]);
            l[nt][0] += p0;
            l[nt][1] += p1;
            pt[nt][hrow] = transpose8x8(h2_as_u32(__floats2half2_rn(p0, p1)));
          }
        const uint32_t vb = base + k * B::BYTES + B::OFF_V;
#pragma unroll
        for (int gh = 0; gh < GH; ++gh) {
          uint32_t v0[W], v1[W];            // tokens 2t, 2t+1 and 2t+8, 2t+9: W / 2 words each
          lds_words<W>(vb + ((0 * GH + gh) * 32 + lane) * 4 * W, v0);
          lds_words<W>(vb + ((1 * GH + gh) * 32 + lane) * 4 * W, v1);
#pragma unroll
          for (int gw2 = 0; gw2 < W; ++gw2) {
            const int g = gh * W + gw2;
            const uint32_t sel = (gw2 & 1) ? 0x7632u : 0x5410u;
            const uint32_t z0 = __byte_perm(v0[gw2 / 2], v0[W / 2 + gw2 / 2], sel);
            const uint32_t z1 = __byte_perm(v1[gw2 / 2], v1[W / 2 + gw2 / 2], sel);
            const uint32_t y0 = z0 >> 8, y1 = z1 >> 8;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint32_t b0 = h2_as_u32(__hmul2(u32_as_h2(pt[nt][0]), u32_as_h2(dv[k][g][0])));
              const uint32_t b1 = h2_as_u32(__hmul2(u32_as_h2(pt[nt][1]), u32_as_h2(dv[k][g][1])));
              mma_16816_nv(o[g][0][nt], z0 & 0x000F000Fu, z0 & 0x00F000F0u, z1 & 0x000F000Fu,
                           z1 & 0x00F000F0u, b0, b1);
              mma_16816_nv(o[g][1][nt], y0 & 0x000F000Fu, y0 & 0x00F000F0u, y1 & 0x000F000Fu,
                           y1 & 0x00F000F0u, b0, b1);
              // the offset: -8 in each row's unit
              mma_16816_nv(ofs[g][nt], 0x80088008u, 0x80808080u, 0x80088008u, 0x80808080u, b0, b1);
            }
          }
        }
      }
      // every load of the stage has fed an instruction before its next copy is issued
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          keep_before_release<4>(o[g][0][nt]);
          keep_before_release<4>(o[g][1][nt]);
        }
      __syncwarp();
      produce(stage);
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
    if (!ok) break;

    // ---- the segment's rows: whole, or a partial
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float sum = l[nt][i];
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        const int col = nt * 8 + 2 * lt + i;
        if (col >= it.rows) continue;
        const bool whole = from_start && to_end;
        const float k24 = 16777216.f, k20 = 1048576.f;
        const float inv = whole ? (sum > 0.f ? 1.f / sum : 0.f) : 1.f;
        const int row = it.row0 + col, tokq = row / p.group, uq = row - tokq * p.group;
        const int64_t qrow = it.first + tokq;
        const int head = it.h * p.group + uq;
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const float x[4] = {(o[g][0][nt][i] + ofs[g][nt][i]) * (k24 * inv),
                              (o[g][0][nt][2 + i] + ofs[g][nt][2 + i]) * (k20 * inv),
                              (o[g][1][nt][i] + ofs[g][nt][i]) * (k24 * inv),
                              (o[g][1][nt][2 + i] + ofs[g][nt][2 + i]) * (k20 * inv)};
          if (whole)
            store_out4(p, qrow * p.out_stride + (int64_t)head * D + 32 * g + 4 * lr, x);
          else
            *(float4*)(ws.o + (((int64_t)gw * 2 + slot) * C::ROWS + col) * D + 32 * g + 4 * lr) =
                make_float4(x[0], x[1], x[2], x[3]);
        }
        if (lr == 0) {
          if (!whole)
            ws.ml[((int64_t)gw * 2 + slot) * C::ROWS + col] = make_float2(M[nt][i], sum);
          else if (p.lse)
            p.lse[qrow * p.n_q_heads + head] =
                sum > 0.f ? (M[nt][i] + log2f(sum)) * kLn2 : -INFINITY;
        }
      }
    if (from_start && !to_end && lane == 0) {
      // the item starts here and goes on in the next warps: how many of them
      const int64_t last = iu + it.tiles - 1;
      ws.desc[gw] = make_int4(it.r, it.h, it.row0, ((share_of(last, N, U) - gw) << 1) | slot);
    }
    if (!(from_start && to_end)) slot = 1;
    iu += it.tiles;
    if (u < u1) Wk::next(p, it);
  }
}

// Joins the partials of the items that go over several warps' shares.  CTA c
// looks after the items that start in CTA c of the kernel above; a warp takes a
// row of an item and one of SUB interleaved shares of its partials.
constexpr int kSub = 4;

template <int D, int NT>
__global__ void __launch_bounds__(1024) kv_stream_join_kernel(const __grid_constant__ AttnParams p) {
  using C = StreamCfg<D, NT>;
  constexpr int V = D / 32;                // values of a row per lane
  __shared__ float acc_s[8][kSub][D];
  __shared__ float2 ml_s[8][kSub];
  pdl_wait();
  pdl_trigger();
  const StreamWs ws = stream_ws(p.ws);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = warp >> 3, rw = warp & 7;
  for (int w = 0; w < C::NW; ++w) {
    const int gw = blockIdx.x * C::NW + w;
    const int4 d = __ldcg(ws.desc + gw);
    const int follow = d.w >> 1;
    if (follow == 0) continue;             // uniform for the CTA
    int first;
    const int n = q_rows(p, d.x, &first);
    const int rows = min(C::ROWS, n * p.group - d.z);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int col = nt * 8 + rw;
      const bool live = col < rows;
      // partial i: warp gw's slot (i = 0), then the first slot of the warps after it
      auto part = [&](int i) -> int64_t {
        return (((int64_t)(gw + i) * 2 + (i == 0 ? (d.w & 1) : 0)) * C::ROWS + col);
      };
      float m = kNone, l = 0.f, acc[V];
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] = 0.f;
      if (live) {
        for (int i = sub + kSub * lane; i <= follow; i += kSub * 32) m = fmaxf(m, __ldcg(ws.ml + part(i)).x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll 4
        for (int i = sub; i <= follow; i += kSub) {
          const int64_t at = part(i);
          const float2 ml = __ldcg(ws.ml + at);
          const float f = ex2(ml.x - m);
          l = fmaf(ml.y, f, l);
#pragma unroll
          for (int v = 0; v < V; v += 2) {
            const float2 x = __ldcg((const float2*)(ws.o + at * D + v * 32 + 2 * lane));
            acc[v] = fmaf(x.x, f, acc[v]);
            acc[v + 1] = fmaf(x.y, f, acc[v + 1]);
          }
        }
      }
#pragma unroll
      for (int v = 0; v < V; v += 2)
        *(float2*)&acc_s[rw][sub][v * 32 + 2 * lane] = make_float2(acc[v], acc[v + 1]);
      if (lane == 0) ml_s[rw][sub] = make_float2(m, l);
      __syncthreads();
      if (sub == 0 && live) {
        float mt = kNone;
        for (int k = 0; k < kSub; ++k) mt = fmaxf(mt, ml_s[rw][k].x);
        float f[kSub], lt = 0.f;
#pragma unroll
        for (int k = 0; k < kSub; ++k) {
          f[k] = ex2(ml_s[rw][k].x - mt);
          lt = fmaf(ml_s[rw][k].y, f[k], lt);
        }
        const float inv = lt > 0.f ? 1.f / lt : 0.f;
        const int row = d.z + col, tokq = row / p.group, uq = row - tokq * p.group;
        const int64_t qrow = first + tokq;
        const int head = d.y * p.group + uq;
        for (int c = lane; c < D / 4; c += 32) {
          float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < kSub; ++k) {
            const float4 a = *(const float4*)&acc_s[rw][k][4 * c];
            x[0] = fmaf(a.x, f[k], x[0]);
            x[1] = fmaf(a.y, f[k], x[1]);
            x[2] = fmaf(a.z, f[k], x[2]);
            x[3] = fmaf(a.w, f[k], x[3]);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) x[k] *= inv;
          store_out4(p, qrow * p.out_stride + (int64_t)head * D + 4 * c, x);
        }
        if (lane == 0 && p.lse)
          p.lse[qrow * p.n_q_heads + head] =
              lt > 0.f ? (mt + log2f(lt)) * kLn2 : -INFINITY;
      }
      __syncthreads();
    }
  }
}

template <int D, int NT>
int launch_stream(const AttnParams& p, int ctas, cudaStream_t s) {
  using C = StreamCfg<D, NT>;
  static bool attr[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DQ_ERR_CUDA;
  if (dev >= 64 || !attr[dev]) {
    if (cudaFuncSetAttribute(kv_stream_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::SMEM) != cudaSuccess)
      return DQ_ERR_CUDA;
    if (dev < 64) attr[dev] = true;
  }
  if (launch_pdl(kv_stream_kernel<D, NT>, dim3(ctas), dim3(C::NW * 32), C::SMEM, s, 0, p) !=
      cudaSuccess)
    return DQ_ERR_CUDA;
  if (launch_pdl(kv_stream_join_kernel<D, NT>, dim3(ctas), dim3(1024), 0, s, 0, p) != cudaSuccess)
    return DQ_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? DQ_OK : DQ_ERR_CUDA;
}

}  // namespace

size_t kv_stream_workspace() { return kStreamO + kStreamMl + kStreamDesc; }

int launch_kv_stream(const AttnParams& p, int head_dim, cudaStream_t s) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return DQ_ERR_CUDA;
  const int ctas = std::min(sms, kMaxCtas);
  // more than 8 rows per K/V head: 16 at a time where the registers allow it
  const bool two = std::min<int64_t>((int64_t)p.max_q_len * p.group, p.rows_upto) > 8;
  if (head_dim == 64) return two ? launch_stream<64, 2>(p, ctas, s) : launch_stream<64, 1>(p, ctas, s);
  if (head_dim == 128)
    return two ? launch_stream<128, 2>(p, ctas, s) : launch_stream<128, 1>(p, ctas, s);
  return launch_stream<256, 1>(p, ctas, s);
}

}  // namespace dqmoe
