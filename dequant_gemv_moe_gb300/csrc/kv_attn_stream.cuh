// kv_attn_stream.cuh — attention of few query rows over the 4-bit paged cache:
// a decode step, or a handful of drafted tokens per request.
//
// Mathematics.  For one K/V head and up to 8 query rows (the query heads that
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
//   P' = fp16(p) * d (one HMUL2 for two tokens).  The codes lose their offset before the product (one
//   more addition per register: taking 8 sum(p') off the sums instead left 1e-7 of the largest scale in
//   values whose own scales are small).  O's even and odd values carry 2^-24 and 2^-20 to the end.
// * fp16 weights: p = 2^(s - M) with M = max - 10, renewed only when a score passes
//   M + 14, so p <= 2^14 and weights down to 2^-34 of the largest keep at least one bit.
//   A group whose V scales reach 2 is taken in units of a power of two that brings them below
//   it (p' < 2^15: no overflow), each group in its own, so that a group of small scales loses
//   nothing beside a large one.  Rounding p and p' to fp16 (2^-11 each) is the price of
//   16-bit operands; s, M, the sum of p and O stay fp32.
//
// Work.  All (request, K/V head, row tile, 32-token tile) units of the call in
// one line, cut into equal contiguous shares, one per warp: any mix of lengths
// fills the GPU, and no warp waits for another.  The host never sees a length:
// every CTA sums the requests' units itself.  A warp that holds a whole item
// writes its rows; otherwise it leaves a partial (at most two per warp) in shared
// memory, and the CTA's warps join them in order when all have ended.  What goes on
// in another CTA (again at most two partials) is left to kv_stream_join_kernel.  The
// order of every sum is fixed, so results do not depend on timing.
//
// What bounds it: next to HBM the decoding of a tile, a chain of loads, products and exponentials that three
// warps a scheduler do not hide (issue in 57 % of the cycles, ALU pipe 51 %): a warp's tile of 32 tokens
// and 8 rows takes 1.3 us with heads of 128 when 12 warps share an SM, which is 6.4 TB/s at most.  64
// requests of up to 16384 tokens, 8 K/V heads of 128, 576 MB: 106 us, 5.4 TB/s, 80 % of what a copy
// reaches; 3 requests of up to 131072 tokens 81 %; the 64 requests with heads of 256 200 us, 84 %, with heads
// of 64, whose tile has half the bytes for the same fixed work, 79 us, 53 %.  Rows above 8 decode the
// page again: 20 requests of up to 42 rows 38 us for 36 MB.
//
// Each warp has a ring of tiles filled by its own bulk copies (a tile of a page
// is one contiguous run), all but one in flight while one is computed.
// Modes other than kPlain: prefixes and first positions, capped scores, a distance bias (dq_kv_scores), an instance each.
// Scores that are changed are taken into units of log 2 first; everything else is the same.  64 requests of up to 16384
// tokens (642 MB) capped at 50: 133 us, 117 without the cap; 20 requests of up to 42 rows with a bias 40.
#pragma once

#include <algorithm>
#include <type_traits>

#include "kv_attn.h"

namespace dqmoe {

namespace {

constexpr int kTile = 32;                 // tokens per unit
constexpr int kBlks = kTile / kKvBlk;
constexpr int kMaxCtas = 160;
// Where the row tiles fit the GPU a CTA each, they may be left whole: no walk to find the shares and no
// second launch, which take 4 to 5 us, but a warp has more tiles, at 1.2 us each (heads of 64), 1.3 (128) or
// 1.8 (256).  Where that would be more than 3 tiles, a row tile takes a cluster of 2 or 4 CTAs, whose
// first one joins what the others leave (2 to 3 us, its launch included).  Whole if a warp has at most
// kAloneTiles (half as many in a cluster) more than equal shares would give it.  Whole and in shares, us:
//   heads of 128, 8 row tiles: 977 tokens 9.2, 11.0; 4000 tokens in fours 12.0, 12.0; 16000 tokens 23.0, 14.5
//   64 row tiles: 1900 tokens in twos 11.8, 13.3; 4000 tokens 15.3, 15.4; 8000 tokens 22.3, 19.2
//   128 row tiles: 977 tokens 9.6, 13.3; 2500 tokens 14.8, 16.6; 4000 tokens 20.1, 20.0
//   heads of 256, 64 row tiles: a window of 256 tokens 9.4, 12.1; of 1024, in twos 13.2, 14.2
//   heads of 64, 8 row tiles: 4000 tokens in twos 9.9, 11.1; 12000 tokens in fours 14.1, 12.7
template <int D>
constexpr int kAloneTiles = D == 256 ? 2 : 4;
constexpr int kAloneMost = 10;             // and this many in all
constexpr int kClusterCtas = 128;          // (not every SM is in reach of a whole cluster)

// what a warp did not finish
struct Left {
  int r, h, row0, rows;
  int has, open;                          // open: the item goes on behind this share
  int64_t last;                           // the unit of its last tile
};

// Where a warp is in its share, kept in shared memory: the tile loop needs its registers.  [0] is the
// item that is computed, [1] the one that is copied; lo, hi: the positions that each row sees.
struct Place {
  Item it;
  int64_t iu;
  int a, b;
};
struct WarpState {
  Place at[2];
  int64_t u0, u1;
  int lo[8], hi[8];
  int pos[8];                             // EXT: the rows' positions, and the slopes of their bias
  float slope[8];
};

template <int D>
struct StreamCfg {
  // O (D / 4 registers), Q, its sums and the scores: 16 warps of 128 registers, 12 of 168 or 8 of 255.
  // (64 requests, 576 MB, heads of 128: 12 warps with three tiles each 107.3 us, 16 with two 112.3.)
  static constexpr int NW = D <= 64 ? 16 : D <= 128 ? 12 : 8;
  static constexpr int ROWS = 8;
  static constexpr int STG = kBlks * KvBlk<D>::BYTES;
  static constexpr int STAGES = D == 256 ? 2 : 3;
  static constexpr int NTH = NW * 32;
  static constexpr int PART = ROWS * D * 4 + ROWS * 8;              // rows of O, then (M, l)
  static constexpr int OFF_LEFT = 512;                              // Left [NW][2]
  static constexpr int OFF_PRE = 1792;                              // int64 [NTH + 1 + NW]
  static constexpr int OFF_KNOWN = OFF_PRE + (NTH + 1 + NW) * 8;   // int [4 NTH]
  static constexpr int OFF_STATE = (OFF_KNOWN + NTH * 16 + 15) / 16 * 16;
  static constexpr int OFF_RING = (OFF_STATE + NW * (int)sizeof(WarpState) + 127) / 128 * 128;
  static constexpr int OFF_HEAD = OFF_RING + NW * STAGES * STG;     // the warps' first partials
  static constexpr int SMEM = OFF_HEAD + NW * PART;                 // (the second ones lie in the rings)
  static_assert(NW <= 16 && SMEM <= 232448 && STAGES * STG >= PART &&
                    NW * STAGES * 8 <= OFF_LEFT && NW * 2 * sizeof(Left) <= OFF_PRE - OFF_LEFT, "shared memory");
};

// workspace: partial O [ctas][2][ROWS][D] fp32, (M, l) [ctas][2][ROWS], descriptors [ctas]
struct StreamWs {
  float* o;
  float2* ml;
  int4* desc;
};
constexpr size_t kStreamO = (size_t)kMaxCtas * 2 * 8 * 256 * 4;     // ROWS * D is at most 8 * 256
constexpr size_t kStreamMl = (size_t)kMaxCtas * 2 * 8 * 8;
constexpr size_t kStreamDesc = (size_t)kMaxCtas * 16;

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

// Nibble n (0 or 1) of each half less 8, as fp16 subnormals in units of 2^-24 or 2^-20.
__device__ __forceinline__ uint32_t less8(uint32_t w, int n) {
  return n == 0 ? h2_as_u32(__hadd2(u32_as_h2(w & 0x000F000Fu), u32_as_h2(0x80088008u)))
                : h2_as_u32(__hadd2(u32_as_h2(w & 0x00F000F0u), u32_as_h2(0x80808080u)));
}

// D = A B + C with C the same for both rows of a lane
__device__ __forceinline__ void mma_16816_c(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1, float c0, float c1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%11,%10,%11};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}

template <int D, int MODE>
__global__ void __launch_bounds__(StreamCfg<D>::NTH, 1)
kv_stream_kernel(const __grid_constant__ AttnParams p) {
  constexpr bool EXT = MODE != kPlain, CAPS = MODE == kCaps || MODE == kAnyScores, BIAS = MODE == kBias || MODE == kAnyScores;
  using B = KvBlk<D>;
  using C = StreamCfg<D>;
  constexpr int G = B::G, W = B::W, GH = G / W;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lr = lane >> 2, lt = lane & 3;
  uint64_t* bars = (uint64_t*)smem + warp * C::STAGES;
  Left* left = (Left*)(smem + C::OFF_LEFT);
  int64_t* pre = (int64_t*)(smem + C::OFF_PRE);
  uint8_t* ring = smem + C::OFF_RING + warp * C::STAGES * C::STG;
  if (lane < C::STAGES) mbar_init(&bars[lane], 1);
  if (lane < 2) left[warp * 2 + lane].has = 0;
  fence_barrier_init();
  pdl_wait();
  pdl_trigger();

  using Wk = StreamWalkOf<EXT>;
  static_assert(C::ROWS == 8 && kTile == 32, "as StreamWalk has them");
  int* known = (int*)(smem + C::OFF_KNOWN);
  const StreamWs ws = stream_ws(p.ws);
  int64_t U;
  int w0 = blockIdx.x * C::NW, N;          // the CTA's first share of N
  Place x;
  if (p.alone) {
    const int cl = (int)cluster_nctarank();             // CTAs of the row tile
    if (!Wk::nth(p, blockIdx.x / cl, p.alone, x.it)) return;
    U = Wk::cost(p, x.it);
    N = (int)min((int64_t)cl * C::NW, U);
    w0 = (int)cluster_ctarank() * C::NW;
  } else {
    Wk::template sum_units<C::NTH>(p, pre, known);
    U = pre[C::NTH];
    // at least one unit per warp of the CTAs that take part
    const int ctas = (int)min((int64_t)gridDim.x, (U + C::NW - 1) / C::NW);
    if (threadIdx.x == 0) ws.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
    if (blockIdx.x >= ctas) return;
    N = (int)min((int64_t)ctas * C::NW, U);             // every one of the N shares holds a unit
  }
  const int gw = w0 + warp;
  const int64_t u0 = share_start(U, N, min(gw, N)), u1 = share_start(U, N, min(gw + 1, N));

  // ---- the first item of the share, and its tiles [a, b) that lie in it
  WarpState& S = ((WarpState*)(smem + C::OFF_STATE))[warp];
  bool more = u0 < u1;
  if (more) {
    x.iu = p.alone ? 0 : Wk::template seek<C::NTH>(p, pre, u0, x.it, known);
    more = Wk::here(p, x.it, x.iu, u0, u1, x.a, x.b);
    if (lane == 0) {
      S.at[0] = S.at[1] = x;
      S.u0 = u0;
      S.u1 = u1;
    }
  }
  __syncwarp();
  // on to the next item of the share; every lane computes it
  auto advance = [&](Place& at) {
    Place x = at;
    const bool m = Wk::after(p, x.it, x.iu, S.u0, S.u1, x.a, x.b);
    __syncwarp();
    if (lane == 0) at = x;
    __syncwarp();
    return m;
  };

  // ---- the next tile to copy.  A tile is one contiguous run of a page,
  // or two of 16-token pages; each lane holds the address of one of the next 32 runs and issues its
  // copy, so that page numbers are looked up once in 32 runs.
  int pt = more ? S.at[1].a : 0, ptb = more ? S.at[1].b : 0;
  bool pmore = more;
  const uint64_t pol = l2_evict_first_policy();
  const int runs = p.g.page_size < kTile ? kTile / kKvBlk : 1;      // page_size is 16 or at least kTile
  const uint32_t run_bytes = C::STG / runs;
  int used = 32;                           // runs of the 32 that were issued
  const uint8_t* src = nullptr;
  auto produce = [&](int stage) {
    if (!pmore) return;
    if (used == 32) {
      used = 0;
      const Item& x = S.at[1].it;
      const int ahead = lane * (kTile / runs);
      const int pg = listed_page(p, x.t0 + pt, kTile, ahead);
      int page = pg >= 0 ? __ldg(p.table + (int64_t)x.r * p.max_pages + pg) : 0;
      if (page < 0 || page >= p.g.n_pages) page = 0;
      const uint32_t in_page = ((uint32_t)(x.t0 + pt) * kTile + ahead) & (p.g.page_size - 1);
      src = p.g.pages + (int64_t)page * p.g.page_bytes + x.h * p.g.head_bytes + in_page / kKvBlk * B::BYTES;
    }
    if (lane == 0) mbar_arrive_expect_tx(&bars[stage], C::STG);
    __syncwarp();
    const uint32_t mine = lane - used;
    if (mine < runs) bulk_g2s(ring + stage * C::STG + mine * run_bytes, src, run_bytes, &bars[stage], pol);
    used += runs;
    if (++pt == ptb) {
      pmore = advance(S.at[1]);
      pt = S.at[1].a;
      ptb = S.at[1].b;
      used = 32;
    }
  };
  // The rows of item x: column lr of each 8-row tile, values 8 lt.. of every group.  Loaded before the
  // copies are issued, or before the item in front is written, and used after.
  uint4 raw[G];
  auto load_rows = [&](const Item& x) {
    const int row = x.row0 + lr;
    const bool live = lr < x.rows;
    const int tokq = row_token(p, row), uq = row - tokq * p.group;
    const uint16_t* q = (const uint16_t*)p.q + (int64_t)(x.first + tokq) * p.q_stride +
                        ((int64_t)x.h * p.group + uq) * D + 8 * lt;
#pragma unroll
    for (int g = 0; g < G; ++g)
      raw[g] = live ? __ldg((const uint4*)(q + 32 * g)) : make_uint4(0, 0, 0, 0);
  };
  if (more) load_rows(S.at[0].it);
  __syncwarp();
#pragma unroll
  for (int s = 0; s < C::STAGES; ++s) produce(s);

  // ---- consumer state
  uint32_t qf[G][4];
  float qi[G][2], cf[2];
  float o[G][2][4];
  float M[2], lim[2];
  float2 l;
  uint32_t unit = 0;                       // four bits a group: V is taken in units of 2^unit
  bool ok = true;

  int stage = 0, phase = 0;
  while (more) {
    const Item it = S.at[0].it;
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
    const float c = fmaxf(p.scale * kLog2e * 16777216.f * __uint_as_float((uint32_t)(127 - e) << 23),
                          kLeastScale) * (CAPS ? p.cap_inv : 1.f);
    float sum[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      sum[g] = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float f = (i & 1) ? up * 0.0625f : up;
        const __half2 hv = __floats2half2_rn(x[g][2 * i] * f, x[g][2 * i + 1] * f);
        qf[g][i] = h2_as_u32(hv);
        const float2 back = __half22float2(hv);
        sum[g] += (back.x + back.y) * ((i & 1) ? 16.f : 1.f);
      }
      sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 1);
      sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 2);
      const float s8 = sum[g] * (-8.f / 16777216.f);
      qi[g][0] = __shfl_sync(0xffffffffu, s8, 8 * lt);
      qi[g][1] = __shfl_sync(0xffffffffu, s8, 8 * lt + 4);
    }
    cf[0] = __shfl_sync(0xffffffffu, c, 8 * lt);
    cf[1] = __shfl_sync(0xffffffffu, c, 8 * lt + 4);
    M[0] = M[1] = kNone;
    lim[0] = lim[1] = kNone;
    l = make_float2(0.f, 0.f);
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[g][0][k] = o[g][1][k] = 0.f;
    unit = 0;
    // the positions that every row of the item sees, and each row's own limits
    int lo_all, hi_all;
    {
      const int lo_pos = it.shift + row_token(p, it.row0);
      const int hi_pos = it.shift + row_token(p, it.row0 + it.rows - 1);
      const int prefix = EXT ? it.prefix : 0;
      hi_all = seen_end(p, it.len, lo_pos, prefix);
      lo_all = first_seen(p, hi_pos);
      if (lane < C::ROWS) {
        const int row = EXT ? min(it.row0 + lane, it.row0 + it.rows - 1) : it.row0 + lane;
        const int tokq = row_token(p, row), pos = it.shift + tokq;
        S.hi[lane] = seen_end(p, it.len, pos, prefix);
        S.lo[lane] = first_seen(p, pos);
        if (EXT) {
          const int lo = max(S.lo[lane], row_first(p, it.first + tokq));
          S.lo[lane] = lo;
          lo_all = max(lo_all, lo);
          S.pos[lane] = pos;
          S.slope[lane] = BIAS && p.slopes ? __ldg(p.slopes + it.h * p.group + row - tokq * p.group) * kLog2e : 0.f;
        }
      }
      if (EXT) lo_all = __reduce_max_sync(0xffffffffu, lo_all);
      __syncwarp();
    }

    // The item's tiles.  UNITS false: every group's unit is 1, and true comes back at the first tile that needs
    // another one (its copy is still there).  An instance of its own, so that caches without such scales
    // do not pay: one loop for both took 111.4 us for 64 requests, this 106.8 (where every tile has such
    // scales, 122).
    const int tb = S.at[0].b;
    int tl = S.at[0].a;
    auto tiles = [&](auto units_c) -> bool {
      constexpr bool UNITS = decltype(units_c)::value;
      for (; tl < tb; ++tl) {
        const int tok0 = (it.t0 + tl) * kTile;
        ok = ok && mbar_wait(&bars[stage], phase);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return false;
        const uint32_t base = smem_u32(ring + stage * C::STG);
        const bool inner = tok0 >= lo_all && tok0 <= hi_all - kTile;

        // ---- scores
        float s[kBlks][4];
#pragma unroll
        for (int k = 0; k < kBlks; ++k) {
          const uint32_t kb = base + k * B::BYTES;
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
              float acc[4];
              mma_16816_c(acc, x & 0x000F000Fu, y & 0x000F000Fu, x & 0x00F000F0u, y & 0x00F000F0u,
                          qf[g][0], qf[g][1], qi[g][0], qi[g][1]);
              mma_16816_nv(acc, x8 & 0x000F000Fu, y8 & 0x000F000Fu, x8 & 0x00F000F0u,
                           y8 & 0x00F000F0u, qf[g][2], qf[g][3]);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                s[k][i] = g == 0 ? (i < 2 ? sa : sb) * acc[i] : fmaf(i < 2 ? sa : sb, acc[i], s[k][i]);
            }
          }
        }
        if (CAPS || BIAS) {
          float2 u[4];                                    // in units of log 2, or of the cap
#pragma unroll
          for (int i = 0; i < 4; ++i)
            u[i] = fmul2(make_float2(s[i >> 1][2 * (i & 1)], s[i >> 1][2 * (i & 1) + 1]), make_float2(cf[0], cf[1]));
          if (CAPS && p.cap > 0.f) {
            float far = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) far = fmaxf(far, fmaxf(fabsf(u[i].x), fabsf(u[i].y)));
            if (__any_sync(0xffffffffu, far > 1.f)) soft_cap_far(p, u);
            else soft_cap(p, u);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s[i >> 1][2 * (i & 1)] = u[i].x;
            s[i >> 1][2 * (i & 1) + 1] = u[i].y;
          }
          if (BIAS && p.slopes) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float d = (float)(S.pos[2 * lt + i] - tok0 - lr), slope = -S.slope[2 * lt + i];
#pragma unroll
              for (int k = 0; k < kBlks; ++k)
#pragma unroll
                for (int hrow = 0; hrow < 2; ++hrow)
                  s[k][2 * hrow + i] = fmaf(fabsf(d - (float)(k * 16 + 8 * hrow)), slope, s[k][2 * hrow + i]);
            }
          }
        }
        // tokens 2t + 8j of block k, and the one behind: those that no row sees may hold anything, their V scales
        // become 0
        uint32_t seen = 0;
        if (EXT && !inner) seen = __ballot_sync(0xffffffffu, token_seen<EXT>(p, S.at[0].it, tok0 + lane));
        auto kept = [&](int k, int j) -> uint32_t {
          const int a = tok0 + k * 16 + 8 * j + 2 * lt;
          if (EXT) return (seen >> (a - tok0) & 1 ? 0x0000FFFFu : 0u) | (seen >> (a + 1 - tok0) & 1 ? 0xFFFF0000u : 0u);
          const int from = S.at[0].it.begin, to = S.at[0].it.end;
          return ((a >= from && a < to) ? 0x0000FFFFu : 0u) | ((a + 1 >= from && a + 1 < to) ? 0xFFFF0000u : 0u);
        };
        // the V scales of block k and group g for this lane's tokens, pairs (2t, 2t + 1) and (2t + 8, 2t + 9)
        auto v_scales = [&](int k, int g) -> uint2 {
          uint2 x = lds_u64(base + k * B::BYTES + B::OFF_VD + 8 * (lt * G + g));
          if (!inner) {
            x.x &= kept(k, 0);
            x.y &= kept(k, 1);
          }
          return x;
        };
        // Some bit of `kBig` is set in `big` if some V scale is 2 units of its group or more: bit 14 where every
        // unit is 1, else the carry into bit 15 of the magnitude and 2^15 less that limit.
        constexpr uint32_t kBig = UNITS ? 0x80008000u : 0x40004000u;
        auto carry = [&](uint32_t x, int g) -> uint32_t {
          return UNITS ? (x & 0x7FFF7FFFu) + (0x8000u - ((16 + (unit >> 4 * g & 15)) << 10)) * 0x10001u : x;
        };
        uint32_t big = 0;
        if (inner) {
          // the tile's scales once over the lanes
          const uint32_t va = base + (lane >> 4) * B::BYTES + B::OFF_VD + (lane & 15) * (D / 16);
          if (D == 64) {
            big = carry(lds_u32(va), lane >> 1 & 1);
          } else if (D == 128) {
            const uint2 x = lds_u64(va);
            big = carry(x.x, lane & 3) | carry(x.y, lane & 3);
          } else {
            const uint4 x = lds_u128(va);
            big = carry(x.x, 2 * (lane & 3)) | carry(x.y, 2 * (lane & 3)) | carry(x.z, 2 * (lane & 3) + 1) |
                  carry(x.w, 2 * (lane & 3) + 1);
          }
        } else {
#pragma unroll
          for (int k = 0; k < kBlks; ++k)
#pragma unroll
            for (int g = 0; g < G; ++g) {
              const uint2 x = v_scales(k, g);
              big |= carry(x.x, g) | carry(x.y, g);
            }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int lo = S.lo[2 * lt + i], hi = S.hi[2 * lt + i];
#pragma unroll
            for (int k = 0; k < kBlks; ++k)
#pragma unroll
              for (int hrow = 0; hrow < 2; ++hrow) {
                const int a = tok0 + k * 16 + 8 * hrow + lr;
                if (a < lo || a >= hi) s[k][2 * hrow + i] = -INFINITY;
              }
          }
        }
        // ---- weights
        float top[2];
        bool over = (big & kBig) != 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          top[i] = fmaxf(fmaxf(s[0][i], s[0][2 + i]), fmaxf(s[1][i], s[1][2 + i])) * (CAPS || BIAS ? 1.f : cf[i]);
          over = over || top[i] > lim[i];
        }
        if (__any_sync(0xffffffffu, over)) {
          if (__any_sync(0xffffffffu, (big & kBig) != 0)) {
            if (!UNITS) return true;
#pragma unroll
            for (int g = 0; g < G; ++g) {
              uint32_t m = 0;
#pragma unroll
              for (int k = 0; k < kBlks; ++k) {
                const uint2 x = v_scales(k, g);
                m = max(max(m, max(x.x & 0x7FFFu, x.x >> 16 & 0x7FFFu)), max(x.y & 0x7FFFu, x.y >> 16 & 0x7FFFu));
              }
              // the exponent of the group's largest scale above that of 1 (12 at most: 8188)
              const int had = unit >> 4 * g & 15;
              const int add = min((int)(__reduce_max_sync(0xffffffffu, m) >> 10) - 15, 14) - had;
              if (add > 0) {
                unit += (uint32_t)add << 4 * g;
                const float f = __uint_as_float((uint32_t)(127 - add) << 23);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  o[g][0][k] *= f;
                  o[g][1][k] *= f;
                }
              }
            }
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float m = top[i];
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
            const float mo = M[i], mn = fmaxf(mo, m - 10.f), corr = ex2(mo - mn);
            M[i] = mn;
            lim[i] = mn + 14.f;
            (i == 0 ? l.x : l.y) *= corr;
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
              for (int k = i; k < 4; k += 2) {
                o[g][0][k] *= corr;
                o[g][1][k] *= corr;
              }
          }
        }
        // ---- p and P V
#pragma unroll
        for (int k = 0; k < kBlks; ++k) {
          uint32_t pt[2];
#pragma unroll
          for (int hrow = 0; hrow < 2; ++hrow) {
            const float2 w = make_float2(ex2(CAPS || BIAS ? s[k][2 * hrow] - M[0] : fmaf(s[k][2 * hrow], cf[0], -M[0])),
                                         ex2(CAPS || BIAS ? s[k][2 * hrow + 1] - M[1] : fmaf(s[k][2 * hrow + 1], cf[1], -M[1])));
            l = fadd2(l, w);
            pt[hrow] = transpose8x8(h2_as_u32(__floats2half2_rn(w.x, w.y)));
          }
          uint32_t dv[G][2];
#pragma unroll
          for (int g = 0; g < G; g += 2) {
            const uint4 x = lds_u128(base + k * B::BYTES + B::OFF_VD + 8 * (lt * G + g));
            dv[g][0] = x.x; dv[g][1] = x.y;
            dv[g + 1][0] = x.z; dv[g + 1][1] = x.w;
          }
          if (!inner) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t keep = kept(k, j);
#pragma unroll
              for (int g = 0; g < G; ++g) dv[g][j] &= keep;
            }
          }
          if (UNITS) {
#pragma unroll
            for (int g = 0; g < G; ++g) {
              const uint32_t f = (15 - (unit >> 4 * g & 15)) * 0x04000400u;    // 2^-unit, twice
#pragma unroll
              for (int j = 0; j < 2; ++j) dv[g][j] = h2_as_u32(__hmul2(u32_as_h2(dv[g][j]), u32_as_h2(f)));
            }
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
              const uint32_t b0 = h2_as_u32(__hmul2(u32_as_h2(pt[0]), u32_as_h2(dv[g][0])));
              const uint32_t b1 = h2_as_u32(__hmul2(u32_as_h2(pt[1]), u32_as_h2(dv[g][1])));
              mma_16816_nv(o[g][0], less8(z0, 0), less8(z0, 1), less8(z1, 0), less8(z1, 1), b0, b1);
              mma_16816_nv(o[g][1], less8(y0, 0), less8(y0, 1), less8(y1, 0), less8(y1, 1), b0, b1);
            }
          }
        }
        // every load of the stage has fed an instruction before its next copy is issued
#pragma unroll
        for (int g = 0; g < G; ++g) {
          keep_before_release<4>(o[g][0]);
          keep_before_release<4>(o[g][1]);
        }
        __syncwarp();
        produce(stage);
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
      return false;
    };
    if (tiles(std::false_type())) tiles(std::true_type());
    if (!ok) break;

    // ---- the item's rows: whole, or a partial (the second one over the ring, whose copies have all
    // been used: the share ends here)
    const Item done = S.at[0].it;
    const int64_t done_last = Wk::last_unit(p, done, S.at[0].iu);
    const bool from_start = S.at[0].a == 0, to_end = S.at[0].b == done.tiles;
    const bool whole = from_start && to_end;
    float* part = (float*)(from_start ? ring : smem + C::OFF_HEAD + warp * C::PART);
    more = advance(S.at[0]);
    if (more) load_rows(S.at[0].it);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float sum = i == 0 ? l.x : l.y;
      sum += __shfl_xor_sync(0xffffffffu, sum, 4);
      sum += __shfl_xor_sync(0xffffffffu, sum, 8);
      sum += __shfl_xor_sync(0xffffffffu, sum, 16);
      const int col = 2 * lt + i;
      if (col >= done.rows) continue;
      const float k24 = 16777216.f, k20 = 1048576.f;
      const float inv = whole ? (sum > 0.f ? 1.f / sum : 0.f) : 1.f;
      const int row = done.row0 + col, tokq = row_token(p, row), uq = row - tokq * p.group;
      const int64_t qrow = done.first + tokq;
      const int head = done.h * p.group + uq;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const float f = inv * __uint_as_float((127 + (unit >> 4 * g & 15)) << 23);
        const float x[4] = {o[g][0][i] * (k24 * f), o[g][0][2 + i] * (k20 * f), o[g][1][i] * (k24 * f),
                            o[g][1][2 + i] * (k20 * f)};
        if (whole)
          store_out4(p, qrow * p.out_stride + (int64_t)head * D + 32 * g + 4 * lr, x);
        else
          *(float4*)(part + col * D + 32 * g + 4 * lr) = make_float4(x[0], x[1], x[2], x[3]);
      }
      if (lr == 0) {
        if (!whole)
          ((float2*)(part + C::ROWS * D))[col] = make_float2(M[i], sum);
        else if (p.lse)
          p.lse[qrow * p.n_q_heads + head] = sum > 0.f ? (M[i] + log2f(sum)) * kLn2 : -INFINITY;
      }
    }
    if (!whole && lane == 0) {
      Left& x = left[warp * 2 + (from_start ? 1 : 0)];
      x.r = done.r;
      x.h = done.h;
      x.row0 = done.row0;
      x.rows = done.rows;
      x.has = 1;
      x.open = to_end ? 0 : 1;
      x.last = done_last;
    }
  }
  if (!ok) {
    // the copies of this tile and of those behind it may be under way (a stage that none was issued for costs
    // the whole time)
    for (int s = 0; s < C::STAGES; ++s) {
      const int at = stage + s < C::STAGES ? stage + s : stage + s - C::STAGES;
      mbar_drain(&bars[at], stage + s < C::STAGES ? phase : phase ^ 1);
    }
  }
  __syncthreads();

  // ---- the CTA's partials.  An item starts with a warp's second partial (or with the first warp's
  // first one, if it comes from the CTA before) and goes on in the next warps' first ones.  Bit w of
  // head / tail: warp w has a first / second partial; of on: its first one goes on in warp w + 1's.
  const int fl = lane < C::NW ? left[lane * 2].has | (left[lane * 2].open & 1) << 1 | left[lane * 2 + 1].has << 2 : 0;
  const uint32_t head = __ballot_sync(0xffffffffu, fl & 1), open_head = __ballot_sync(0xffffffffu, (fl & 3) == 3),
                 tail = __ballot_sync(0xffffffffu, fl & 4);
  const uint32_t on = open_head & (head >> 1);
  int job = 0, begun = -1;                 // the warp whose second partial goes on behind this CTA
  for (uint32_t todo = (head & 1) | tail << 1; todo; todo &= todo - 1) {
    const int w = __ffs(todo) - 2;         // -1: the first warp's first partial, else warp w's second
    const Left& x = w < 0 ? left[0] : left[w * 2 + 1];
    const int w0 = w < 0 ? 0 : w;
    const int s0 = w < 0 ? 0 : w + 1;      // the first of the item's first partials
    // a second partial always goes on; where the next warp has none, in the next CTA
    const bool more_here = w < 0 || (head >> s0 & 1);
    const int run = more_here ? __ffs(~(on >> s0)) : 0;               // first partials: s0 .. s0 + run - 1
    const int n = run + (w < 0 ? 0 : 1);   // partials of the item in this CTA
    const bool open = more_here ? open_head >> (s0 + run - 1) & 1 : true;
    const bool whole = w >= 0 && !open;
    if (w >= 0 && open) begun = w;
    auto part = [&](int i) -> const float* {
      return (const float*)(i == 0 && w >= 0 ? smem + C::OFF_RING + w * C::STAGES * C::STG
                                             : smem + C::OFF_HEAD + (w0 + i) * C::PART);
    };
    if (open && w >= 0 && !p.alone && threadIdx.x == 0)
      ws.desc[blockIdx.x] = make_int4(x.r, x.h, x.row0, share_of(x.last, N, U) / C::NW - (int)blockIdx.x);
    for (int col = 0; col < x.rows; ++col, ++job) {
      if (job % C::NW != warp) continue;
      // a lane weighs a partial, then all lanes add them up
      const float2 ml = lane < n ? ((const float2*)(part(lane) + C::ROWS * D))[col] : make_float2(kNone, 0.f);
      float m = ml.x;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float f = ex2(ml.x - m);
      float sum = ml.y * f, acc[G];
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      m = __shfl_sync(0xffffffffu, m, 0);  // lanes 16.. hold none
      sum = __shfl_sync(0xffffffffu, sum, 0);
#pragma unroll
      for (int v = 0; v < G; ++v) acc[v] = 0.f;
#pragma unroll 4
      for (int i = 0; i < n; ++i) {
        const float fi = __shfl_sync(0xffffffffu, f, i);
        const float* src = part(i) + col * D + lane * G;
#pragma unroll
        for (int v = 0; v < G; v += 2) {
          const float2 y = *(const float2*)(src + v);
          acc[v] = fmaf(y.x, fi, acc[v]);
          acc[v + 1] = fmaf(y.y, fi, acc[v + 1]);
        }
      }
      if (whole) {
        store_row<D>(p, x.r, x.h, x.row0 + col, lane, acc, m, sum);
      } else {
        const int64_t at = ((int64_t)blockIdx.x * 2 + (w < 0 ? 0 : 1)) * C::ROWS + col;
#pragma unroll
        for (int v = 0; v < G; v += 2)
          *(float2*)(ws.o + at * D + lane * G + v) = make_float2(acc[v], acc[v + 1]);
        if (lane == 0) ws.ml[at] = make_float2(m, sum);
      }
    }
  }
  // ---- a row tile's cluster: the first CTA joins what the others left, in their order
  const int cl = p.alone ? (int)cluster_nctarank() : 1;
  if (cl == 1) return;
  if (threadIdx.x == 0) ws.desc[blockIdx.x] = make_int4(0, 0, 0, head & 1);
  __syncwarp();
  cluster_sync_all();
  if (cluster_ctarank() != 0 || begun < 0) return;
  const Left& x1 = left[begun * 2 + 1];
  if (warp >= x1.rows) return;
  const uint32_t have = __ballot_sync(0xffffffffu, lane > 0 && lane < cl && __ldcg(ws.desc + blockIdx.x + lane).w);
  float m = kNone, sum = 0.f, acc[G];
#pragma unroll
  for (int v = 0; v < G; ++v) acc[v] = 0.f;
#pragma unroll 4
  for (int i = 0; i < cl; ++i) {
    if (i > 0 && !(have >> i & 1)) continue;
    const int64_t at = ((int64_t)(blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * C::ROWS + warp;
    const float2 ml = __ldcg(ws.ml + at);
    float2 y[G / 2];
#pragma unroll
    for (int v = 0; v < G / 2; ++v) y[v] = __ldcg((const float2*)(ws.o + at * D + lane * G) + v);
    const float mn = fmaxf(m, ml.x), f0 = ex2(m - mn), f1 = ex2(ml.x - mn);
    m = mn;
    sum = sum * f0 + ml.y * f1;
#pragma unroll
    for (int v = 0; v < G / 2; ++v) {
      acc[2 * v] = acc[2 * v] * f0 + y[v].x * f1;
      acc[2 * v + 1] = acc[2 * v + 1] * f0 + y[v].y * f1;
    }
  }
  store_row<D>(p, x1.r, x1.h, x1.row0 + warp, lane, acc, m, sum);
}

// Joins the partials of the items that go over several CTAs' shares.  CTA c
// looks after the item that starts in CTA c of the kernel above and goes on behind
// it; a warp takes a row and one of kSub interleaved shares of its partials.  Bound by latency:
// about 3 us behind the kernel above, whose CTAs leave no room for these before they end, so small CTAs
// start sooner: a kernel behind an empty join waits 3.6 us less for 2 shares than for 4.
// (Heads of 256, with four values more per lane, are joined 0.5 us sooner by 4.)
template <int D>
constexpr int kSub = D == 256 ? 4 : 2;

template <int D>
__global__ void __launch_bounds__(256 * kSub<D>) kv_stream_join_kernel(const __grid_constant__ AttnParams p) {
  using C = StreamCfg<D>;
  constexpr int G = D / 32;                // values of a row per lane
  __shared__ float acc_s[8][kSub<D>][D];
  __shared__ float2 ml_s[8][kSub<D>];
  pdl_wait();
  pdl_trigger();
  const StreamWs ws = stream_ws(p.ws);
  const int4 d = __ldcg(ws.desc + blockIdx.x);
  const int follow = d.w;                  // CTAs behind this one that the item goes on in
  if (follow == 0) return;                 // uniform for the CTA
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = warp >> 3, col = warp & 7;
  int first, all;
  const int rows = min(C::ROWS, q_rows(p, d.x, &first, &all) * p.group - d.z);
  const bool live = col < rows;
  // partial 0 is this CTA's second one, the others the first ones of the CTAs after it
  auto part = [&](int i) -> int64_t {
    return ((int64_t)(blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * C::ROWS + col;
  };
  // The loads wait for nothing but the descriptor (a row behind the item's last is read and not used).
  float m = kNone, l = 0.f, acc[G];
#pragma unroll
  for (int v = 0; v < G; ++v) acc[v] = 0.f;
#pragma unroll (G > 4 ? 2 : 4)
  for (int i = sub; i <= follow; i += kSub<D>) {
    const int64_t at = part(i);
    const float2 ml = __ldcg(ws.ml + at);
    float2 x[G / 2];
#pragma unroll
    for (int v = 0; v < G / 2; ++v) x[v] = __ldcg((const float2*)(ws.o + at * D + lane * G) + v);
    const float mn = fmaxf(m, ml.x), f0 = ex2(m - mn), f1 = ex2(ml.x - mn);
    m = mn;
    l = l * f0 + ml.y * f1;
#pragma unroll
    for (int v = 0; v < G / 2; ++v) {
      acc[2 * v] = acc[2 * v] * f0 + x[v].x * f1;
      acc[2 * v + 1] = acc[2 * v + 1] * f0 + x[v].y * f1;
    }
  }
#pragma unroll
  for (int v = 0; v < G; v += 2)
    *(float2*)&acc_s[col][sub][lane * G + v] = make_float2(acc[v], acc[v + 1]);
  if (lane == 0) ml_s[col][sub] = make_float2(m, l);
  __syncthreads();
  if (sub == 0 && live) {
    float mt = kNone, lt = 0.f, x[G];
    for (int k = 0; k < kSub<D>; ++k) mt = fmaxf(mt, ml_s[col][k].x);
#pragma unroll
    for (int v = 0; v < G; ++v) x[v] = 0.f;
#pragma unroll
    for (int k = 0; k < kSub<D>; ++k) {
      const float f = ex2(ml_s[col][k].x - mt);
      lt = fmaf(ml_s[col][k].y, f, lt);
#pragma unroll
      for (int v = 0; v < G; v += 2) {
        const float2 y = *(const float2*)&acc_s[col][k][lane * G + v];
        x[v] = fmaf(y.x, f, x[v]);
        x[v + 1] = fmaf(y.y, f, x[v + 1]);
      }
    }
    store_row<D>(p, d.x, d.y, d.z + col, lane, x, mt, lt);
  }
}

template <int D, int MODE>
int launch_stream(AttnParams p, int ctas, cudaStream_t s) {
  using C = StreamCfg<D>;
  static bool attr[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DQ_ERR_CUDA;
  if (dev >= 64 || !attr[dev]) {
    if (cudaFuncSetAttribute(kv_stream_kernel<D, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::SMEM) != cudaSuccess)
      return DQ_ERR_CUDA;
    if (dev < 64) attr[dev] = true;
  }
  // what a row tile sees: the table's tokens, or a window and the tokens of 8 rows
  const int64_t tokens = std::min<int64_t>((int64_t)p.max_pages << p.g.page_shift,
                                           p.window > 0 ? (int64_t)p.window + 7 : INT64_MAX);
  const int64_t per = (std::min<int64_t>((int64_t)p.max_q_len * p.group, p.rows_upto) + C::ROWS - 1) / C::ROWS;
  const int64_t items = per * p.B * p.g.heads;
  const int64_t tiles = tokens / kTile + 2;
  int cl = 1;
  while (cl < 4 && items * cl * 2 <= kClusterCtas && tiles > 3 * cl * C::NW) cl *= 2;
  const int more = cl > 1 ? kAloneTiles<D> / 2 : kAloneTiles<D>;
  const bool alone = items <= ctas && tiles * (ctas - items * cl) <= (int64_t)more * C::NW * cl * ctas &&
                     tiles <= kAloneMost * C::NW * cl;
  p.alone = alone ? (int)per : 0;
  if (launch_pdl(kv_stream_kernel<D, MODE>, dim3(alone ? (int)items * cl : ctas), dim3(C::NTH), C::SMEM, s,
                 alone && cl > 1 ? cl : 0, p) != cudaSuccess)
    return DQ_ERR_CUDA;
  if (alone) return cudaGetLastError() == cudaSuccess ? DQ_OK : DQ_ERR_CUDA;
  if (launch_pdl(kv_stream_join_kernel<D>, dim3(ctas), dim3(256 * kSub<D>), 0, s, 0, p) != cudaSuccess)
    return DQ_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? DQ_OK : DQ_ERR_CUDA;
}

template <int MODE>
int launch_stream_any(const AttnParams& p, int head_dim, cudaStream_t s) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return DQ_ERR_CUDA;
  const int ctas = std::min(sms, kMaxCtas);
  if (head_dim == 64) return launch_stream<64, MODE>(p, ctas, s);
  if (head_dim == 128) return launch_stream<128, MODE>(p, ctas, s);
  return launch_stream<256, MODE>(p, ctas, s);
}

}  // namespace
}  // namespace dqmoe
