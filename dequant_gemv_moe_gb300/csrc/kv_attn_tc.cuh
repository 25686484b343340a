// kv_attn_tc.cuh — attention of many query rows (prompts and chunks of prompts)
// over the 4-bit paged cache, on the 5th-generation tensor core.
//
// Mathematics.  A CTA holds up to 256 rows of one K/V head (two 128-row tiles;
// one for head_dim 256) and walks tiles of 64 tokens: S = Q K^T in tensor
// memory, p = 2^(s - M) per row, O += P V with P read from tensor memory.  With
// this many rows the codes are decoded once per tile for all of them:
// * K and V become fp16 values (c - 8) d, one rounding, in 128-byte swizzled
//   panels of 64 values; V's panel keeps its token rows and is read with N along
//   the row.  The V columns stay in the order in which the codes lie in their
//   words; the output is put in order when it is stored.
// * Q rows are scaled by a power of two into fp16 (exact but for values 2^-28
//   below the row's largest); the factor comes back with the softmax's scale.
// * M is a row's maximum less 8 when it is set, and set again only when the sum of
//   a tile's weights passes 2^15: fp16 weights stay between 2^8 and 2^15 at the top, no
//   maximum is taken of most tiles, and O, which lives in tensor memory, is rescaled a
//   few times per row at most.  Rounding K, V and p to fp16 (2^-11 each) is the price of
//   16-bit operands; S, M, the sum of p and O are fp32.  (Against 64 bits, norm over norm: fp32 outputs
//   2.8e-4 for 7 prompts of heads of 64, 4.0e-4 for the long chunk below, of which fp16 and bf16 outputs
//   round off 2.1e-4 and 1.7e-3; lse 6.0e-6 and 2.6e-6.  The streaming kernel, which takes K exactly:
//   1.6e-4 to 2.1e-4, lse 1.2e-7.  K exactly here, where scores are masked, capped or biased: lse 2e-7 to 8e-7.)
//
// Roles.  Warp groups of the row tiles do the softmax (a thread per row); eight
// warps decode; one warp copies the pages' blocks (bulk copies, 32 tokens at a
// time); one warp per row tile issues its products.  Every row tile has two score buffers, which
// take turns: while a row's thread works on one tile, the products of the one before
// and the scores of the one after run.
//
// Work is shared as in kv_attn_stream.cuh: the line of all (request, row tile,
// head, token tile) units in equal shares, one per CTA, the partials of items
// that cross shares joined in order by a second kernel.
//
// What bounds it: the turns that softmax, decoding and products take.  The softmax (160
// instructions for 64 scores) and the decoding (13 for 8 values) share four schedulers that
// issue in 0.59 of the cycles, the tensor pipe is busy in half of them, and neither is full.  2
// requests' chunks of 2048 tokens over up to 16384, 32 query heads on 8 of 128: 935 to 945 us, 1.24
// PFLOP/s.  Left out for a measurement (of 955 us then), the decoding's arithmetic took 15 % of
// the time, the exponentials none, three quarters of the products 6 %.  Four warps decoding and 64
// scores a thread at a time took 966 us, two warps to a row 1088 (registers).
// Modes other than kPlain: prefixes and first positions, capped scores, a distance bias (dq_kv_scores), an instance each:
// the softmax's loop misses the instruction cache where it holds more than it needs.  Two cases stand for them in what
// follows: docs_prompts, 7 prompts of documents with prefixes up to 3001 tokens, 12 heads of 64 (159 us in an instance
// that can cap as well, 137 with masks alone, 87 since masks are bits and K and V are released apart), and cap_chunk,
// the chunks of above with scores capped at 30 (1435 us; with a bias instead 1205).  A cap takes an ex2 and half an
// inverse a score beside the softmax's own ex2: their pipe is busy in 0.36 of the cycles, issue in 0.49, the tensor pipe
// in 0.36, and two softmax warps to a scheduler do not hide the chain from a score to its weight.
#pragma once

#include <algorithm>
#include <type_traits>

#include "kv_attn.h"
#include "tc.cuh"

namespace dqmoe {

namespace {

constexpr int kMaxCtas = 160;
constexpr int kPiece = 32;                 // tokens per copy stage

// Bits f to n - 1 of 32: predicates come out of a register's bits by the seven, where a comparison makes one.
__device__ __forceinline__ uint32_t seen_bits(int f, int n) {
  uint32_t m;
  f = max(f, 0);
  asm("bmsk.clamp.b32 %0, %1, %2;" : "=r"(m) : "r"(f), "r"(max(n - f, 0)));
  return m;
}

template <int D, int MODE = kPlain>
struct TcCfg {
  static constexpr int NQ = kTcRowTiles<D>;          // 128-row tiles
  static constexpr int TT = kTcTile;                 // tokens per tile
  static constexpr int KVS = D == 256 ? 2 : 4;   // decoded tiles of K and of V
  static constexpr int ROWS = 128 * NQ;
  static constexpr int Q_TILE = 128 * D * 2;
  static constexpr int KV_BUF = TT * D * 2;
  static constexpr int PIECE_B = kPiece / kKvBlk * KvBlk<D>::BYTES;
  static constexpr int RS = D == 64 ? 8 : D == 128 ? 6 : 3;
  static constexpr int OFF_SHARE = 496;              // int64 [2], behind the barriers
  static constexpr int OFF_PRE = 512;
  static constexpr int OFF_Q = 6144;
  static constexpr int OFF_K = OFF_Q + NQ * Q_TILE;
  static constexpr int OFF_V = OFF_K + KVS * KV_BUF;
  static constexpr int OFF_RAW = OFF_V + KVS * KV_BUF;
  static constexpr int SMEM = OFF_RAW + RS * PIECE_B;
  static constexpr int DEC0 = 4 * NQ;                // first decoding warp
  // decoding warps: capped scores keep the softmax so long that four are enough, and the registers of the others
  // let its threads hold 64 scores, but not with one row tile to twice the values a token (chunks of 2048 over 16384 with four
  // and eight: capped, 32 heads of 128 1432 and 1680 us, of 64 1330 and 1541, 16 of 256 2625 and 2380; capped and biased
  // 2106 and 2195, 2040 and 2105, 2755 and 2466; biased, 2 % faster then, 1213 and 1178, 972 and 974, 2609 and 2361)
  static constexpr int DW = (MODE == kCaps || MODE == kAnyScores) && D != 256 ? 4 : 8;
  static constexpr int PROD = DEC0 + DW, MMA = PROD + 1;  // one warp of products per row tile
  static constexpr int NTH = 32 * (MMA + NQ);
  // tensor memory columns: O of every row tile, then two score buffers of each
  static constexpr int COL_S = NQ * D;
  static_assert(COL_S + NQ * 2 * TT <= 512, "tensor memory");
  static_assert(TT == 2 * kPiece && RS >= 3, "a tile is two pieces");
  static_assert((2 * RS + 3 * KVS + 16) * 8 + 4 <= OFF_SHARE && (NTH + 1 + NTH / 32) * 8 <= OFF_Q - OFF_PRE &&
                    SMEM <= 232448, "shared memory");
};

constexpr size_t kTcO = (size_t)kMaxCtas * 2 * 256 * 128 * 4;   // ROWS * D is at most 256 * 128
constexpr size_t kTcMl = (size_t)kMaxCtas * 2 * 256 * 8;
constexpr size_t kTcDesc = (size_t)kMaxCtas * 16;

struct TcWs {
  float* o;
  float2* ml;
  int4* desc;
};
__device__ __forceinline__ TcWs tc_ws(uint8_t* ws) {
  TcWs w;
  w.o = (float*)ws;
  w.ml = (float2*)(ws + kTcO);
  w.desc = (int4*)(ws + kTcO + kTcMl);
  return w;
}

// 32 columns of this thread's lane; the values are there after tmem_wait_ld and tmem_use.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
// The values pass through here after the wait: nothing that uses them can move before it.
__device__ __forceinline__ void tmem_use(uint32_t* r) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile(""
                 : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]),
                   "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7]));
}
__device__ __forceinline__ void tmem_use8(uint32_t* r) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// tcgen05.mma with descriptors as their 32-bit halves: only the low one (the address) changes from
// product to product, one addition each.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 db, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// One lane of the (converged) warp, as the compiler knows it.
__device__ __forceinline__ bool elect_one() {
  uint32_t v;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(v));
  return v != 0;
}
// A value that is the same in every lane, in a form the compiler can see.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// Shared-memory descriptor of an operand whose rows run along M / N (here V: the
// row of a token holds 64 values of N): 128-byte swizzled panels of 64 values,
// `panel` bytes apart, 8 tokens (K) every 1024 bytes.
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t addr, uint32_t panel) {
  uint64_t d = 0;
  d |= (uint64_t)((addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(panel >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
constexpr uint32_t kBRowsAlongN = 1u << 16;

// The 8 codes of a word as c - 8: four pairs, in the order of the nibble pairs.  By the well-known exponent
// trick: a nibble or-ed into the mantissa of 1024 is 1024 + c, or 1024 + 16 c one nibble up; one addition, or one
// FMA with 1/16, takes off what is too much.
__device__ __forceinline__ void decode8(uint32_t w, __half2 (&c)[4]) {
  const __half2 bias = u32_as_h2(0x64086408u);        // 1032
  const __half2 sixteenth = u32_as_h2(0x2C002C00u), m72 = u32_as_h2(0xD480D480u);
  const uint32_t w8 = w >> 8, magic = 0x64006400u;
  c[0] = __hsub2(u32_as_h2(lop3_and_or(w, 0x000F000Fu, magic)), bias);
  c[1] = __hfma2(u32_as_h2(lop3_and_or(w, 0x00F000F0u, magic)), sixteenth, m72);
  c[2] = __hsub2(u32_as_h2(lop3_and_or(w8, 0x000F000Fu, magic)), bias);
  c[3] = __hfma2(u32_as_h2(lop3_and_or(w8, 0x00F000F0u, magic)), sixteenth, m72);
}
__device__ __forceinline__ uint4 times(const __half2 (&c)[4], __half2 d) {
  return make_uint4(h2_as_u32(__hmul2(c[0], d)), h2_as_u32(__hmul2(c[1], d)), h2_as_u32(__hmul2(c[2], d)),
                    h2_as_u32(__hmul2(c[3], d)));
}
// The first 8 significant bits of a scale: (c - 8) times them is exact in fp16, and so is (c - 8) times the
// rest.  (Cut, not rounded: 8 * 8188 must not pass the largest fp16.)
__device__ __forceinline__ __half2 scale_top(__half2 d) { return u32_as_h2(h2_as_u32(d) & 0xFFF8FFF8u); }

__device__ __forceinline__ void sts_u128(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

// The power of two that brings a row's largest magnitude into [2^14, 2^15) (1 for a row of zeros).
__device__ __forceinline__ float row_up(float mx) {
  const int ex = (int)((__float_as_uint(mx) >> 23) & 255) - 127;
  return mx > 0.f ? __uint_as_float((uint32_t)(127 + min(14 - ex, 100)) << 23) : 1.f;
}

template <int D, int MODE>
__global__ void __launch_bounds__(TcCfg<D, MODE>::NTH, 1) kv_tc_kernel(const __grid_constant__ AttnParams p) {
  using C = TcCfg<D, MODE>;
  using B = KvBlk<D>;
  constexpr bool EXT = MODE != kPlain, ANY = MODE == kAnyScores, BIAS = MODE == kBias || ANY;
  // Masks as bits (docs_prompts 130 -> 115 us, cap_chunk 1400 -> 1378; without masks and
  // with a bias comparisons by the row tile's take less: 880 and 1052 us for the chunk so, 908 and 1086 with bits)
  constexpr bool BITS = MODE != kPlain && MODE != kBias;
  // A bias falls with the distance: from the last tile to the first one, M hardly has to follow.
  constexpr bool BACK = BIAS;
  // Where scores are masked, capped or biased they are exact, from two K's a tile, whatever a row sees: a few tokens may
  // carry its sum (lse 1e-5 to 4e-5 off with K rounded, 1e-7 so).  K and V are then released apart, K once its scores are
  // there: two tiles' K's and four tiles' V's are in turn (cap_chunk 2263 -> 1452 us with exact scores, 1372 with rounded
  // ones; docs_prompts 107 -> 92.  Without masks, where few tiles need it, the chunk takes 903 us so, 878 as it is.)
  constexpr bool SPLIT = EXT;
  using Wk = TcWalk<D, EXT>;
  constexpr int G = B::G, W = B::W, GH = G / W, NQ = C::NQ, TT = C::TT;
  constexpr int LPR = D / 8, RPI = 32 / LPR, QB = D == 64 ? 8 : 4;   // rows to and from the warps
  extern __shared__ __align__(1024) uint8_t smem[];
  pdl_wait();
  pdl_trigger();
  // the swizzle needs a window aligned to 1024 bytes: the kernel has no static shared memory,
  // which the linker would put in front of it
  uint64_t* raw_full = (uint64_t*)smem;
  uint64_t* raw_empty = raw_full + C::RS;
  uint64_t* kv_full = raw_empty + C::RS;
  uint64_t* k_empty = kv_full + C::KVS;
  uint64_t* v_empty = k_empty + C::KVS;
  uint64_t* s_full = v_empty + C::KVS;     // [row tile][tile parity], as the next two
  uint64_t* p_full = s_full + 4;
  uint64_t* pv_done = p_full + 4;
  uint64_t* q_full = pv_done + 4;
  uint64_t* drained = q_full + 2;
  uint32_t* tmem_slot = (uint32_t*)(drained + 2);
  int64_t* pre = (int64_t*)(smem + C::OFF_PRE);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  int* known = (int*)(smem + C::OFF_Q);    // (Q comes after the walk's start)
  static_assert(C::NTH * 16 <= NQ * C::Q_TILE, "shared memory");
  Wk::template sum_units<C::NTH>(p, pre, known);
  const int64_t U = pre[C::NTH];
  const int N = tc_shares(gridDim.x, U);
  const TcWs ws = tc_ws(p.ws);
  if (threadIdx.x == 0) ws.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
  if (blockIdx.x >= N) return;
  // the share, in shared memory: the roles' loops need their registers (prompts with heads of 64 147 -> 141
  // us, the long chunk 947 -> 930)
  int64_t* share = (int64_t*)(smem + C::OFF_SHARE);
  if (threadIdx.x == 0) {
    share[0] = share_start(U, N, blockIdx.x);
    share[1] = share_start(U, N, blockIdx.x + 1);
    for (int i = 0; i < C::RS; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], 4);
    }
    for (int i = 0; i < C::KVS; ++i) {
      mbar_init(&kv_full[i], 32 * C::DW);
      mbar_init(&k_empty[i], NQ);
      mbar_init(&v_empty[i], NQ);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 128);
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(&q_full[0], 128);
    mbar_init(&q_full[1], 128);
    mbar_init(&drained[0], 1);
    mbar_init(&drained[1], 1);
    fence_barrier_init();
  }
  if (warp == C::MMA) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t qs = smem_u32(smem + C::OFF_Q), ks = smem_u32(smem + C::OFF_K),
                 vs = smem_u32(smem + C::OFF_V);

  Item it;
  int64_t iu = Wk::template seek<C::NTH>(p, pre, share[0], it, known);
  int ta, tb;                              // the tiles of the item that this share holds
  bool ok = true;
  __syncthreads();

  if (warp < C::DEC0) {
    // ------------------------------ softmax ------------------------------
    const int tile = warp >> 2;            // row tile
    const int trow = 32 * (warp & 3) + lane;
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t o_addr = tmem + lane_base + (uint32_t)(tile * D);
    const uint32_t qrow = qs + tile * C::Q_TILE;
    int slot = 0;                          // of this CTA's partials
    int gt = 0;                            // tiles so far
    for (bool more = Wk::here(p, it, iu, share[0], share[1], ta, tb); more;
         more = Wk::after(p, it, iu, share[0], share[1], ta, tb)) {
      const bool from_start = ta == 0, to_end = tb == it.tiles;
      int ra, rb;
      row_tile_range<EXT>(p, it, tile, ta, tb, ra, rb);
      const int nt = rb - ra;              // tiles of this row tile
      // the row
      const bool live = tile * 128 + trow < it.rows;
      const int row = it.row0 + min(tile * 128 + trow, it.rows - 1);   // (the last row again behind it)
      const int tokq = row_token(p, row), uq = row - tokq * p.group;
      const int64_t q_at = it.first + tokq;
      const int head = it.h * p.group + uq;
      float cf = 0.f;
      if (nt > 0) {
        // The warp loads its 32 rows, LPR lanes a row: 16 bytes a lane, whole rows at a time.
        float own = 0.f;                   // the largest magnitude of this thread's row
#pragma unroll
        for (int i0 = 0; i0 < 32 / RPI; i0 += QB) {
          uint4 raw[QB];
#pragma unroll
          for (int k = 0; k < QB; ++k) {
            const int lr = tile * 128 + 32 * (warp & 3) + (i0 + k) * RPI + lane / LPR;
            const int rw = it.row0 + lr, tq = row_token(p, rw), u = rw - tq * p.group;
            const uint16_t* src = (const uint16_t*)p.q + (int64_t)(it.first + tq) * p.q_stride +
                                  ((int64_t)it.h * p.group + u) * D + 8 * (lane % LPR);
            raw[k] = lr < it.rows ? __ldg((const uint4*)src) : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int k = 0; k < QB; ++k) {
            const uint32_t w4[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
            float2 f[4];
            float mx = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (p.q_dtype == DQ_BF16)
                f[i] = make_float2(__uint_as_float(w4[i] << 16), __uint_as_float(w4[i] & 0xFFFF0000u));
              else
                f[i] = __half22float2(u32_as_h2(w4[i]));
              mx = fmaxf(mx, fmaxf(fabsf(f[i].x), fabsf(f[i].y)));
            }
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float got = __shfl_sync(0xffffffffu, mx, (lane % RPI) * LPR);
            if (lane / RPI == i0 + k) own = got;
            const float up = row_up(mx);
            uint32_t r4[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) r4[i] = h2_as_u32(__floats2half2_rn(f[i].x * up, f[i].y * up));
            const int tr = 32 * (warp & 3) + (i0 + k) * RPI + lane / LPR, ch = lane % LPR;
            sts_u128(qrow + ch / 8 * 16384 + sw128_offset(tr, ch & 7), make_uint4(r4[0], r4[1], r4[2], r4[3]));
          }
        }
        cf = fmaxf(p.scale * kLog2e / row_up(own), kLeastScale);
        if (MODE == kCaps) cf *= p.cap_inv * (2.f * kLog2e);
        if (ANY) cf *= p.cap_inv;
        fence_proxy_async_smem();
        mbar_arrive(&q_full[tile]);
      }
      const int pos = it.shift + tokq;
      const int prefix = EXT ? it.prefix : 0;
      const int hi = seen_end(p, it.len, pos, prefix);
      int lo = first_seen(p, pos);
      if (EXT) lo = max(lo, row_first(p, (int)q_at));
      int lo_all, hi_all;                  // what all of the row tile's rows see, or of the warp's
      if (EXT) {
        hi_all = __reduce_min_sync(0xffffffffu, hi);
        lo_all = __reduce_max_sync(0xffffffffu, lo);
      } else {
        const int pa = it.shift + row_token(p, it.row0 + min(it.rows - 1, tile * 128));
        const int pb = it.shift + row_token(p, it.row0 + min(it.rows, tile * 128 + 128) - 1);
        hi_all = seen_end(p, it.len, pa);
        lo_all = first_seen(p, pb);
      }
      const float cfs = ANY ? 1.f : cf;    // of the scores that the softmax reads
      const float slope = BIAS && p.slopes ? __ldg(p.slopes + head) * -kLog2e : 0.f;
      float M = kNone, l = 0.f;
      for (int j = 0; j < nt; ++j, ++gt) {
        const int tok0 = (it.t0 + (BACK ? rb - 1 - j : ra + j)) * TT;
        const int sl = tile * 2 + (gt & 1);
        ok = ok && mbar_wait(&s_full[sl], (gt >> 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t s_addr = tmem + lane_base + (uint32_t)(C::COL_S + sl * TT);
        const bool inner = tok0 >= lo_all && tok0 <= hi_all - TT;
        // Any cap, any bias: the scores, in units of log 2, capped and biased, take their own place in a pass in front of
        // the softmax's.  (1050 -> 1870 us for cap_chunk, in its warps or in others: tensor memory's
        // bandwidth.  The polynomial in the softmax's passes misses the instruction cache: 3970.)
        if (ANY) {
          // a bias is linear in the position on either side of the row's own
          const bool one_side = (p.causal && !p.prefix) || __all_sync(0xffffffffu, pos >= tok0 + TT);
#pragma unroll 1
          for (int c = 0; c < TT; c += 16) {
            uint32_t r[16];
            tmem_ld16(s_addr + c, r);
            const float d = (float)(pos - tok0 - c);
            tmem_wait_ld();
            tmem_use8(r);
            tmem_use8(r + 8);
#pragma unroll
            for (int h = 0; h < 16; h += 8) {
              float2 t[4];
              float far = 0.f;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                t[i] = fmul2(make_float2(__uint_as_float(r[h + 2 * i]), __uint_as_float(r[h + 2 * i + 1])),
                             make_float2(cf, cf));
                far = max3(far, fabsf(t[i].x), fabsf(t[i].y));
              }
              if (p.cap > 0.f) {
                if (__any_sync(0xffffffffu, far > 1.f)) soft_cap_far(p, t);
                else soft_cap(p, t);
              }
              if (p.slopes) {
                if (one_side) {
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    const float at = d - (float)(h + 2 * i);
                    t[i] = ffma2(make_float2(at, at - 1.f), make_float2(slope, slope), t[i]);
                  }
                } else {
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    t[i].x = fmaf(fabsf(d - (float)(h + 2 * i)), slope, t[i].x);
                    t[i].y = fmaf(fabsf(d - (float)(h + 2 * i + 1)), slope, t[i].y);
                  }
                }
              }
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                r[h + 2 * i] = __float_as_uint(t[i].x);
                r[h + 2 * i + 1] = __float_as_uint(t[i].y);
              }
            }
            tmem_st16(s_addr + c, r);
          }
          tmem_wait_st();
        }
        // 32 values of this thread's row in units of log 2, capped or biased, less `less`; -inf where it does not see
        auto values = [&](int c, float less, uint32_t (&r)[32]) {
          if (MODE == kCaps) {
            // cap tanh(u) = cap - 2 cap / (1 + e^2u), cf from the score to 2 u log2 e; two inverses from that of the
            // product, which 2^60 keeps finite (tanh is 1 there)
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              const float2 t = fmul2(make_float2(__uint_as_float(r[k]), __uint_as_float(r[k + 1])), make_float2(cf, cf));
              r[k] = __float_as_uint(fminf(t.x, 60.f));
              r[k + 1] = __float_as_uint(fminf(t.y, 60.f));
            }
#pragma unroll
            for (int k = 0; k < 32; ++k) asm volatile("ex2.approx.ftz.f32 %0, %0;" : "+r"(r[k]));
            uint32_t m[16];
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              const float2 t = fadd2(make_float2(__uint_as_float(r[k]), __uint_as_float(r[k + 1])), make_float2(1.f, 1.f));
              r[k] = __float_as_uint(t.x);
              r[k + 1] = __float_as_uint(t.y);
              m[k / 2] = __float_as_uint(t.x * t.y);
            }
#pragma unroll
            for (int k = 0; k < 16; ++k) asm volatile("rcp.approx.ftz.f32 %0, %0;" : "+r"(m[k]));
            const float2 f2 = make_float2(-2.f * p.cap, -2.f * p.cap), m2 = make_float2(p.cap - less, p.cap - less);
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              const float i = __uint_as_float(m[k / 2]);
              const float2 v = fmul2(make_float2(__uint_as_float(r[k + 1]), __uint_as_float(r[k])), make_float2(i, i));
              const float2 t = ffma2(v, f2, m2);
              r[k] = __float_as_uint(t.x);
              r[k + 1] = __float_as_uint(t.y);
            }
          } else {
            // a bias is linear in the position on either side of the row's own
            const float d = (float)(pos - tok0 - c);
            if ((p.causal && !p.prefix) || __all_sync(0xffffffffu, pos >= tok0 + TT)) {
              // (distances are exact; running sums of the slope drift by a rounding each: 1185 us for the chunk instead of 1205,
              // but 1e-4 off for a slope of 30, 5e-6 for small ones)
              float2 at = make_float2(d, d - 1.f);
              const float2 s2 = make_float2(slope, slope), l2 = make_float2(-less, -less);
#pragma unroll
              for (int k = 0; k < 32; k += 2) {
                const float2 t = ffma2(make_float2(__uint_as_float(r[k]), __uint_as_float(r[k + 1])), make_float2(cf, cf),
                                       ffma2(at, s2, l2));
                at = fadd2(at, make_float2(-2.f, -2.f));
                r[k] = __float_as_uint(t.x);
                r[k + 1] = __float_as_uint(t.y);
              }
            } else {
#pragma unroll
              for (int k = 0; k < 32; ++k)
                r[k] = __float_as_uint(fmaf(__uint_as_float(r[k]), cf, fmaf(fabsf(d - (float)k), slope, -less)));
            }
          }
          if (!inner) {
            const int n = hi - tok0 - c, f = lo - tok0 - c;
            const uint32_t see = BITS ? seen_bits(f, n) : 0;
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = (BITS ? see >> i & 1 : i < n && i >= f) ? r[i] : 0xFF800000u;
          }
        };
        // 32 scores of this thread's row, those that it does not see as -inf (not with a bias: `values`)
        auto load = [&](int c, uint32_t (&r)[32]) {
          tmem_ld32(s_addr + c, r);
          tmem_wait_ld();
          tmem_use(r);
          if (BITS && !inner) {
            const uint32_t see = seen_bits(lo - tok0 - c, hi - tok0 - c);
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = see >> i & 1 ? r[i] : 0xFF800000u;
          } else if (!inner) {
            const int n = hi - tok0 - c;
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = i < n ? r[i] : 0xFF800000u;
            if (p.window > 0) {
              const int f = lo - tok0 - c;
#pragma unroll
              for (int i = 0; i < 32; ++i) r[i] = i >= f ? r[i] : 0xFF800000u;
            }
          }
        };
        uint32_t w[TT / 2];
        float sum;
        // The first tile sets M.  After that the sum of the weights tells whether M has to follow: while it
        // is at most 2^15, so is every weight.  If it is not, the tile is done again with a new M.
        for (bool renew = j == 0;; renew = true) {
          if (renew) {
            float mx = -INFINITY;
#pragma unroll 1
            for (int c = 0; c < TT; c += 32) {
              uint32_t r[32];
              if (MODE == kBias) {
                tmem_ld32(s_addr + c, r);
                tmem_wait_ld();
                tmem_use(r);
                values(c, 0.f, r);
              } else {
                load(c, r);
              }
              float mx4[4] = {mx, mx, mx, mx};
#pragma unroll
              for (int i = 0; i < 32; i += 8)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  mx4[k] = max3(mx4[k], __uint_as_float(r[i + 2 * k]), __uint_as_float(r[i + 2 * k + 1]));
              mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
            }
            if (MODE != kBias) mx *= cfs;
            // (a cap rises with its score)
            if (MODE == kCaps && mx > -INFINITY) mx = p.cap - 2.f * p.cap * rcp_ftz(1.f + ex2(fminf(mx, 60.f)));
            // (At most M + 9: a sum of 64 2^9 at most.  Scores that a cap is for lie further apart: more room
            // above, for less below; cap_chunk's rows follow 20 % less often.)
            const float mn = mx > M + 9.f ? mx - (MODE == kCaps || ANY ? 4.f : 8.f) : M;
            const float corr = ex2(M - mn);
            M = mn;
            l *= corr;
            if (j > 0) {
              // the product of the tile before may still be running
              ok = mbar_wait(&pv_done[tile * 2 + ((gt - 1) & 1)], ((gt - 1) >> 1) & 1);
              ok = __all_sync(0xffffffffu, ok);
              if (!ok) break;
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                uint32_t v[32];
                tmem_ld32(o_addr + 32 * c, v);
                tmem_wait_ld();
                tmem_use(v);
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * corr);
                tmem_st32(o_addr + 32 * c, v);
              }
            }
          }
          const float2 cf2 = make_float2(cfs, cfs), m2 = make_float2(-M, -M);
          float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          uint32_t both[MODE == kCaps ? TT : 1];
          if (MODE == kCaps) {
            tmem_ld32(s_addr, both);
            tmem_wait_ld();
            tmem_use(both);
            tmem_ld32(s_addr + 32, both + (MODE == kCaps ? 32 : 0));
          }
#pragma unroll
          for (int h = 0; h < TT; h += 32) {
            uint32_t r[32];
            if (MODE == kCaps) {
              if (h > 0) {
                tmem_wait_ld();
                tmem_use(both + (MODE == kCaps ? 32 : 0));
              }
#pragma unroll
              for (int k = 0; k < 32; ++k) r[k] = both[MODE == kCaps ? h + k : 0];
              values(h, M, r);
            } else if (MODE == kBias) {
              tmem_ld32(s_addr + h, r);
              tmem_wait_ld();
              tmem_use(r);
              values(h, M, r);
            } else {
            load(h, r);
            // in three passes over the registers: the exponentials' latencies overlap
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              const float2 t = ffma2(make_float2(__uint_as_float(r[k]), __uint_as_float(r[k + 1])), cf2, m2);
              r[k] = __float_as_uint(t.x);
              r[k + 1] = __float_as_uint(t.y);
            }
            }
#pragma unroll
            for (int k = 0; k < 32; ++k) asm volatile("ex2.approx.ftz.f32 %0, %0;" : "+r"(r[k]));
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              const float2 e = make_float2(__uint_as_float(r[k]), __uint_as_float(r[k + 1]));
              l2[(k >> 1) & 1] = fadd2(l2[(k >> 1) & 1], e);
              w[(h + k) >> 1] = h2_as_u32(__floats2half2_rn(e.x, e.y));
            }
          }
          sum = (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y);
          if (renew || !__any_sync(0xffffffffu, sum > 32768.f)) break;
        }
        if (!ok) break;
        // the weights go over the scores, two to a column
        tmem_st32(s_addr, w);
        l += sum;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&p_full[sl]);
      }
      if (!ok) break;
      // ---- the rows: whole, or a partial
      {
        if (nt > 0) {
          ok = mbar_wait(&pv_done[tile * 2 + ((gt - 1) & 1)], ((gt - 1) >> 1) & 1);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
        }
        const bool whole = from_start && to_end;
        const float inv = whole ? (l > 0.f ? 1.f / l : 0.f) : 1.f;
        const int64_t part = ((int64_t)blockIdx.x * 2 + slot) * C::ROWS + tile * 128 + trow;
        // The rows go through the row tile's place in shared memory (its last scores are done): a thread
        // puts its own there, the warp takes them out row by row.  16-bit outputs in one round, fp32 in
        // two of half a row.
        const bool f32 = !whole || p.out_dtype == DQ_F32;
        for (int round = 0; round < (f32 ? 2 : 1); ++round) {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            if (f32 && D > 64 && c / (D / 64) != round) continue;
            uint32_t r[32];
            tmem_ld32(o_addr + 32 * c, r);
            tmem_wait_ld();
            tmem_use(r);
            float v[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = nt > 0 ? __uint_as_float(r[i]) * inv : 0.f;
            // column 8 a + 2 n + k of panel w is value 4 a + n of group 2 w + k
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int dim = ((c & ~1) + k) * 32 + (c & 1) * 16;    // 16 values from here
              if (f32) {
                if (D == 64 && k != round) continue;
#pragma unroll
                for (int a = 0; a < 4; ++a) {
                  const int ch = (dim - round * (D / 2)) / 4 + a;
                  sts_u128(qrow + ch / 8 * 16384 + sw128_offset(trow, ch & 7),
                           make_uint4(__float_as_uint(v[8 * a + k]), __float_as_uint(v[8 * a + 2 + k]),
                                      __float_as_uint(v[8 * a + 4 + k]), __float_as_uint(v[8 * a + 6 + k])));
                }
              } else {
#pragma unroll
                for (int a = 0; a < 4; a += 2) {
                  uint32_t h[4];
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    const int j = 8 * (a + i / 2) + 4 * (i & 1) + k;
                    if (p.out_dtype == DQ_BF16) {
                      const __nv_bfloat162 t = __floats2bfloat162_rn(v[j], v[j + 2]);
                      h[i] = *(const uint32_t*)&t;
                    } else {
                      h[i] = h2_as_u32(__floats2half2_rn(v[j], v[j + 2]));
                    }
                  }
                  const int ch = dim / 8 + a / 2;
                  sts_u128(qrow + ch / 8 * 16384 + sw128_offset(trow, ch & 7), make_uint4(h[0], h[1], h[2], h[3]));
                }
              }
            }
          }
          __syncwarp();
#pragma unroll 4
          for (int i = 0; i < 32 / RPI; ++i) {
            const int tr = 32 * (warp & 3) + i * RPI + lane / LPR, lr = tile * 128 + tr, ch = lane % LPR;
            const uint4 v = lds_u128(qrow + ch / 8 * 16384 + sw128_offset(tr, ch & 7));
            if (lr >= it.rows) continue;
            const int rw = it.row0 + lr, tq = row_token(p, rw), u = rw - tq * p.group;
            const int64_t at = (int64_t)(it.first + tq) * p.out_stride + ((int64_t)it.h * p.group + u) * D;
            if (!whole)
              *(uint4*)(ws.o + (((int64_t)blockIdx.x * 2 + slot) * C::ROWS + lr) * D + round * (D / 2) + 4 * ch) = v;
            else if (f32)
              *(uint4*)((float*)p.out + at + round * (D / 2) + 4 * ch) = v;
            else
              *(uint4*)((uint16_t*)p.out + at + 8 * ch) = v;
          }
          __syncwarp();
        }
        if (live) {
          if (!whole)
            ws.ml[part] = make_float2(M, l);
          else if (p.lse)
            p.lse[q_at * p.n_q_heads + head] = l > 0.f ? (M + log2f(l)) * kLn2 : -INFINITY;
        }
        tc_fence_before();
        if (from_start && !to_end && threadIdx.x == 0)
          ws.desc[blockIdx.x] = make_int4(
              it.r, it.h, it.row0,
              ((share_of(Wk::last_unit(p, it, iu), N, U) - (int)blockIdx.x) << 1) | slot);
        if (!whole) slot = 1;
      }
    }
  } else if (warp < C::PROD) {
    // ------------------------------ decoding ------------------------------
    const int dw = warp - C::DEC0;
    // piece of the tile (four warps: one after the other), block, its half
    constexpr int PIECES = 8 / C::DW;
    const int pc0 = C::DW == 8 ? dw >> 2 : 0, blk = (dw >> 1) & 1, half = dw & 1;
    // K: lane = (token, t); odd rows take their words in swapped order, so that 8 lanes' stores meet
    // 8 different chunks.  V: lane = (a, t): tokens 2t and 2t + 1 of the half block.
    const int r4 = lane >> 2, t = lane & 3;
    const int ktok = half * 8 + r4, krow = blk * kKvBlk + ktok, vrow = blk * kKvBlk + half * 8 + 2 * t;
    const uint32_t odd = r4 & 1;
    const uint32_t k_at[2] = {sw128_offset(krow, (int)odd * 4 + t), sw128_offset(krow, (int)(odd ^ 1) * 4 + t)};
    const uint32_t k_sel[2] = {odd ? 0x3232u : 0x1010u, odd ? 0x1010u : 0x3232u};
    const uint32_t v_at[2] = {sw128_offset(vrow, r4), sw128_offset(vrow + 1, r4)};
    const uint32_t raw0 = smem_u32(smem + C::OFF_RAW) + blk * B::BYTES;
    int gt = 0;                            // decoded V's so far
    int st = pc0, st_phase = 0;            // every other stage is this warp's, or all are
    for (bool more = Wk::here(p, it, iu, share[0], share[1], ta, tb); more && ok;
         more = Wk::after(p, it, iu, share[0], share[1], ta, tb)) {
      const bool fine = EXT || is_fine(p, it);
      for (int j = ta; j < tb && ok; ++j) {
        const int tok0 = (it.t0 + (BACK ? ta + tb - 1 - j : j)) * TT;
        const bool inner = tok0 >= it.begin && tok0 <= (EXT ? it.sure : it.end) - TT;
        const int kr = SPLIT ? 2 * gt : gt;
        const int buf = gt % C::KVS, kb1 = kr % C::KVS, k2 = (kr + 1) % C::KVS;
        if (gt >= C::KVS) ok = mbar_wait(&v_empty[buf], (gt / C::KVS - 1) & 1);
        uint64_t* const k_free = SPLIT ? k_empty : v_empty;
        if (SPLIT && ok && kr >= C::KVS) ok = mbar_wait(&k_free[kb1], (kr / C::KVS - 1) & 1);
        if (fine && ok && kr + 1 >= C::KVS) ok = mbar_wait(&k_free[k2], ((kr + 1) / C::KVS - 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t kb = ks + kb1 * C::KV_BUF, kb2 = ks + k2 * C::KV_BUF, vb = vs + buf * C::KV_BUF;
#pragma unroll 1
        for (int pc = pc0; pc < pc0 + PIECES; ++pc) {
        ok = mbar_wait(&raw_full[st], st_phase);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t rb = raw0 + st * C::PIECE_B;
        // a token that no row sees may hold anything: its V scale becomes 0
        const int at0 = tok0 + pc * kPiece + vrow;
        uint32_t keep = 0;
        if (!inner)
          keep = (token_seen<EXT>(p, it, at0) ? 0x0000FFFFu : 0u) | (token_seen<EXT>(p, it, at0 + 1) ? 0xFFFF0000u : 0u);
        const uint32_t row_b = pc * kPiece * 128;          // 32 rows of 128 bytes
        auto decode = [&](auto fine_c) {
          constexpr bool FINE = decltype(fine_c)::value;
#pragma unroll
          for (int gh = 0; gh < GH; ++gh) {
            uint32_t kw[W], kd[W / 2], vw[W], vx[W / 2], vy[W / 2];
            lds_words<W>(rb + ((gh * 16 + ktok) * 4 + t) * W * 4, kw);
            if (W == 4) {
              const uint2 x = lds_u64(rb + B::OFF_KD + 2 * (ktok * G + gh * W));
              kd[0] = x.x;
              kd[W / 2 - 1] = x.y;
            } else {
              kd[0] = lds_u32(rb + B::OFF_KD + 2 * ktok * G);
            }
            lds_words<W>(rb + B::OFF_V + ((half * GH + gh) * 32 + lane) * 4 * W, vw);
#pragma unroll
            for (int k = 0; k < W / 2; ++k) {
              const int g = gh * W + 2 * k;
              vx[k] = lds_u32(rb + B::OFF_VD + ((t * G + g) * 4 + half * 2) * 2);
              vy[k] = lds_u32(rb + B::OFF_VD + ((t * G + g + 1) * 4 + half * 2) * 2);
            }
            if (!inner) {
#pragma unroll
              for (int k = 0; k < W / 2; ++k) {
                vx[k] &= keep;
                vy[k] &= keep;
              }
            }
#pragma unroll
            for (int i = 0; i < W; ++i) {
              const uint32_t word = odd ? kw[i ^ 1] : kw[i];
              const __half2 dd = u32_as_h2(__byte_perm(kd[i / 2], 0, k_sel[i & 1]));
              const uint32_t at = row_b + (gh * W + i) / 2 * (TT * 128) + k_at[i & 1];
              __half2 c[4];
              decode8(word, c);
              if (FINE) {
                const __half2 top = scale_top(dd);
                sts_u128(kb + at, times(c, top));
                sts_u128(kb2 + at, times(c, __hsub2(dd, top)));
              } else {
                sts_u128(kb + at, times(c, dd));
              }
            }
#pragma unroll
            for (int k = 0; k < W / 2; ++k) {
              const __half2 d0 = u32_as_h2(__byte_perm(vx[k], vy[k], 0x5410));
              const __half2 d1 = u32_as_h2(__byte_perm(vx[k], vy[k], 0x7632));
              const uint32_t at = vb + row_b + (gh * (W / 2) + k) * (TT * 128);
              __half2 c[4];
              decode8(vw[k], c);
              sts_u128(at + v_at[0], times(c, d0));
              decode8(vw[W / 2 + k], c);
              sts_u128(at + v_at[1], times(c, d1));
            }
          }
        };
        if (EXT || fine) decode(std::true_type());
        else decode(std::false_type());
        __syncwarp();
        if (lane == 0) mbar_arrive(&raw_empty[st]);
        st += 2 / PIECES;
        if (st >= C::RS) {
          st -= C::RS;
          st_phase ^= 1;
        }
        }
        if (!ok) break;
        fence_proxy_async_smem();
        mbar_arrive(&kv_full[buf]);
        if (!SPLIT && fine) mbar_arrive(&kv_full[k2]);
        gt += !SPLIT && fine ? 2 : 1;
      }
    }
  } else {
    if (warp == C::PROD) {
    // ------------------------------ copies ------------------------------
    const uint64_t pol = l2_evict_first_policy();
    const int shift = p.g.page_shift;
    int piece = 0, st = 0, st_phase = 0;
    for (bool more = Wk::here(p, it, iu, share[0], share[1], ta, tb); more && ok;
         more = Wk::after(p, it, iu, share[0], share[1], ta, tb)) {
      int tbase = -1, tent = 0;
      for (int j = ta; j < tb && ok; ++j) {
        const int tok0 = (it.t0 + (BACK ? ta + tb - 1 - j : j)) * TT;
        for (int pc = 0; pc < TT / kPiece && ok; ++pc) {
          if (piece >= C::RS) ok = mbar_wait(&raw_empty[st], st_phase ^ 1);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&raw_full[st], C::PIECE_B);
          __syncwarp();
          const int tok = tok0 + pc * kPiece;
          int run = 0;
          while (run < kPiece) {
            const int pg = (tok + run) >> shift;
            if (tbase < 0 || pg < tbase || pg >= tbase + 32) {
              tbase = BACK ? max(pg - 31, 0) : pg;
              const int e = tbase + lane;
              tent = e < p.max_pages ? __ldg(p.table + (int64_t)it.r * p.max_pages + e) : 0;
              if (tent < 0 || tent >= p.g.n_pages) tent = 0;
            }
            const int page = __shfl_sync(0xffffffffu, tent, pg - tbase);
            const int cnt = min(p.g.page_size, kPiece - run);
            const int off = (tok + run) & (p.g.page_size - 1);
            if (lane == 0)
              bulk_g2s(smem + C::OFF_RAW + st * C::PIECE_B + run / kKvBlk * B::BYTES,
                       p.g.pages + (int64_t)page * p.g.page_bytes + it.h * p.g.head_bytes +
                           off / kKvBlk * B::BYTES,
                       cnt / kKvBlk * B::BYTES, &raw_full[st], pol);
            run += cnt;
          }
          if (piece < C::RS) ++piece;
          if (++st == C::RS) {
            st = 0;
            st_phase ^= 1;
          }
        }
      }
    }
    // every copy has landed when the CTA ends, whichever wait ran out
    for (int s = 0; s < piece; ++s) mbar_drain(&raw_full[s], s < st ? st_phase : st_phase ^ 1);
    } else {
      // ------------------------------ products ------------------------------
      // A warp per row tile, so that neither waits for the other's softmax.  The whole warp walks the loop,
      // so that descriptors and addresses are uniform values (the instruction takes them from uniform
      // registers: from one lane's own registers each of its operands is moved first, which took 70 cycles a
      // product); one lane issues.
      constexpr uint32_t id_s = idesc_f16_f32(128, TT);
      constexpr uint32_t id_o = idesc_f16_f32(128, D) | kBRowsAlongN;
      const uint32_t tm = (uint32_t)uniform((int)tmem);
      const uint64_t q_desc = sw128_kmajor_desc(qs), k_desc = sw128_kmajor_desc(ks),
                     v_desc = sw128_mnmajor_desc(vs, TT * 128);
      const uint32_t q_lo = (uint32_t)uniform((int)(uint32_t)q_desc), k_lo = (uint32_t)uniform((int)(uint32_t)k_desc),
                     v_lo = (uint32_t)uniform((int)(uint32_t)v_desc);
      const uint32_t hi = (uint32_t)(k_desc >> 32);      // the same for all three: stride, version, swizzle
      const int i = warp - C::MMA;
      const uint32_t q_i = q_lo + (uint32_t)(i * (C::Q_TILE >> 4)), o_i = tm + (uint32_t)(i * D);
      const uint32_t s_i = tm + (uint32_t)(C::COL_S + i * 2 * TT);
      int gt = 0, ring = 0, seg = 0;         // tiles of this row tile, decoded V's of the CTA; items
      // S of this row tile's tile g, whose V is the decoded one r and its K the one kr (and the next); its buffer's last
      // weights must have been used
      auto scores = [&](int g, int r, int kr, auto fine_c) {
        constexpr bool FINE = decltype(fine_c)::value;
        const int par = g & 1, k1 = kr % C::KVS, k2 = (kr + 1) % C::KVS;
        bool good = g < 2 || mbar_wait(&pv_done[i * 2 + par], ((g - 2) >> 1) & 1);
        good = good && mbar_wait(&kv_full[r % C::KVS], (r / C::KVS) & 1);
        if (!SPLIT && FINE) good = good && mbar_wait(&kv_full[k2], ((kr + 1) / C::KVS) & 1);
        if (!__all_sync(0xffffffffu, good)) return false;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t b = k_lo + (uint32_t)(k1 * (C::KV_BUF >> 4));
          const uint32_t d = s_i + (uint32_t)(par * TT);
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            mma_ss(d, q_i + (k >> 2) * (16384 >> 4) + 2 * (k & 3), b + (k >> 2) * (TT * 128 >> 4) + 2 * (k & 3),
                   hi, id_s, k ? 1u : 0u);
          if (FINE) {
            const uint32_t b2 = k_lo + (uint32_t)(k2 * (C::KV_BUF >> 4));
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              mma_ss(d, q_i + (k >> 2) * (16384 >> 4) + 2 * (k & 3), b2 + (k >> 2) * (TT * 128 >> 4) + 2 * (k & 3),
                     hi, id_s, 1u);
          }
          tc_commit(&s_full[i * 2 + par]);
          if (SPLIT) {
            tc_commit(&k_empty[k1]);
            tc_commit(&k_empty[k2]);
          }
        }
        __syncwarp();
        return true;
      };
      auto weighted = [&](int g, int r, bool first, auto fine_c) {
        constexpr bool FINE = decltype(fine_c)::value;
        const int par = g & 1, buf = r % C::KVS;
        if (!__all_sync(0xffffffffu, mbar_wait(&p_full[i * 2 + par], (g >> 1) & 1))) return false;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t a = s_i + (uint32_t)(par * TT);
          const uint32_t b = v_lo + (uint32_t)(buf * (C::KV_BUF >> 4));
#pragma unroll
          for (int k = 0; k < TT / 16; ++k)
            mma_ts(o_i, a + 8 * k, b + k * (2048 >> 4), hi, id_o, (first && k == 0) ? 0u : 1u);
          tc_commit(&pv_done[i * 2 + par]);
          tc_commit(&v_empty[buf]);
          if (!SPLIT && FINE) tc_commit(&v_empty[(r + 1) % C::KVS]);
        }
        __syncwarp();
        return true;
      };
      // a decoded V that this row tile has no part in, and its K's
      auto pass = [&](int r) {
        const int buf = r % C::KVS;
        if (!__all_sync(0xffffffffu, mbar_wait(&kv_full[buf], (r / C::KVS) & 1))) return false;
        if (lane == 0) {
          mbar_arrive(&v_empty[buf]);
          if (SPLIT) {
            mbar_arrive(&k_empty[2 * r % C::KVS]);
            mbar_arrive(&k_empty[(2 * r + 1) % C::KVS]);
          }
        }
        return true;
      };
      for (bool more = Wk::here(p, it, iu, share[0], share[1], ta, tb); more && ok;
           more = Wk::after(p, it, iu, share[0], share[1], ta, tb)) {
        int ra, rb;
        row_tile_range<EXT>(p, it, i, ta, tb, ra, rb);
        auto item = [&](auto fine_c) {
          constexpr int KSTEP = decltype(fine_c)::value ? 2 : 1;    // decoded K's a tile takes
          constexpr int STEP = SPLIT ? 1 : KSTEP;                   // decoded V's
          // scores run two tiles ahead of the weights, or one where two tiles' buffers are not there
          constexpr int AHEAD = C::KVS >= 2 * STEP ? 2 : 1;
          const int before = uniform(BACK ? tb - rb : ra - ta) * STEP, nt = uniform(rb - ra),
                    behind = uniform(BACK ? ra - ta : tb - rb) * STEP;
          // (every tile of an instance that splits them takes two K's)
          auto k_of = [&](int r) { return SPLIT ? 2 * r : r; };
          for (int k = 0; k < before && ok; ++k) ok = pass(ring++);
          if (nt > 0 && ok) {
            ok = __all_sync(0xffffffffu, mbar_wait(&q_full[i], seg & 1));
            ++seg;
            ok = ok && scores(gt, ring, k_of(ring), fine_c);
            if (nt > 1 && AHEAD == 2) ok = ok && scores(gt + 1, ring + STEP, k_of(ring + STEP), fine_c);
            for (int k = 0; k < nt && ok; ++k, ++gt, ring += STEP) {
              ok = weighted(gt, ring, k == 0, fine_c);
              if (k + AHEAD < nt)
                ok = ok && scores(gt + AHEAD, ring + AHEAD * STEP, k_of(ring + AHEAD * STEP), fine_c);
            }
          }
          for (int k = 0; k < behind && ok; ++k) ok = pass(ring++);
        };
        if (EXT || is_fine(p, it)) item(std::true_type());
        else item(std::false_type());
      }
      // no arrival and no product is under way when the CTA ends, whichever wait ran out
      if (ok && ring > 0) mbar_wait(&v_empty[(ring - 1) % C::KVS], ((ring - 1) / C::KVS) & 1);
      if (SPLIT && ok)
        for (int k = max(2 * ring - 2, 0); k < 2 * ring; ++k) mbar_wait(&k_empty[k % C::KVS], (k / C::KVS) & 1);
      if (elect_one()) tc_commit(&drained[i]);
      __syncwarp();
      mbar_drain(&drained[i], 0);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == C::MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the partials of the items that go over several CTAs' shares: the CTAs (c, y)
// take the rows of the item that starts in CTA c's share and goes on behind it, four
// values of a row per thread.  Bound by latency (partials are in L2), so all of it runs at
// once: kJoinRows rows a thread whose loads overlap, and few registers.  (7 prompts, 12
// heads of 64: 12.5 us with a warp to a row and 87 registers, 6.6 us so.)
constexpr int kJoinRows = 2;
template <int D>
constexpr int kJoinPass = 256 / (D / 4);   // rows a CTA takes at once

template <int D>
__global__ void __launch_bounds__(256, 6) kv_tc_join_kernel(const __grid_constant__ AttnParams p) {
  using C = TcCfg<D>;
  pdl_wait();
  pdl_trigger();
  const TcWs ws = tc_ws(p.ws);
  const int4 d = __ldcg(ws.desc + blockIdx.x);
  const int follow = d.w >> 1;
  if (follow == 0) return;
  int first, all;
  const int rows = min(C::ROWS, q_rows(p, d.x, &first, &all) * p.group - d.z);
  const int c = threadIdx.x % (D / 4), row0 = blockIdx.y * (kJoinPass<D> * kJoinRows) + threadIdx.x / (D / 4);
  float m[kJoinRows], l[kJoinRows];
  float4 acc[kJoinRows];
#pragma unroll
  for (int k = 0; k < kJoinRows; ++k) {
    m[k] = kNone;
    l[k] = 0.f;
    acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
#pragma unroll 2
  for (int i = 0; i <= follow; ++i) {
    const int64_t part = ((int64_t)(blockIdx.x + i) * 2 + (i == 0 ? (d.w & 1) : 0)) * C::ROWS + row0;
#pragma unroll
    for (int k = 0; k < kJoinRows; ++k) {
      const int64_t at = part + k * kJoinPass<D>;        // (a row behind the item's last is read and not used)
      const float2 ml = __ldcg(ws.ml + at);
      const float4 x = __ldcg((const float4*)(ws.o + at * D) + c);
      const float mn = fmaxf(m[k], ml.x), f0 = ex2(m[k] - mn), f1 = ex2(ml.x - mn);
      m[k] = mn;
      l[k] = l[k] * f0 + ml.y * f1;
      acc[k].x = acc[k].x * f0 + x.x * f1;
      acc[k].y = acc[k].y * f0 + x.y * f1;
      acc[k].z = acc[k].z * f0 + x.z * f1;
      acc[k].w = acc[k].w * f0 + x.w * f1;
    }
  }
#pragma unroll
  for (int k = 0; k < kJoinRows; ++k) {
    const int in = row0 + k * kJoinPass<D>;
    if (in >= rows) continue;
    const int row = d.z + in, tokq = row_token(p, row), uq = row - tokq * p.group;
    const int64_t qrow = first + tokq;
    const int head = d.y * p.group + uq;
    const float inv = l[k] > 0.f ? 1.f / l[k] : 0.f;
    const float x[4] = {acc[k].x * inv, acc[k].y * inv, acc[k].z * inv, acc[k].w * inv};
    store_out4(p, qrow * p.out_stride + (int64_t)head * D + 4 * c, x);
    if (c == 0 && p.lse) p.lse[qrow * p.n_q_heads + head] = l[k] > 0.f ? (m[k] + log2f(l[k])) * kLn2 : -INFINITY;
  }
}

template <int D, int MODE>
int launch_tc(const AttnParams& p, int ctas, cudaStream_t s) {
  using C = TcCfg<D, MODE>;
  static bool attr[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DQ_ERR_CUDA;
  if (dev >= 64 || !attr[dev]) {
    if (cudaFuncSetAttribute(kv_tc_kernel<D, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) !=
        cudaSuccess)
      return DQ_ERR_CUDA;
    if (dev < 64) attr[dev] = true;
  }
  if (launch_pdl(kv_tc_kernel<D, MODE>, dim3(ctas), dim3(C::NTH), C::SMEM, s, 0, p) != cudaSuccess)
    return DQ_ERR_CUDA;
  if (launch_pdl(kv_tc_join_kernel<D>, dim3(ctas, C::ROWS / (kJoinPass<D> * kJoinRows)), dim3(256), 0, s, 0, p) != cudaSuccess)
    return DQ_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? DQ_OK : DQ_ERR_CUDA;
}

template <int MODE>
int launch_tc_any(const AttnParams& p, int head_dim, cudaStream_t s) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return DQ_ERR_CUDA;
  const int ctas = std::min(sms, kMaxCtas);
  if (head_dim == 64) return launch_tc<64, MODE>(p, ctas, s);
  if (head_dim == 128) return launch_tc<128, MODE>(p, ctas, s);
  return launch_tc<256, MODE>(p, ctas, s);
}

}  // namespace
}  // namespace dqmoe
