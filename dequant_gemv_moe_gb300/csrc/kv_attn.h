// kv_attn.h — what the attention kernels over the 4-bit cache share: the call's
// parameters, the workspace plan, and the arithmetic that cuts a call's work into
// shares.  That arithmetic is host code too: tests/csrc/kv_walk.cu walks every
// share of a call on the CPU.
#pragma once

#include "kv.cuh"

namespace dqmoe {

struct AttnParams {
  KvGeom g;
  const void* q;
  int64_t q_stride;
  int q_dtype, n_q_heads, group, T, B;
  uint32_t group_inv;          // floor(2^32 / group), 2^32 - 1 for 1
  const int32_t* q_start;
  const int32_t* kv_len;
  const int32_t* table;
  int max_pages, max_q_len;
  float scale;
  int causal, window;
  void* out;
  int out_dtype;
  int64_t out_stride;
  float* lse;
  uint8_t* ws;
  int rows_above, rows_upto;   // the kernel looks after requests with rows_above < rows <= rows_upto
  int alone;                   // streaming: 0, or every row tile has a CTA of its own, and a request this many
  // what the kernels with EXT read besides (dq_kv_scores)
  float cap;                   // of a score in units of log 2, 0: none
  float cap_inv;               // its inverse
  int cap_small;               // so small that tanh's absolute error may be taken times it (kv_attn.cu)
  float2 cap_c[7];             // times tanh's polynomial, every coefficient twice (soft_cap)
  const float* slopes;         // per query head, or null
  const int32_t* prefix;       // per request, or null
  const int32_t* first_pos;    // per row of q, or null
};

// The kernels' instances: plain, masks alone, capped scores (many rows: caps up to 100), biased ones, anything.
enum ScoreMode { kPlain, kMasks, kCaps, kBias, kAnyScores };

// few rows per K/V head (kv_attn_stream.cuh); ext: scores and masks other than the plain ones
size_t kv_stream_workspace();
int launch_kv_stream(const AttnParams& p, int head_dim, bool ext, cudaStream_t s);
// many rows (kv_attn_tc.cuh)
size_t kv_tc_workspace();
int launch_kv_tc(const AttnParams& p, int head_dim, bool ext, cudaStream_t s);

#define DQ_HD __host__ __device__ __forceinline__

DQ_HD int load_length(const int32_t* p) {
#ifdef __CUDA_ARCH__
  return __ldg(p);
#else
  return *p;
#endif
}

inline uint32_t group_inverse(int group) {
  return group == 1 ? 0xFFFFFFFFu : (uint32_t)((1ULL << 32) / (uint32_t)group);
}

// The token of row (token * group + head).  floor(row * floor(2^32 / g) / 2^32) is row / g or one less.
DQ_HD int row_token(const AttnParams& p, int row) {
  const int t = (int)((uint64_t)(uint32_t)row * p.group_inv >> 32);
  return row - t * p.group >= p.group ? t + 1 : t;
}

// The first position that a row at `pos` (below 0 where the cache starts behind it) sees.  The window may be
// any positive int: pos - window is formed only where it is not negative.
DQ_HD int first_seen(const AttnParams& p, int pos) {
  return p.window > 0 && pos >= p.window ? pos - p.window + 1 : 0;
}

// The entry of a request's row of the block table that lists the token `ahead` tokens behind the start of a
// tile (ahead below 1024), or -1.  A token behind the last that a table can list may pass the largest int.
DQ_HD int listed_page(const AttnParams& p, int tile, int tile_tokens, int ahead) {
  const uint32_t page = ((uint32_t)tile * tile_tokens + ahead) >> p.g.page_shift;
  return page < (uint32_t)p.max_pages ? (int)page : -1;
}

// the length of request r as the kernels read it
DQ_HD int kv_length(const AttnParams& p, int r) {
  const int64_t cap = (int64_t)p.max_pages << p.g.page_shift;
  return (int)min((int64_t)max(load_length(p.kv_len + r), 0), cap);
}
// The rows of request r that are looked after, and how many it has in all (at least as many: rows past
// max_q_len and past T are left out, the others stand where they stand).
DQ_HD int q_rows(const AttnParams& p, int r, int* first, int* all) {
  const int a = load_length(p.q_start + r), b = load_length(p.q_start + r + 1);
  *first = a;
  *all = a >= 0 && b > a ? b - a : 0;
  // memory-safe whatever q_start holds
  return a < 0 ? 0 : max(0, min(min(b, p.T) - a, p.max_q_len));
}
// A row at `pos` sees the positions below this one; of a request with a prefix, those in it too.
DQ_HD int seen_end(const AttnParams& p, int len, int pos, int prefix = 0) {
  return p.causal ? max(0, min(len, max(pos + 1, prefix))) : len;
}
// The prefix of request r, and the first position that row `row` of q may see.
DQ_HD int prefix_of(const AttnParams& p, int r) { return p.prefix ? max(load_length(p.prefix + r), 0) : 0; }
DQ_HD int row_first(const AttnParams& p, int row) { return p.first_pos ? max(load_length(p.first_pos + row), 0) : 0; }


// One row tile of a request and the tokens that its rows may see.
struct Item {
  int r, h, row0, rows;        // request, K/V head, first row (token * group + head), rows
  int len, qlen, first;        // kv length, tokens of the request, its first row of q
  int shift;                   // position of its first token
  int begin, end;              // tokens that some row sees
  int t0, tiles;               // first tile, tiles (at least one)
  int prefix;                  // EXT: the request's
  int sure;                    // EXT: the tokens from begin up to here are seen by its first row
};

// Whether some row of the item sees token a.  Of a window or a prefix every token of [begin, end) is seen; rows with
// first positions may see nothing, between two documents or at the end, and a token that its own row does not see
// is seen by none: the rows in front of it do not reach it, those behind it start later.
template <bool EXT>
DQ_HD bool token_seen(const AttnParams& p, const Item& it, int a) {
  if (a < it.begin || a >= it.end) return false;
  return !EXT || a < it.sure || row_first(p, it.first + (a - it.shift)) <= a;
}

// A call's work as one line of units: (request, row tile, K/V head, tile of
// TILE tokens), the tokens fastest.  An item (all of them but the tokens) takes
// OV units before its tiles: what starting and ending one costs.  A tile takes one
// unit, or WEIGHT::of(item).  EXT: rows may have a prefix and a first position.
struct UnitWeight {
  DQ_HD static int of(const AttnParams&, const Item&) { return 1; }
};
template <int ROWS, int TILE, int OV, typename WEIGHT = UnitWeight, bool EXT = false>
struct Walk {
  DQ_HD static int cost(const AttnParams& p, const Item& it) {
    return it.tiles * WEIGHT::of(p, it) + OV;
  }
  DQ_HD static void range(const AttnParams& p, Item& it) {
    it.rows = min(ROWS, it.qlen * p.group - it.row0);
    const int lo = it.shift + row_token(p, it.row0), hi = it.shift + row_token(p, it.row0 + it.rows - 1);
    it.end = seen_end(p, it.len, hi, EXT ? it.prefix : 0);
    it.begin = first_seen(p, lo);
    if (EXT) {
      // first positions ascend within a request: the first row's is the least
      it.begin = min(max(it.begin, row_first(p, it.first + lo - it.shift)), it.end);
      it.sure = p.first_pos ? min(seen_end(p, it.len, lo, it.prefix), it.end) : it.end;
    }
    it.t0 = it.begin / TILE;
    it.tiles = it.end > it.begin ? (it.end - 1) / TILE + 1 - it.t0 : 1;
  }
  // the request's rows of q if this kernel looks after it, else 0
  DQ_HD static int tokens(const AttnParams& p, int r, int* first, int* all) {
    const int n = q_rows(p, r, first, all);
    const int64_t rows = (int64_t)n * p.group;
    return rows > p.rows_above && rows <= p.rows_upto ? n : 0;
  }
  // Request r.  `known`: rows, length, first row of q and first position of every request, in shared
  // memory, or null.
  DQ_HD static void request(const AttnParams& p, int r, Item& it, const int* known = nullptr) {
    it.r = r;
    if (known) {
      it.qlen = known[4 * r];
      it.len = known[4 * r + 1];
      it.first = known[4 * r + 2];
      it.shift = known[4 * r + 3];
    } else {
      int all;
      it.qlen = tokens(p, r, &it.first, &all);
      it.len = kv_length(p, r);
      it.shift = it.len - all;
    }
    if (EXT) it.prefix = prefix_of(p, r);
  }
  // Units of the row tiles k, k + step, .. of the request in `it` (one head's).
  DQ_HD static int64_t row_tile_units(const AttnParams& p, Item& it, int k, int step) {
    int64_t u = 0;
    for (it.row0 = k * ROWS; it.row0 < it.qlen * p.group; it.row0 += step * ROWS) {
      range(p, it);
      u += cost(p, it);
    }
    return u;
  }
  DQ_HD static void next(const AttnParams& p, Item& it) {
    if (++it.h < p.g.heads) return;
    it.h = 0;
    it.row0 += ROWS;
    if (it.row0 >= it.qlen * p.group) {
      it.row0 = 0;
      int all;
      do {
        if (++it.r >= p.B) return;       // past the last unit: never read
        it.qlen = tokens(p, it.r, &it.first, &all);
      } while (it.qlen == 0);
      it.len = kv_length(p, it.r);
      it.shift = it.len - all;
      if (EXT) it.prefix = prefix_of(p, it.r);
    }
    range(p, it);
  }
  // Row tile i of all (request, row tile, K/V head) where every request takes the place of `per` row tiles.
  DQ_HD static bool nth(const AttnParams& p, int i, int per, Item& it) {
    const int k = i / p.g.heads;
    it.h = i - k * p.g.heads;
    const int r = k / per;
    it.row0 = (k - r * per) * ROWS;
    request(p, r, it);
    if (it.row0 >= it.qlen * p.group) return false;
    range(p, it);
    return true;
  }
  // The units before every of the block's NTH chunks of requests, pre[NTH] in all
  // (every thread of the block calls it).  The warps' sums lie behind them: NTH + 1 + NTH / 32
  // entries, in the caller's dynamic shared memory (static shared memory in front of it would
  // shift it off the alignment that swizzled operands need).
  // `known` (4 NTH ints, may be null) is filled where every thread has one request at most.
  template <int NTH>
  __device__ __forceinline__ static void sum_units(const AttnParams& p, int64_t* pre, int* known = nullptr) {
    int64_t* wsum = pre + NTH + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int chunk = (p.B + NTH - 1) / NTH;
    Item it;
    int64_t u = 0;
    for (int i = 0; i < chunk; ++i) {
      const int r = threadIdx.x * chunk + i;
      if (r < p.B) request(p, r, it);
      else it.qlen = it.len = it.first = it.shift = it.prefix = 0;
      // a request of few row tiles by its thread, one of many by the warp
      const bool few = (int64_t)it.qlen * p.group <= 8 * ROWS;
      if (few) u += row_tile_units(p, it, 0, 1) * p.g.heads;
      for (uint32_t m = __ballot_sync(0xffffffffu, !few); m; m &= m - 1) {
        const int src = __ffs(m) - 1;
        Item x;
        x.qlen = __shfl_sync(0xffffffffu, it.qlen, src);
        x.len = __shfl_sync(0xffffffffu, it.len, src);
        x.shift = __shfl_sync(0xffffffffu, it.shift, src);
        if (EXT) {
          x.first = __shfl_sync(0xffffffffu, it.first, src);
          x.prefix = __shfl_sync(0xffffffffu, it.prefix, src);
        }
        int64_t n = row_tile_units(p, x, lane, 32);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
        if (lane == src) u += n * p.g.heads;
      }
    }
    if (known && chunk == 1 && (int)threadIdx.x < p.B) {
      known[4 * threadIdx.x] = it.qlen;
      known[4 * threadIdx.x + 1] = it.len;
      known[4 * threadIdx.x + 2] = it.first;
      known[4 * threadIdx.x + 3] = it.shift;
    }
    int64_t inc = u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    int64_t base = 0;
    for (int i = 0; i < warp; ++i) base += wsum[i];
    pre[threadIdx.x] = base + inc - u;
    if (threadIdx.x == NTH - 1) pre[NTH] = base + inc;
    __syncthreads();
  }
  // The item that unit u lies in, and the unit at which it starts (a whole warp calls it).
  template <int NTH>
  __device__ __forceinline__ static int64_t seek(const AttnParams& p, const int64_t* pre, int64_t u,
                                                 Item& it, const int* known = nullptr) {
    const int chunk = (p.B + NTH - 1) / NTH;
    // the last chunk with pre <= u: 32 at a time, then among 32
    constexpr int STEP = (NTH + 31) / 32;
    const int lane = threadIdx.x & 31;
    const int big = 31 - __clz(__ballot_sync(0xffffffffu, pre[min(lane * STEP, NTH)] <= u));
    const int at = big * STEP + lane;
    const int small = 31 - __clz(__ballot_sync(0xffffffffu, lane < STEP && at < NTH && pre[min(at, NTH)] <= u));
    const int c = big * STEP + small;
    int64_t iu = pre[c];
    // the request, 32 row tiles at a time; then the row tile and the head (a row tile's heads cost the same)
    for (int r = c * chunk;; ++r) {
      request(p, r, it, chunk == 1 ? known : nullptr);
      for (int row0 = 0; row0 < it.qlen * p.group; row0 += 32 * ROWS) {
        it.row0 = row0 + lane * ROWS;
        int64_t n = 0;
        if (it.row0 < it.qlen * p.group) {
          range(p, it);
          n = (int64_t)cost(p, it) * p.g.heads;
        }
        int64_t inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += v;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, u < iu + inc);
        if (past) {
          const int l = __ffs(past) - 1;
          iu += __shfl_sync(0xffffffffu, inc - n, l);
          it.row0 = row0 + l * ROWS;
          range(p, it);
          const int each = cost(p, it);
          // the heads in front of u (of 1024 at most, whose units may pass 32 bits), 32 at a time
          int h = 31 - __clz(__ballot_sync(0xffffffffu, (int64_t)(32 * lane) * each <= u - iu));
          h = 32 * h + 31 - __clz(__ballot_sync(0xffffffffu, (int64_t)(32 * h + lane) * each <= u - iu));
          it.h = h;
          return iu + (int64_t)it.h * each;
        }
        iu += __shfl_sync(0xffffffffu, inc, 31);
      }
    }
  }
  // The tiles [a, b) of the item at unit iu that lie in the share [u0, u1); none: on to the next
  // item that has some.  False: the share holds no more.
  DQ_HD static bool here(const AttnParams& p, Item& it, int64_t& iu, int64_t u0, int64_t u1, int& a,
                         int& b) {
    for (;;) {
      // tile t lies in the share that its first unit lies in
      const int w = WEIGHT::of(p, it);
      const int64_t lo = max(u0 - iu - OV, (int64_t)0), hi = min(u1 - iu - OV, (int64_t)it.tiles * w);
      a = (int)lo;
      b = (int)hi;
      if (w > 1) {
        a = (a + w - 1) / w;
        b = b > 0 ? (b + w - 1) / w : 0;
      }
      if (b > a) return true;
      iu += cost(p, it);
      if (iu >= u1) return false;
      next(p, it);
    }
  }
  DQ_HD static bool after(const AttnParams& p, Item& it, int64_t& iu, int64_t u0, int64_t u1, int& a,
                          int& b) {
    iu += cost(p, it);
    if (iu >= u1) return false;
    next(p, it);
    return here(p, it, iu, u0, u1, a, b);
  }
  // the first unit of the item's last tile
  DQ_HD static int64_t last_unit(const AttnParams& p, const Item& it, int64_t iu) {
    return iu + OV + (int64_t)(it.tiles - 1) * WEIGHT::of(p, it);
  }
};

// The line of U units is cut into N <= U equal shares: share w is [floor(U w / N), floor(U (w + 1) / N)),
// and unit u lies in share ceil((u + 1) N / U) - 1.
DQ_HD int64_t share_start(int64_t U, int N, int w) {
  if (U < (1LL << 31)) {                   // 32-bit divisions: U w / N = (U / N) w + (U mod N) w / N
    const uint32_t q = (uint32_t)U / (uint32_t)N, r = (uint32_t)U - q * (uint32_t)N;
    return (int64_t)q * w + r * (uint32_t)w / (uint32_t)N;
  }
  return U * w / N;
}
DQ_HD int share_of(int64_t u, int N, int64_t U) {
  return (int)(((u + 1) * N + U - 1) / U - 1);
}

// Few rows: 8 rows and tiles of 32 tokens, a tile's worth for starting and ending an item.
template <bool EXT>
using StreamWalkOf = Walk<8, 32, 1, UnitWeight, EXT>;
using StreamWalk = StreamWalkOf<false>;

// Rounding K to fp16 moves a score by about 2^-12 of itself.  Over many tokens that averages out, but where
// a row sees few of them its lse and weights carry it (rel. 4e-5 in the lse of a 17-token prompt).  There K is
// taken as two exact fp16 products, with the scale's top 8 bits and with the rest, and Q K^T as two sums; the
// second one takes the K half of a second decoded buffer.
// (7 prompts up to 3001 tokens, 12 heads of 64: 142 us so, 136 with one product everywhere, 180 with two.
// The long chunk, none of whose rows sees that few: 935 us so, 1856 with two products.)
constexpr int kFineTokens = 1024;
DQ_HD bool is_fine(const AttnParams& p, const Item& it) {
  return (p.window > 0 ? min(p.window, it.end) : it.end) <= kFineTokens;
}

// Two sums for a score, and half the decoded buffers: such a tile takes about twice as long.  (EXT: all tiles are such.)
template <bool EXT>
struct TcWeightOf {
  DQ_HD static int of(const AttnParams& p, const Item& it) { return !EXT && is_fine(p, it) ? 2 : 1; }
};

// Many rows: row tiles of 128 rows, two a CTA (one for head_dim 256), and tiles of 64 tokens; starting and
// ending an item takes as long as four of them, or eight where scores are masked, capped or biased (7 prompts of
// documents up to 3001 tokens, 12 heads of 64: 93 us with four, 90 with six, 87 with eight; 32 heads of 128 on 8: 275,
// 246, 238, with a bias and no masks 576, 508, 458, capped at 50 336, 320, 329).
constexpr int kTcTile = 64;
template <int D>
constexpr int kTcRowTiles = D == 256 ? 1 : 2;
template <int D, bool EXT = false>
using TcWalk = Walk<128 * kTcRowTiles<D>, kTcTile, EXT ? 8 : 4, TcWeightOf<EXT>, EXT>;
// a line of U units is cut into this many shares, of two units at least: none inside an item is without a tile
DQ_HD int tc_shares(int ctas, int64_t U) { return (int)min((int64_t)ctas, U / 2); }

// The tiles [a, b) of the item's [ta, tb) that row tile i sees anything of: a causal item's first row
// tile is done before its last one, a windowed item's last one starts behind its first one (with one head
// to a K/V head two tiles behind, which may be behind tb), and rows behind the item's end see nothing.
// ta <= a <= b <= tb, so that the tiles before, in and behind are the tb - ta that the share decodes.
template <bool EXT = false>
DQ_HD void row_tile_range(const AttnParams& p, const Item& it, int i, int ta, int tb, int& a, int& b) {
  a = b = ta;
  const int last = min(it.rows, 128 * i + 128) - 1;
  if (last < 128 * i) return;
  const int end = seen_end(p, it.len, it.shift + row_token(p, it.row0 + last), EXT ? it.prefix : 0);
  const int tok = row_token(p, it.row0 + 128 * i);
  int begin = first_seen(p, it.shift + tok);
  if (EXT) begin = max(begin, row_first(p, it.first + tok));
  if (end <= begin) return;
  a = min(tb, max(ta, begin / kTcTile - it.t0));
  b = max(a, min(tb, (end - 1) / kTcTile + 1 - it.t0));
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

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLeastScale = 1.17549435e-38f;   // of a row's scores: times 0, a masked score would be NaN
constexpr float kNone = -1e30f;           // the running maximum of a row that has seen nothing
constexpr float kLn2 = 0.693147180559945309f, kLog2e = 1.44269504088896341f;

__device__ __forceinline__ float rcp_ftz(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Capped scores in units of log 2 from u = score / cap.  tanh(u) / u is a polynomial in u^2 of degree 6 where
// |u| <= 1 (its Chebyshev interpolation: 2.5e-7 of itself, fp32's roundings included); beyond,
// tanh(|u|) = 1 - 2 / (1 + e^2|u|), whose terms do not cancel there.
//
// Eight scores at a time: chains of packed steps keep the pipe busy, and a coefficient is fetched once.
template <int N>
__device__ __forceinline__ void soft_cap(const AttnParams& p, float2 (&u)[N]) {
  float2 y[N], r[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    y[i] = fmul2(u[i], u[i]);
    r[i] = p.cap_c[6];
  }
#pragma unroll
  for (int k = 5; k >= 0; --k)
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = ffma2(r[i], y[i], p.cap_c[k]);
#pragma unroll
  for (int i = 0; i < N; ++i) u[i] = fmul2(r[i], u[i]);
}
// The same for any u.
template <int N>
__device__ __forceinline__ void soft_cap_far(const AttnParams& p, float2 (&u)[N]) {
  float2 near[N];
#pragma unroll
  for (int i = 0; i < N; ++i) near[i] = u[i];
  soft_cap(p, near);
  auto far = [&](float x) {
    return copysignf(p.cap - 2.f * p.cap * rcp_ftz(1.f + ex2(fabsf(x) * (2.f * kLog2e))), x);
  };
#pragma unroll
  for (int i = 0; i < N; ++i) {
    u[i].x = fabsf(u[i].x) > 1.f ? far(u[i].x) : near[i].x;
    u[i].y = fabsf(u[i].y) > 1.f ? far(u[i].y) : near[i].y;
  }
}


template <int DT>
__device__ __forceinline__ void store_dims4(void* out, int64_t at, const float (&x)[4]) {
  if (DT == DQ_F32) {
    *(float4*)((float*)out + at) = make_float4(x[0], x[1], x[2], x[3]);
  } else if (DT == DQ_F16) {
    *(uint2*)((__half*)out + at) = make_uint2(h2_as_u32(__floats2half2_rn(x[0], x[1])),
                                              h2_as_u32(__floats2half2_rn(x[2], x[3])));
  } else {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    *(uint2*)((__nv_bfloat16*)out + at) = make_uint2(*(const uint32_t*)&a, *(const uint32_t*)&b);
  }
}
__device__ __forceinline__ void store_out4(const AttnParams& p, int64_t at, const float (&x)[4]) {
  if (p.out_dtype == DQ_BF16) store_dims4<DQ_BF16>(p.out, at, x);
  else if (p.out_dtype == DQ_F16) store_dims4<DQ_F16>(p.out, at, x);
  else store_dims4<DQ_F32>(p.out, at, x);
}

// A joined row: a warp's lane holds values D / 32 * lane.. of the weighted sum, all lanes the maximum
// and the sum of the weights.  `row` is the row (token * group + head) of request r and K/V head h.
template <int D>
__device__ __forceinline__ void store_row(const AttnParams& p, int r, int h, int row, int lane,
                                          const float (&acc)[D / 32], float m, float l) {
  constexpr int V = D / 32;
  const float inv = l > 0.f ? 1.f / l : 0.f;
  const int tokq = row_token(p, row), uq = row - tokq * p.group;
  const int64_t qrow = __ldg(p.q_start + r) + tokq;
  const int head = h * p.group + uq;
  const int64_t base = qrow * p.out_stride + (int64_t)head * D + lane * V;
#pragma unroll
  for (int v = 0; v < V; v += 4) {
    float x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = acc[V < 4 ? k & 1 : v + k] * inv;
    if (V < 4) {                           // 64 values: two lanes' pairs make one four
      x[2] = __shfl_down_sync(0xffffffffu, x[0], 1);
      x[3] = __shfl_down_sync(0xffffffffu, x[1], 1);
    }
    if (V >= 4 || (lane & 1) == 0) store_out4(p, base + v, x);
  }
  if (lane == 0 && p.lse)
    p.lse[qrow * p.n_q_heads + head] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

}  // namespace dqmoe
