// kv_walk_ext.cu — the work sharing of the attention kernels for requests with prefixes and rows with first
// positions, on the CPU with the kernels' own arithmetic (kv_attn.h), held to the definition in 64 bits:
//   * the tiles of every item lie in the shares once each, in order;
//   * an item's tokens are those that its rows see, a 128-row tile's tiles [ra, rb) lie in its share's and hold
//     every token that its rows see;
//   * whatever the arrays hold (descending first positions, values out of range), an item's tokens are
//     tokens of the cache and a row tile's tiles are tiles of the share.
// Built with traps on signed overflow.
//   kv_walk_ext MODE SEED CALLS     MODE: sorted, wild
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <random>
#include <vector>

#include "../../dequant_gemv_moe_gb300/csrc/kv_attn.h"

using namespace dqmoe;

namespace {

using Rng = std::mt19937_64;
int upto(Rng& g, int lo, int hi) { return lo + (int)(g() % (uint64_t)((int64_t)hi - lo + 1)); }

struct Call {
  int heads, group, causal, window, ctas, page_size, max_pages;
  std::vector<int32_t> rows, kv, prefix, first, start;
  bool sorted;
};

#define CHECK(cond, ...)                                                                                     \
  do {                                                                                                       \
    if (!(cond)) {                                                                                           \
      fprintf(stderr, "%s fails: ", #cond);                                                                  \
      fprintf(stderr, __VA_ARGS__);                                                                          \
      fprintf(stderr, "\n  %d heads, group %d, causal %d, window %d\n", c.heads, c.group, c.causal, c.window); \
      exit(1);                                                                                               \
    }                                                                                                        \
  } while (0)

Call draw(Rng& g, bool sorted, int most_rows) {
  static const int groups[] = {1, 1, 2, 3, 4, 5, 7, 8, 16};
  Call c;
  c.sorted = sorted;
  c.heads = upto(g, 1, 6);
  c.group = groups[g() % 9];
  c.causal = g() % 6 != 0;
  c.window = g() % 2 ? 0 : upto(g, 1, 3000);
  c.ctas = upto(g, 0, 3) ? 152 : upto(g, 1, 160);
  c.page_size = 16 << upto(g, 0, 4);
  const int n = upto(g, 1, 6);
  c.start.push_back(0);
  int most = 1;
  for (int i = 0; i < n; ++i) {
    const int rows = g() % 6 == 0 && i ? 0 : upto(g, 1, most_rows);
    const int kv = g() % 5 == 0 ? upto(g, 0, rows + 50) : rows + (g() % 2 ? 0 : upto(g, 0, 6000));
    c.rows.push_back(rows);
    c.kv.push_back(kv);
    most = std::max(most, kv);
    c.prefix.push_back(!sorted && g() % 3 == 0 ? (int)(uint32_t)g() : g() % 2 ? 0 : upto(g, 0, kv + 10));
    int at = 0;
    for (int k = 0; k < rows; ++k) {
      if (g() % 100 == 0) at = sorted ? std::max(at, kv - rows + k + (g() % 20 == 0 ? 5 : 0)) : upto(g, -5, kv + 9);
      c.first.push_back(!sorted && g() % 50 == 0 ? (int)(uint32_t)g() : at);
    }
    c.start.push_back(c.start.back() + rows);
  }
  c.max_pages = most / c.page_size + 1;
  return c;
}

AttnParams params(const Call& c) {
  AttnParams p;
  memset(&p, 0, sizeof p);
  p.g.heads = c.heads;
  p.g.page_size = c.page_size;
  while ((1 << p.g.page_shift) < c.page_size) ++p.g.page_shift;
  p.group = c.group;
  p.group_inv = group_inverse(c.group);
  p.n_q_heads = c.heads * c.group;
  p.T = c.start.back();
  p.B = (int)c.rows.size();
  p.q_start = c.start.data();
  p.kv_len = c.kv.data();
  p.max_pages = c.max_pages;
  p.max_q_len = *std::max_element(c.rows.begin(), c.rows.end());
  p.causal = c.causal;
  p.window = c.window;
  p.prefix = c.causal ? c.prefix.data() : nullptr;
  p.first_pos = c.first.data();
  return p;
}

// What row `tok` of request r sees, from the definition; empty: lo >= hi.
void seen(const Call& c, int r, int tok, int64_t* lo, int64_t* hi) {
  const int64_t len = c.kv[r], pos = len - c.rows[r] + tok;
  *hi = c.causal ? std::min(len, std::max<int64_t>(pos + 1, c.prefix[r])) : len;
  *lo = std::max<int64_t>(c.window > 0 ? std::max<int64_t>(0, pos - c.window + 1) : 0, c.first[c.start[r] + tok]);
}
void seen_any(const Call& c, int r, int a, int b, int64_t* lo, int64_t* hi) {
  *lo = INT64_MAX;
  *hi = INT64_MIN;
  for (int t = a / c.group; t <= b / c.group; ++t) {
    int64_t l, h;
    seen(c, r, t, &l, &h);
    if (l >= h) continue;
    *lo = std::min(*lo, l);
    *hi = std::max(*hi, h);
  }
}

template <typename Wk, typename F>
void check(const Call& c, const AttnParams& p, int tile, int shares_of, F part) {
  std::vector<Item> items;
  std::vector<int64_t> at;
  int64_t U = 0;
  Item it;
  for (int r = 0; r < p.B; ++r) {
    Wk::request(p, r, it);
    if (it.qlen == 0) continue;
    for (int row0 = 0; row0 < it.qlen * p.group; row0 += it.rows) {
      it.row0 = row0;
      Wk::range(p, it);
      CHECK(0 <= it.begin && it.begin <= it.end && it.end <= std::max(0, it.len), "[%d, %d) of %d", it.begin, it.end, it.len);
      CHECK(it.tiles >= 1 && (int64_t)(it.t0 + it.tiles - 1) * tile <= std::max(it.len, 0), "tiles %d + %d", it.t0, it.tiles);
      int64_t lo, hi;
      seen_any(c, r, row0, row0 + it.rows - 1, &lo, &hi);
      if (c.sorted && lo < hi)
        CHECK(it.begin <= lo && hi <= it.end && it.t0 <= lo / tile && it.t0 + it.tiles > (hi - 1) / tile,
              "request %d, row %d: [%d, %d) for [%lld, %lld)", r, row0, it.begin, it.end, (long long)lo, (long long)hi);
      for (int h = 0; h < p.g.heads; ++h) {
        it.h = h;
        items.push_back(it);
        at.push_back(U);
        U += Wk::cost(p, it);
      }
    }
  }
  if (U == 0) return;
  const int N = shares_of ? (int)std::min<int64_t>(shares_of, U) : tc_shares(c.ctas, U);
  if (N < 1) return;
  std::vector<int> done(items.size(), 0);
  size_t i0 = 0;
  for (int w = 0; w < N; ++w) {
    const int64_t u0 = share_start(U, N, w), u1 = share_start(U, N, w + 1);
    while (i0 + 1 < items.size() && at[i0 + 1] <= u0) ++i0;
    Item x = items[i0];
    int64_t iu = at[i0];
    int a, b;
    size_t i = i0;
    for (bool more = Wk::here(p, x, iu, u0, u1, a, b); more; more = Wk::after(p, x, iu, u0, u1, a, b)) {
      while (at[i] < iu) ++i;
      CHECK(at[i] == iu && items[i].r == x.r && items[i].h == x.h && items[i].row0 == x.row0 && items[i].sure == x.sure &&
                items[i].prefix == x.prefix && items[i].tiles == x.tiles, "share %d: item %zu", w, i);
      CHECK(a == done[i] && a < b && b <= x.tiles, "share %d, item %zu: [%d, %d) after %d", w, i, a, b, done[i]);
      done[i] = b;
      if (b == x.tiles) CHECK(share_of(Wk::last_unit(p, x, iu), N, U) == w, "share %d ends item %zu", w, i);
      part(x, a, b);
    }
  }
  for (size_t i = 0; i < items.size(); ++i) CHECK(done[i] == items[i].tiles, "item %zu: %d of %d", i, done[i], items[i].tiles);
}

template <int D>
void many(const Call& c) {
  AttnParams p = params(c);
  p.rows_upto = 1 << 30;
  check<TcWalk<D, true>>(c, p, kTcTile, 0, [&](const Item& it, int ta, int tb) {
    for (int i = 0; i < kTcRowTiles<D>; ++i) {
      int ra, rb;
      row_tile_range<true>(p, it, i, ta, tb, ra, rb);
      CHECK(ta <= ra && ra <= rb && rb <= tb, "row tile %d: [%d, %d) of [%d, %d)", i, ra, rb, ta, tb);
      const int last = std::min(it.rows, 128 * i + 128) - 1;
      if (last < 128 * i || !c.sorted) continue;
      int64_t lo, hi;
      seen_any(c, it.r, it.row0 + 128 * i, it.row0 + last, &lo, &hi);
      if (lo >= hi) continue;
      const int64_t a = std::max<int64_t>(lo / kTcTile - it.t0, ta), b = std::min<int64_t>((hi - 1) / kTcTile + 1 - it.t0, tb);
      CHECK(a >= b || (ra <= a && b <= rb), "row tile %d takes [%d, %d), needs [%lld, %lld)", i, ra, rb, (long long)a,
            (long long)b);
    }
  });
}

}  // namespace

int main(int argc, char** argv) {
  if (argc != 4) return 2;
  Rng g(strtoull(argv[2], nullptr, 10));
  for (int i = atoi(argv[3]); i > 0; --i) {
    const bool sorted = !strcmp(argv[1], "sorted");
    Call c = draw(g, sorted, 1500);
    many<64>(c);
    many<256>(c);
    c = draw(g, sorted, 8);
    AttnParams p = params(c);
    p.rows_upto = 64;
    check<StreamWalkOf<true>>(c, p, 32, c.ctas * 12, [](const Item&, int, int) {});
  }
  return 0;
}
