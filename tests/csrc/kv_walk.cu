// kv_walk.cu — the attention kernels' work sharing on the CPU: every share of a
// call is walked as the kernels walk it, with their own arithmetic (kv_attn.h), and
// held to what attention's definition says in 64 bits.
//   * the tiles of every item lie in the shares once each, in order;
//   * of the tiles [ta, tb) that a share holds of an item, a 128-row tile takes
//     [ra, rb) with ta <= ra <= rb <= tb (the decoded tiles before, in and behind it are
//     then those that the share decodes: none is waited for that nobody decodes);
//   * no token that a row sees lies outside its row tile's [ra, rb).
// Built with traps on signed overflow.
//   kv_walk MODE SEED CALLS   (MODE: a function below)
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <random>
#include <vector>

#include "../../dequant_gemv_moe_gb300/csrc/kv_attn.h"

using namespace dqmoe;

namespace {

struct Call {
  int heads, group, page_size, max_pages, causal, window, ctas;
  std::vector<int> rows, kv;               // of each request
  int most = 0, behind = 0;                // max_q_len if not the largest of rows; rows of q that are missing at its end
};

#define CHECK(cond, ...)                                                              \
  do {                                                                                \
    if (!(cond)) {                                                                    \
      fprintf(stderr, "%s fails: ", #cond);                                           \
      fprintf(stderr, __VA_ARGS__);                                                   \
      fprintf(stderr, "\n  %d heads, group %d, causal %d, window %d, %d CTAs; rows, kv:", c.heads, c.group, \
              c.causal, c.window, c.ctas);                                            \
      for (size_t i_ = 0; i_ < c.rows.size() && i_ < 8; ++i_)                         \
        fprintf(stderr, " (%d, %d)", c.rows[i_], c.kv[i_]);                           \
      fprintf(stderr, "\n");                                                          \
      exit(1);                                                                        \
    }                                                                                 \
  } while (0)

struct Params {
  AttnParams p;
  std::vector<int32_t> start, kv;
  explicit Params(const Call& c) {
    memset(&p, 0, sizeof p);
    start.push_back(0);
    for (int n : c.rows) start.push_back(start.back() + n);
    kv.assign(c.kv.begin(), c.kv.end());
    p.g.heads = c.heads;
    p.g.page_size = c.page_size;
    while ((1 << p.g.page_shift) < c.page_size) ++p.g.page_shift;
    p.group = c.group;
    p.group_inv = group_inverse(c.group);
    p.n_q_heads = c.heads * c.group;
    p.T = start.back() - c.behind;
    p.B = (int)c.rows.size();
    p.q_start = start.data();
    p.kv_len = kv.data();
    p.max_pages = c.max_pages;
    p.max_q_len = c.most ? c.most : *std::max_element(c.rows.begin(), c.rows.end());
    p.causal = c.causal;
    p.window = c.window;
  }
};

// The tokens that rows [a, b] of request r see any of, from the definition: [lo, hi).
void seen(const Call& c, int r, int a, int b, int64_t* lo, int64_t* hi) {
  const int64_t len = c.kv[r], shift = len - c.rows[r];
  const int64_t pa = shift + a / c.group, pb = shift + b / c.group;
  *hi = c.causal ? std::min(len, pb + 1) : len;
  *lo = c.window > 0 ? std::max<int64_t>(0, pa - c.window + 1) : 0;
}

struct Placed {
  Item it;
  int64_t iu;
};

// All items in the order of the line, and its length.
template <typename Wk>
int64_t line(const AttnParams& p, std::vector<Placed>* items) {
  int64_t u = 0;
  Item it;
  for (int r = 0; r < p.B; ++r) {
    Wk::request(p, r, it);
    if (it.qlen == 0) continue;
    u += Wk::row_tile_units(p, it, 0, 1) * p.g.heads;
  }
  int64_t at = 0;
  int r = 0;
  while (r < p.B && (Wk::request(p, r, it), it.qlen == 0)) ++r;
  if (r == p.B) return 0;
  it.h = it.row0 = 0;
  Wk::range(p, it);
  while (at < u) {
    items->push_back({it, at});
    at += Wk::cost(p, it);
    if (at < u) Wk::next(p, it);
  }
  if (at != u) {
    fprintf(stderr, "items end at %lld of %lld units\n", (long long)at, (long long)u);
    exit(1);
  }
  return u;
}

// Walks the shares; `part(item, ta, tb)` checks what one holds of an item.
template <typename Wk, typename F>
void walk(const Call& c, const AttnParams& p, int64_t U, int N, const std::vector<Placed>& items, F part) {
  std::vector<int> done(items.size(), 0);
  size_t at = 0;
  for (int w = 0; w < N; ++w) {
    const int64_t u0 = share_start(U, N, w), u1 = share_start(U, N, w + 1);
    CHECK(u0 < u1 && (w > 0 || u0 == 0) && (w < N - 1 || u1 == U), "share %d of %d: [%lld, %lld)", w, N,
          (long long)u0, (long long)u1);
    while (at + 1 < items.size() && items[at + 1].iu <= u0) ++at;
    Item it = items[at].it;
    int64_t iu = items[at].iu;
    int a, b;
    size_t i = at;
    for (bool more = Wk::here(p, it, iu, u0, u1, a, b); more; more = Wk::after(p, it, iu, u0, u1, a, b)) {
      while (items[i].iu < iu) ++i;
      const Item& x = items[i].it;
      CHECK(items[i].iu == iu && x.r == it.r && x.h == it.h && x.row0 == it.row0 && x.tiles == it.tiles,
            "share %d: item %zu", w, i);
      CHECK(a == done[i] && a < b && b <= it.tiles, "share %d, item %zu: tiles [%d, %d) after %d of %d", w, i, a, b,
            done[i], it.tiles);
      done[i] = b;
      if (b == it.tiles)
        CHECK(share_of(Wk::last_unit(p, it, iu), N, U) == w, "share %d ends item %zu", w, i);
      part(it, a, b, w);
    }
  }
  for (size_t i = 0; i < items.size(); ++i)
    CHECK(done[i] == items[i].it.tiles, "item %zu: %d of %d tiles", i, done[i], items[i].it.tiles);
}

void check_item(const Call& c, const Item& it, int tile) {
  int64_t lo, hi;
  seen(c, it.r, it.row0, it.row0 + it.rows - 1, &lo, &hi);
  CHECK(it.tiles >= 1 && it.t0 >= 0, "tiles %d from %d", it.tiles, it.t0);
  if (lo >= hi) return;
  CHECK(it.begin == lo && it.end == hi, "row %d of request %d: [%d, %d), not [%lld, %lld)", it.row0, it.r, it.begin,
        it.end, (long long)lo, (long long)hi);
  CHECK(it.t0 == lo / tile && (int64_t)it.t0 + it.tiles == (hi - 1) / tile + 1, "tiles of [%lld, %lld)", (long long)lo,
        (long long)hi);
}

template <int D>
void many_rows(const Call& c) {
  using Wk = TcWalk<D>;
  Params q(c);
  q.p.rows_upto = 1 << 30;
  std::vector<Placed> items;
  const int64_t U = line<Wk>(q.p, &items);
  const int N = tc_shares(c.ctas, U);
  for (const Placed& x : items) check_item(c, x.it, kTcTile);
  walk<Wk>(c, q.p, U, N, items, [&](const Item& it, int ta, int tb, int w) {
    for (int i = 0; i < kTcRowTiles<D>; ++i) {
      int ra, rb;
      row_tile_range(q.p, it, i, ta, tb, ra, rb);
      CHECK(ta <= ra && ra <= rb && rb <= tb, "share %d, rows from %d: row tile %d takes [%d, %d) of [%d, %d)", w,
            it.row0, i, ra, rb, ta, tb);
      const int last = std::min(it.rows, 128 * i + 128) - 1;
      if (last < 128 * i) continue;
      int64_t lo, hi;
      seen(c, it.r, it.row0 + 128 * i, it.row0 + last, &lo, &hi);
      if (lo >= hi) continue;
      const int64_t need_a = std::max<int64_t>(lo / kTcTile - it.t0, ta),
                    need_b = std::min<int64_t>((hi - 1) / kTcTile + 1 - it.t0, tb);
      CHECK(need_a >= need_b || (ra <= need_a && need_b <= rb), "share %d, rows from %d: row tile %d needs [%lld, %lld)",
            w, it.row0, i, (long long)need_a, (long long)need_b);
    }
  });
}

void few_rows(const Call& c) {
  using Wk = StreamWalk;
  Params q(c);
  q.p.rows_upto = 64;
  std::vector<Placed> items;
  const int64_t U = line<Wk>(q.p, &items);
  if (U == 0) return;
  for (const Placed& x : items) check_item(c, x.it, 32);
  const int N = (int)std::min<int64_t>((int64_t)c.ctas * 12, U);
  walk<Wk>(c, q.p, U, N, items, [&](const Item& it, int, int tb, int) {
    // the page of every run that is looked up ahead of a share's last tile
    for (int ahead = 0; ahead < 1024; ahead += 16) {
      const int64_t page = ((int64_t)(it.t0 + tb - 1) * 32 + ahead) / c.page_size;
      const int got = listed_page(q.p, it.t0 + tb - 1, 32, ahead);
      CHECK(got == (page < c.max_pages ? page : -1), "page %d for %lld of %d", got, (long long)page, c.max_pages);
    }
  });
}

using Rng = std::mt19937_64;
int upto(Rng& g, int lo, int hi) { return lo + (int)(g() % (uint64_t)(hi - lo + 1)); }

// prompts and chunks, most of them windowed
Call prompts(Rng& g) {
  static const int groups[] = {1, 1, 1, 2, 3, 4, 5, 7, 8, 16}, pages[] = {16, 32, 64, 128}, ctas[] = {152, 152, 148, 1, 7, 160};
  Call c;
  c.heads = upto(g, 1, 8);
  c.group = groups[g() % 10];
  c.page_size = pages[g() % 4];
  c.causal = g() % 8 != 0;
  c.window = g() % 4 == 0 ? 0 : 1 << upto(g, 0, 12);
  if (c.window) c.window += upto(g, 0, c.window);
  c.ctas = ctas[g() % 6];
  const int n = upto(g, 1, 6);
  int most = 1;
  for (int i = 0; i < n; ++i) {
    const int rows = upto(g, 0, 7) == 0 ? 0 : upto(g, 16, 3001);
    c.rows.push_back(i == 0 ? std::max(rows, 16) : rows);
    c.kv.push_back(upto(g, 0, 3) == 0 ? upto(g, 0, rows + 5000) : rows);   // a cache that starts behind its first rows too
    most = std::max(most, c.kv.back());
  }
  c.max_pages = most / c.page_size + 1;
  return c;
}

// windows up to the largest int ("no limit" to a caller), caches that start behind the requests' first rows
Call wide_windows(Rng& g) {
  Call c = prompts(g);
  c.window = g() % 2 ? 2147483647 - upto(g, 0, 3000) : 2147483647;
  for (int& n : c.kv) n = g() % 2 ? upto(g, 0, 40) : n;
  return c;
}

// lengths up to the last that a block table can list, and so many heads that an item's units pass 32 bits
Call long_caches(Rng& g) {
  Call c = prompts(g);
  c.max_pages = 2147483647 / c.page_size;
  const int most = c.max_pages * c.page_size;
  for (int& n : c.kv) n = g() % 4 == 0 ? upto(g, 0, 3000) : 2147483647 - upto(g, 0, 2000);
  c.window = g() % 3 == 0 ? 0 : g() % 3 == 0 ? upto(g, 1, 2147483647) : upto(g, 1, 100000);
  if (g() % 2) c.heads = upto(g, 900, 1024);
  for (int& n : c.kv) n = std::min(n, most);
  for (int& n : c.rows) n = std::min(n, c.heads > 8 ? 40 : 600);
  c.rows[0] = std::max(c.rows[0], 16);
  return c;
}

// requests with more rows than the call looks after: the others stand where they stood
Call more_rows(Rng& g) {
  Call c = prompts(g);
  c.most = upto(g, 1, c.rows[0]);
  if (g() % 2) c.behind = upto(g, 0, c.rows.back());
  return c;
}

void run(const char* mode, Rng& g) {
  if (!strcmp(mode, "prompts")) {
    const Call c = prompts(g);
    many_rows<64>(c);
    many_rows<256>(c);
  } else if (!strcmp(mode, "few")) {
    Call c = prompts(g);
    for (int& n : c.rows) n = n ? 1 + n % std::max(1, 64 / c.group) : 0;
    few_rows(c);
  } else if (!strcmp(mode, "wide_windows")) {
    Call c = wide_windows(g);
    many_rows<128>(c);
    many_rows<256>(c);
    for (int& n : c.rows) n = n ? 1 + n % std::max(1, 64 / c.group) : 0;
    few_rows(c);
  } else if (!strcmp(mode, "more_rows")) {
    Call c = more_rows(g);
    many_rows<64>(c);
    many_rows<256>(c);
    if (c.group <= 8) {
      c.most = upto(g, 1, 8);
      few_rows(c);
    }
  } else if (!strcmp(mode, "long_caches")) {
    Call c = long_caches(g);
    many_rows<128>(c);
    for (int& n : c.rows) n = n ? 1 + n % std::max(1, 64 / c.group) : 0;
    few_rows(c);
  } else {
    fprintf(stderr, "unknown mode %s\n", mode);
    exit(2);
  }
}

}  // namespace

int main(int argc, char** argv) {
  if (argc != 4) return 2;
  Rng g(strtoull(argv[2], nullptr, 10));
  for (int i = atoi(argv[3]); i > 0; --i) run(argv[1], g);
  return 0;
}
