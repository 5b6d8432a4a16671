// Brute-force check of the sliding-window work decomposition
// (csrc/win_schedule.cuh) on the host: every visible (head, query, key) pair
// is reached exactly once by the forward's units, by the dQ units and by the
// dK/dV units; tiles called fully visible are; every row that a unit reads or
// writes lies inside the tensors; every part of a cut walk has its slot.
// Prints "ok <pairs>" or a message and returns 1.
//   window_schedule_check b sq skv hq hkv window sinks            uniform
//   window_schedule_check packed hq hkv window sinks len len ...  packed
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "../context_blockwise_causal_gb300/csrc/win_schedule.cuh"

using namespace cpattn;

static bool sees(const CpGeom& g, int p, int j) { return j <= p && (p - j < g.window || j < g.sinks); }

#define CHECK(c, ...)               \
  do {                              \
    if (!(c)) {                     \
      std::printf(__VA_ARGS__);     \
      std::printf(" (%s)\n", #c);   \
      return 1;                     \
    }                               \
  } while (0)

struct Count {
  // per (head, query row): one counter per key of its sequence
  std::vector<std::vector<unsigned char>> c;
  int rows;
  Count(int heads, int rows_) : c(size_t(heads) * rows_), rows(rows_) {}
  std::vector<unsigned char>& at(int h, int row) { return c[size_t(h) * rows + row]; }
};

static int verify(const CpGeom& g, Count& n, const char* what, long* pairs) {
  long total = 0;
  for (int h = 0; h < g.hq; ++h)
    for (int i = 0; i < num_seqs(g); ++i) {
      const WinSeq s = win_seq(g, i);
      for (int t = 0; t < s.qlen; ++t) {
        auto& c = n.at(h, s.q0 + t);
        for (int j = 0; j < s.klen; ++j) {
          const int want = sees(g, s.off + t, j) ? 1 : 0;
          const int got = j < int(c.size()) ? c[j] : 0;
          CHECK(got == want, "%s: head %d seq %d query %d key %d reached %d times, expected %d", what, h, i, t, j, got, want);
          total += want;
        }
      }
    }
  *pairs = total;
  return 0;
}

// A block of query rows [qt, qt + qv) and key tile kt of sequence s.
static int block(const CpGeom& g, const WinSeq& s, Count& n, int h, int qt, int qv, int kt, int kvrows) {
  const int kb = kt * kTile;
  CHECK(kb < s.klen && s.kv0 + kb < kvrows, "key tile %d outside its sequence", kt);
  const bool full = win_block_full(g, s.off + qt, kb);
  for (int r = 0; r < qv; ++r) {
    auto& c = n.at(h, s.q0 + qt + r);
    c.resize(s.klen, 0);
    for (int k = 0; k < kTile; ++k) {
      if (full) CHECK(kb + k < s.klen && sees(g, s.off + qt + r, kb + k), "block (%d, %d) called full is not", qt, kt);
      if (kb + k < s.klen && sees(g, s.off + qt + r, kb + k)) ++c[kb + k];
    }
  }
  return 0;
}

template <bool kPairs>
static int forward(CpGeom g, long* pairs) {
  win_finish(g, kPairs);
  win_set_parts(g);
  win_set_divs(g, kPairs);
  const int qrows = g.b * g.s, kvrows = g.b * g.kv_s;
  Count n(g.hq, qrows);
  const long units = win_fwd_units(g, kPairs);
  for (long idx = 0; idx < units; ++idx) {
    const WinUnit U = win_fwd_unit<kPairs>(g, int(idx));
    const WinSeq s = win_seq(g, U.seq);
    CHECK(U.n >= 1 && U.g0 == U.g1 && U.h0 / (g.hq / g.hkv) == U.g0, "unit %ld", idx);
    CHECK(U.tok0 == s.q0 && U.kv0 == s.kv0 && U.off == s.off, "unit %ld", idx);
    for (int sub = 0; sub < 2; ++sub) {
      const int qt = sub ? U.q_t1 : U.q_t0, qv = sub ? U.q_valid1 : U.q_valid;
      CHECK(qt >= 0 && qv >= 1 && qv <= kTile && qt + qv <= s.qlen && U.tok0 + qt < qrows, "unit %ld", idx);
      int last = -1;
      for (int j = 0; j < U.n; ++j) {
        const int kt = win_tile(U, j);
        CHECK(kt > last, "unit %ld: key tiles out of order", idx);
        last = kt;
        CHECK(U.kv0 + kt * kTile < kvrows && kt * kTile < s.klen, "unit %ld key tile %d", idx, kt);
        if (sub == 1 && !U.store1) continue;
        if (block(g, s, n, sub ? U.h1 : U.h0, qt, qv, kt, kvrows)) return 1;
      }
    }
  }
  return verify(g, n, "forward", pairs);
}

static int backward(CpGeom g, long* dq_pairs, long* kv_pairs) {
  win_finish(g, false);
  win_set_parts(g);
  win_set_divs(g, false);
  const int qrows = g.b * g.s, kvrows = g.b * g.kv_s, G = g.hq / g.hkv;
  Count n(g.hq, qrows);
  for (long idx = 0; idx < win_dq_units(g); ++idx) {
    const WinUnit U = win_dq_unit(g, int(idx));
    const WinSeq s = win_seq(g, U.seq);
    CHECK(U.q_t0 + U.q_valid <= s.qlen && U.q_valid >= 1 && U.n >= 1 && U.u < g.tpc, "dq unit %ld", idx);
    for (int j = 0; j < U.n; ++j)
      if (block(g, s, n, U.h0, U.q_t0, U.q_valid, win_tile(U, j), kvrows)) return 1;
  }
  if (verify(g, n, "dQ", dq_pairs)) return 1;

  Count m(g.hq, qrows);
  std::vector<int> owner(size_t(g.hkv) * kvrows, 0);  // units that write a key row of a KV head
  std::vector<char> slot(size_t(win_cut_units(g)), 0);
  for (long idx = 0; idx < win_dkdv_units(g); ++idx) {
    const BwdWinUnit U = win_dkdv_unit(g, int(idx));
    if (U.k_valid == 0) {
      CHECK(U.items == 0, "dkdv unit %ld", idx);
      continue;
    }
    const WinSeq s = win_seq(g, U.seq);
    CHECK(U.kv0 == s.kv0 && U.k_t0 + U.k_valid <= s.klen && U.items == U.nq * G, "dkdv unit %ld", idx);
    if (U.slot >= 0) {
      CHECK(U.slot < win_cut_units(g) && !slot[U.slot] && U.items > 0, "dkdv unit %ld slot %d", idx, U.slot);
      slot[U.slot] = 1;
      // the join kernel adds the tile's first win_parts parts
      int qa, nq;
      win_query_tiles(g, s, U.v, qa, nq);
      CHECK(U.slot % g.sink_parts < win_parts(g, nq), "dkdv unit %ld: part beyond those joined", idx);
      // rows past U.rows are neither stored nor joined: none of the part's queries sees them
      CHECK(U.rows >= 1 && U.rows == win_part_rows(g, s, U.v, qa + (U.slot % g.sink_parts) * g.part_tiles), "rows");
      for (int r = U.rows; r < U.k_valid; ++r)
        for (int t = U.qa * kTile; t < (U.qa + U.nq) * kTile && t < s.qlen; ++t)
          CHECK(!sees(g, s.off + t, U.k_t0 + r), "dkdv unit %ld: row %d is seen", idx, r);
    } else {
      for (int r = 0; r < U.k_valid; ++r) ++owner[size_t(U.g) * kvrows + U.kv0 + U.k_t0 + r];
    }
    for (int i = 0; i < U.nq; ++i) {
      const int qt = (U.qa + i) * kTile;
      CHECK(qt < s.qlen, "dkdv unit %ld query tile %d", idx, U.qa + i);
      const int qv = s.qlen - qt < kTile ? s.qlen - qt : kTile;
      for (int h = U.g * G; h < (U.g + 1) * G; ++h)
        if (block(g, s, m, h, qt, qv, U.v, kvrows)) return 1;
    }
  }
  // the joined tiles' rows, and that every part to be added was written
  const int cut = win_cut_tiles(g);
  for (int i = 0; i < num_seqs(g) && cut > 0; ++i) {
    const WinSeq s = win_seq(g, i);
    for (int h = 0; h < g.hkv; ++h)
      for (int kt = 0; kt < cut && kt * kTile < s.klen; ++kt) {
        int qa, nq;
        win_query_tiles(g, s, kt, qa, nq);
        CHECK(win_parts(g, nq) <= g.sink_parts, "more parts than slots");
        for (int p = 0; p < win_parts(g, nq); ++p)
          CHECK(slot[((size_t(i) * g.hkv + h) * cut + kt) * g.sink_parts + p], "seq %d tile %d part %d not written", i, kt, p);
        for (int r = kt * kTile; r < s.klen && r < (kt + 1) * kTile; ++r) ++owner[size_t(h) * kvrows + s.kv0 + r];
      }
  }
  for (size_t r = 0; r < owner.size(); ++r) CHECK(owner[r] == 1, "key row %zu written %d times", r, owner[r]);
  return verify(g, m, "dK/dV", kv_pairs);
}

int main(int argc, char** argv) {
  CpGeom g{};
  g.cp = 1;
  g.causal = 1;
  auto arg = [&](int i) { return std::atoi(argv[i]); };
  if (argc > 6 && !std::strcmp(argv[1], "packed")) {
    g.hq = arg(2);
    g.hkv = arg(3);
    g.window = arg(4);
    g.sinks = arg(5);
    g.nseq = argc - 6;
    g.cu[0] = 0;
    for (int i = 0; i < g.nseq; ++i) g.cu[i + 1] = g.cu[i] + arg(6 + i);
    g.b = 1;
    g.s = g.kv_s = g.cu[g.nseq];
  } else if (argc == 8) {
    g.b = arg(1);
    g.s = arg(2);
    g.kv_s = arg(3);
    g.hq = arg(4);
    g.hkv = arg(5);
    g.window = arg(6);
    g.sinks = arg(7);
  } else {
    return 2;
  }
  if (g.window > g.kv_s) g.window = g.kv_s;
  if (g.sinks > g.kv_s) g.sinks = g.kv_s;
  long f = 0, q = 0, k = 0;
  const bool pairs = (g.hq / g.hkv) % 2 != 0;
  if (pairs ? forward<true>(g, &f) : forward<false>(g, &f)) return 1;
  if (backward(g, &q, &k)) return 1;
  CHECK(f == q && q == k, "pairs differ: %ld %ld %ld", f, q, k);
  std::printf("ok %ld\n", f);
  return 0;
}
