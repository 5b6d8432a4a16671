// The fp32 results of cut walks in the dK/dV schedule (csrc/win_schedule.cuh):
// every part unit has a place of its own, the join finds each tile's parts at
// theirs, and what the schedule costs. Prints
//   ok <units> <part units> <blocks of the longest unit> <blocks in all> <blocks of the busiest of 152 CTAs>
// (a block: 128 queries of one head by 128 keys) or a message and returns 1.
//   window_parts_check b sq skv hq hkv window sinks            uniform
//   window_parts_check packed hq hkv window sinks len len ...  packed
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "../context_blockwise_causal_gb300/csrc/win_schedule.cuh"

using namespace cpattn;

#define CHECK(c, ...)               \
  do {                              \
    if (!(c)) {                     \
      std::printf(__VA_ARGS__);     \
      std::printf(" (%s)\n", #c);   \
      return 1;                     \
    }                               \
  } while (0)

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
  win_finish(g, false);
  win_set_parts(g);
  win_set_divs(g, false);

  struct Part {
    int seq = -1, h = 0, kt = 0, qa = 0, nq = 0;
  };
  const int64_t units = win_dkdv_units(g), parts = g.part_units;
  std::vector<Part> at(static_cast<size_t>(parts));
  int64_t longest = 0, all = 0;
  constexpr int kGrid = 152;
  std::vector<int64_t> cta(kGrid, 0);
  for (int rd = 0; int64_t(rd) * kGrid < units; ++rd)
    for (int c = 0; c < kGrid; ++c) {
      const int idx = snake_unit(rd, c, kGrid);
      if (idx >= units) continue;
      const BwdWinUnit U = win_dkdv_unit(g, idx);
      CHECK((U.place >= 0) == (idx < parts), "unit %d place %d", idx, U.place);
      longest = U.items > longest ? U.items : longest;
      all += U.items;
      cta[c] += U.items;
      if (U.place < 0) continue;
      CHECK(U.place < parts && at[U.place].seq < 0, "unit %d place %d taken", idx, U.place);
      at[U.place].seq = U.seq;
      at[U.place].h = U.g;
      at[U.place].kt = U.v;
      at[U.place].qa = U.qa;
      at[U.place].nq = U.nq;
    }
  // the join
  WinCuts cuts;
  int64_t tiles = int64_t(g.b) * g.hkv * win_cut_tiles(g);
  if (g.nseq > 0) {
    win_set_cuts(g, cuts);
    tiles = int64_t(g.hkv) * cuts.first[g.nseq];
  }
  CHECK((tiles > 0) == (parts > 0), "%ld join tiles", long(tiles));
  std::vector<char> joined(static_cast<size_t>(parts), 0);
  for (int64_t x = 0; x < tiles; ++x) {
    int seq = -1, h = -1, kt = -1;
    if (g.nseq > 0) win_cut_tile(g, cuts, int(x), seq, h, kt);
    else win_cut_tile(g, int(x), seq, h, kt);
    CHECK(seq >= 0 && seq < num_seqs(g) && h >= 0 && h < g.hkv && kt >= 0 && kt < win_cut_tiles(g), "join tile %ld", long(x));
    const WinSeq s = win_seq(g, seq);
    if (kt * kTile >= s.klen) continue;
    int qa, nq;
    win_query_tiles(g, s, kt, qa, nq);
    for (int p = 0; p < win_parts(g, nq); ++p) {
      const int64_t i = win_first_part(g, seq, h, kt) + p;
      CHECK(i >= 0 && i < parts && !joined[i], "tile %ld part %d", long(x), p);
      joined[i] = 1;
      CHECK(at[i].seq == seq && at[i].h == h && at[i].kt == kt && at[i].qa == qa + p * g.part_tiles && at[i].nq > 0,
            "tile %ld part %d is not where the join looks", long(x), p);
    }
  }
  for (int64_t i = 0; i < parts; ++i)
    CHECK(joined[i] == (at[i].nq > 0), "place %ld written but not joined", long(i));
  int64_t busiest = 0;
  for (const int64_t c : cta) busiest = c > busiest ? c : busiest;
  std::printf("ok %ld %ld %ld %ld %ld\n", long(units), long(parts), long(longest), long(all), long(busiest));
  return 0;
}
