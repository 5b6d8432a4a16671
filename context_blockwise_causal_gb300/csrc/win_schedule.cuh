// Work decomposition of sliding-window attention with visible first tokens.
//
// Query at position p of its sequence sees key j when
//     j <= p  and  (p - j < window  or  j < sinks).
// A sequence has qlen queries and klen >= qlen keys; its queries are the last
// qlen positions (query row t is position off + t, off = klen - qlen), so a
// chunk of a prompt can attend to what was read before it. Tiles are 128
// queries or keys counted from the sequence's first row.
//
// Forward and dQ units: a query tile (two, see win_fwd_unit) visits the key
// tiles that hold visible first tokens, then the tiles its windows cover.
// dK/dV units: a key tile visits the query tiles whose windows reach it; a
// tile holding first tokens is seen by every later query, so its walk is cut
// into parts of about an ordinary tile's work, each a unit of its own, whose
// fp32 results a second kernel adds in a fixed order (win_set_parts).
//
// Window units differ little in cost, so their order follows the data:
// consecutive units are neighbouring tiles of one KV head, and the CTAs in
// flight read the same K/V (or Q/dO) rows from L2.
#pragma once
#include "cp_schedule.cuh"

namespace cpattn {

// A sequence's rows and lengths in the window form.
struct WinSeq {
  int q0, kv0;     // first row on the query side and on the key/value side
  int qlen, klen;
  int off;         // position of query row 0
};

__host__ __device__ inline WinSeq win_seq(const CpGeom& g, int seq) {
  WinSeq s;
  if (g.nseq > 0) {
    s.q0 = s.kv0 = g.cu[seq];
    s.qlen = s.klen = g.cu[seq + 1] - g.cu[seq];
  } else {
    s.q0 = seq * g.s;
    s.kv0 = seq * g.kv_s;
    s.qlen = g.s;
    s.klen = g.kv_s;
  }
  s.off = s.klen - s.qlen;
  return s;
}

struct WinUnit : FwdUnit {
  int kv0;      // first key row of the unit's sequence
  int off;      // position of its query row 0
  int ns, w0;   // tiles of first tokens visited, then tiles from w0 on
  // The one tile of first tokens is visited for its first kSinkKeys keys only:
  // all of the unit's queries see exactly the first `sinks` of them.
  bool narrow;
};

// First tokens up to this many take a product of their own width instead of a
// whole tile's (in the forward and dQ kernels).
constexpr int kSinkKeys = 16;

// Query tiles (kPairs: pairs of tiles) of a sequence of qlen queries.
__host__ __device__ inline int win_unit_tiles(int qlen, bool pairs) {
  const int t = (qlen + kTile - 1) / kTile;
  return pairs ? (t + 1) / 2 : t;
}

// Packed samples: prefix sums of the tiles (or tile pairs, or key tiles) of
// the samples; a uniform batch needs none.
__host__ __device__ inline void win_finish(CpGeom& g, bool pairs) {
  g.tpc = win_unit_tiles(g.s, false);
  if (g.nseq > 0) {
    g.b = 1;
    g.s = g.kv_s = g.cu[g.nseq];
    g.tpc = 0;
    g.tile0[0] = 0;
    for (int i = 0; i < g.nseq; ++i) {
      const int len = g.cu[i + 1] - g.cu[i];
      const int t = win_unit_tiles(len, false);
      g.tpc = t > g.tpc ? t : g.tpc;
      g.tile0[i + 1] = g.tile0[i] + win_unit_tiles(len, pairs);
    }
  }
}

// Key tile of walk position j.
__host__ __device__ inline int win_tile(const WinUnit& U, int j) { return j < U.ns ? j : U.w0 + (j - U.ns); }

// Key tiles that the positions p_first .. p_last see.
__host__ __device__ inline void win_fill_walk(const CpGeom& g, WinUnit& U, int p_first, int p_last) {
  const int lo = p_first - g.window + 1;
  U.w0 = lo > 0 ? lo / kTile : 0;
  const int st = (g.sinks + kTile - 1) / kTile;
  U.ns = st < U.w0 ? st : U.w0;
  U.narrow = U.ns == 1 && g.sinks <= kSinkKeys;
  U.n = U.ns + p_last / kTile - U.w0 + 1;
}

// Whether a block of 128 queries from position p0 and 128 keys from kb is
// visible as a whole.
__host__ __device__ inline bool win_block_full(const CpGeom& g, int p0, int kb) {
  return kb + kTile - 1 <= p0 && (p0 + kTile - 1 - kb < g.window || kb + kTile <= g.sinks);
}

// What 32 queries from position p0 see of 32 keys from kb: none, all, or some.
// The kernels' warps skip the exponentials of hidden pieces and mask only
// mixed ones.
enum WinPiece { kHidden = 0, kMixed = 1, kVisible = 2 };
__host__ __device__ inline int win_piece(const CpGeom& g, int p0, int kb) {
  if (kb > p0 + 31 || (kb + 31 <= p0 - g.window && kb >= g.sinks)) return kHidden;
  return kb + 31 <= p0 && (p0 + 31 - kb < g.window || kb + 31 < g.sinks) ? kVisible : kMixed;
}

// Forward units per launch: a query tile for a pair of query heads of one KV
// group, or -- when the group's heads are odd in number -- two query tiles of
// one head (kPairs), so that both sub-tiles always share their K/V tiles.
__host__ __device__ inline int64_t win_fwd_units(const CpGeom& g, bool pairs) {
  const int64_t heads = pairs ? g.hq : g.hq / 2;
  return heads * (g.nseq > 0 ? g.tile0[g.nseq] : int64_t(g.b) * win_unit_tiles(g.s, pairs));
}

template <bool kPairs>
__host__ __device__ inline WinUnit win_fwd_unit(const CpGeom& g, int idx) {
  WinUnit U;
  const int G = g.hq / g.hkv;
  const int per = kPairs ? G : G / 2;  // units of one tile and KV head
  int tile, hp;                        // the unit's tile (or pair) and its head (or head pair)
  if (g.nseq > 0) {
    const int heads = g.hkv * per;
    const int p = idx / heads;
    hp = idx - p * heads;
    int local;
    U.seq = packed_sample_of(g, p, local);
    tile = g.tile0[U.seq + 1] - g.tile0[U.seq] - 1 - local;
  } else {
    const int T = win_unit_tiles(g.s, kPairs);
    const int x = g.fd_per.div(idx);
    hp = idx - x * per;
    const int y = g.fd_T.div(x);
    tile = T - 1 - (x - y * T);  // the shorter walks of the first tiles come last
    U.seq = g.fd_hkv.div(y);
    const int kvh = y - U.seq * g.hkv;
    hp += kvh * per;
  }
  const WinSeq s = win_seq(g, U.seq);
  U.bi = g.nseq > 0 ? 0 : U.seq;
  U.tok0 = s.q0;
  U.lse_t0 = g.nseq > 0 ? s.q0 : 0;
  U.kv0 = s.kv0;
  U.off = s.off;
  U.c = s.qlen;
  U.tpc = g.tpc;
  U.k = U.r = U.half = 0;
  U.h0 = kPairs ? hp : 2 * hp;
  U.h1 = kPairs ? hp : 2 * hp + 1;
  U.g0 = U.g1 = g.fd_G.div(U.h0);
  U.store1 = true;
  U.u = U.u0 = kPairs ? 2 * tile : tile;
  U.q_t0 = U.q_t1 = U.u0 * kTile;
  const int rem = s.qlen - U.q_t0;
  U.q_valid = U.q_valid1 = rem < kTile ? rem : kTile;
  int last = U.q_t0 + U.q_valid - 1;
  if (kPairs) {
    if (rem > kTile) {
      U.q_t1 = U.q_t0 + kTile;
      U.q_valid1 = rem - kTile < kTile ? rem - kTile : kTile;
      last = U.q_t1 + U.q_valid1 - 1;
    } else {
      U.store1 = false;  // an odd tile count: sub-tile 1 repeats sub-tile 0 and stores nothing
    }
  }
  win_fill_walk(g, U, s.off + U.q_t0, s.off + last);
  return U;
}

// dQ units: one query tile of one head.
__host__ __device__ inline int64_t win_dq_units(const CpGeom& g) {
  return int64_t(g.hq) * (g.nseq > 0 ? g.tile0[g.nseq] : int64_t(g.b) * g.tpc);
}

__host__ __device__ inline WinUnit win_dq_unit(const CpGeom& g, int idx) {
  WinUnit U;
  const int G = g.hq / g.hkv;
  if (g.nseq > 0) {
    const int p = idx / g.hq;
    U.h0 = idx - p * g.hq;
    int local;
    U.seq = packed_sample_of(g, p, local);
    U.u = g.tile0[U.seq + 1] - g.tile0[U.seq] - 1 - local;
  } else {
    const int x = g.fd_G.div(idx);
    const int y = g.fd_tpc.div(x);
    U.u = g.tpc - 1 - (x - y * g.tpc);
    U.seq = g.fd_hkv.div(y);
    U.h0 = (y - U.seq * g.hkv) * G + (idx - x * G);
  }
  const WinSeq s = win_seq(g, U.seq);
  U.bi = g.nseq > 0 ? 0 : U.seq;
  U.tok0 = s.q0;
  U.lse_t0 = g.nseq > 0 ? s.q0 : 0;
  U.kv0 = s.kv0;
  U.off = s.off;
  U.c = s.qlen;
  U.tpc = g.tpc;
  U.k = U.r = U.half = 0;
  U.h1 = U.h0;
  U.g0 = U.g1 = g.fd_G.div(U.h0);
  U.store1 = false;
  U.u0 = U.u;
  U.q_t0 = U.q_t1 = U.u * kTile;
  const int rem = s.qlen - U.q_t0;
  U.q_valid = U.q_valid1 = rem < kTile ? rem : kTile;
  win_fill_walk(g, U, s.off + U.q_t0, s.off + U.q_t0 + U.q_valid - 1);
  return U;
}

// ---------------------------------------------------------------- dK / dV
struct BwdWinUnit : BwdUnit {
  int kv0;      // first key row of the unit's sequence
  int off;      // position of its query row 0
  int qlen;
  int qa;       // first query tile visited (nq of them; the walk comes down from the last)
  int place;    // a part of a cut walk: index of its fp32 result; -1: the whole walk
  int rows;     // key rows of the tile that the part's queries see (win_part_rows)
  int64_t slot; // first-token tiles where any walk is cut: the part's number among all that the call's
                // sequences could have, by which the schedule's check knows it; -1: another tile
};

// Query tiles in which some query sees a key of tile kt: [qa, qa + nq).
__host__ __device__ inline void win_query_tiles(const CpGeom& g, const WinSeq& s, int kt, int& qa, int& nq) {
  const int k0 = kt * kTile;
  const int k1 = k0 + kTile < s.klen ? k0 + kTile - 1 : s.klen - 1;  // last key
  const int lo = k0 > s.off ? k0 - s.off : 0;
  int hi = s.qlen - 1;
  if (k0 >= g.sinks) {
    const int64_t reach = int64_t(k1) + g.window - 1 - s.off;
    if (reach < hi) hi = int(reach);
  }
  qa = lo / kTile;
  nq = hi < lo ? 0 : hi / kTile - qa + 1;
}

// Key rows of tile kt that query tiles from qa on see: all of them, or only
// first tokens where the tiles lie beyond every row's window. The other rows'
// results of such a part are zero: they are neither stored nor added.
__host__ __device__ inline int win_part_rows(const CpGeom& g, const WinSeq& s, int kt, int qa) {
  const int k0 = kt * kTile;
  if (int64_t(s.off) + int64_t(qa) * kTile < int64_t(k0) + kTile - 1 + g.window) return kTile;
  return g.sinks - k0 < kTile ? g.sinks - k0 : kTile;
}

// Parts of a cut walk: query tiles [qa + part * per, ...) with per =
// part_tiles; the number of parts that have any.
__host__ __device__ inline int win_parts(const CpGeom& g, int nq) { return (nq + g.part_tiles - 1) / g.part_tiles; }

// First-token tiles of a sequence, whose walks are cut where they are longer
// than a part (0 when no sequence's are).
__host__ __device__ inline int win_cut_tiles(const CpGeom& g) { return g.cut_tiles; }
// Parts there would be if every sequence were as long as the longest.
__host__ __device__ inline int64_t win_cut_units(const CpGeom& g) {
  return int64_t(num_seqs(g)) * g.hkv * win_cut_tiles(g) * g.sink_parts;
}
// Of a packed sample of `tiles` key tiles: those whose walks are cut (samples
// shorter than a part keep theirs whole and need no fp32 result).
__host__ __device__ inline int win_sample_cut(const CpGeom& g, int tiles) {
  const int cut = win_cut_tiles(g);
  return tiles > g.part_tiles ? (cut < tiles ? cut : tiles) : 0;
}
__host__ __device__ inline int win_sample_tiles(const CpGeom& g, int i) {
  return win_unit_tiles(g.cu[i + 1] - g.cu[i], false);
}
// The first part of tile kt of KV head h of a sequence: part units come first,
// so their number is also the place of their fp32 result. Every cut tile has as
// many as the first of its sequence.
__host__ __device__ inline int64_t win_first_part(const CpGeom& g, int seq, int h, int kt) {
  if (g.nseq == 0) return ((int64_t(seq) * g.hkv + h) * win_cut_tiles(g) + kt) * g.sink_parts;
  const int tiles = win_sample_tiles(g, seq);
  return int64_t(g.part0[seq]) * g.hkv + (int64_t(h) * win_sample_cut(g, tiles) + kt) * win_parts(g, tiles);
}
// The sample i with first[i] <= p < first[i + 1] of a prefix sum over samples.
__host__ __device__ inline int win_sample_of(const int* first, int n, int p) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= p) lo = mid; else hi = mid;
  }
  return lo;
}
// The join's tiles: all cut ones, by sequence, KV head and tile. Packed
// samples have as many as they are long for.
__host__ __device__ inline void win_cut_tile(const CpGeom& g, int x, int& seq, int& h, int& kt) {
  const int y = g.fd_cut.div(x);
  kt = x - y * win_cut_tiles(g);
  seq = g.fd_hkv.div(y);
  h = y - seq * g.hkv;
}
struct WinCuts {
  int first[kMaxSeqs + 1];  // cut tiles per KV head of the samples before sample i
};
inline void win_set_cuts(const CpGeom& g, WinCuts& c) {
  c.first[0] = 0;
  for (int i = 0; i < g.nseq; ++i) c.first[i + 1] = c.first[i] + win_sample_cut(g, win_sample_tiles(g, i));
}
__host__ __device__ inline void win_cut_tile(const CpGeom& g, const WinCuts& c, int x, int& seq, int& h, int& kt) {
  seq = win_sample_of(c.first, g.nseq, g.fd_hkv.div(x));
  const int n = c.first[seq + 1] - c.first[seq];
  x -= c.first[seq] * g.hkv;
  h = x / n;
  kt = x - h * n;
}
__host__ __device__ inline int win_key_tiles(const CpGeom& g) { return (g.kv_s + kTile - 1) / kTile; }
__host__ __device__ inline int64_t win_dkdv_units(const CpGeom& g) {
  return g.part_units + int64_t(g.hkv) * (g.nseq > 0 ? g.tile0[g.nseq] : int64_t(g.b) * win_key_tiles(g));
}

__host__ __device__ inline BwdWinUnit win_dkdv_unit(const CpGeom& g, int idx) {
  BwdWinUnit U;
  const int cut = win_cut_tiles(g);
  int kt, part = 0;
  bool elsewhere = false;  // an ordinary unit of a tile whose walk is cut
  U.place = -1;
  if (idx < g.part_units) {
    U.place = idx;
    if (g.nseq > 0) {
      U.seq = win_sample_of(g.part0, g.nseq, g.fd_hkv.div(idx));
      const int tiles = win_sample_tiles(g, U.seq), np = win_parts(g, tiles), nc = win_sample_cut(g, tiles);
      idx -= g.part0[U.seq] * g.hkv;
      U.g = idx / (nc * np);
      idx -= U.g * (nc * np);
      kt = idx / np;
      part = idx - kt * np;
    } else {
      const int x = g.fd_parts.div(idx);
      part = idx - x * g.sink_parts;
      const int y = g.fd_cut.div(x);
      kt = x - y * cut;
      U.seq = g.fd_hkv.div(y);
      U.g = y - U.seq * g.hkv;
    }
  } else {
    idx -= g.part_units;
    if (g.nseq > 0) {
      const int p = idx / g.hkv;
      U.g = idx - p * g.hkv;
      U.seq = packed_sample_of(g, p, kt);
      elsewhere = kt < win_sample_cut(g, g.tile0[U.seq + 1] - g.tile0[U.seq]);
    } else {
      const int T = win_key_tiles(g);
      const int y = g.fd_kt.div(idx);
      kt = idx - y * T;
      U.seq = g.fd_hkv.div(y);
      U.g = y - U.seq * g.hkv;
      elsewhere = kt < cut;
    }
  }
  U.slot = kt < cut ? ((int64_t(U.seq) * g.hkv + U.g) * cut + kt) * g.sink_parts + part : -1;
  const WinSeq s = win_seq(g, U.seq);
  U.bi = g.nseq > 0 ? 0 : U.seq;
  U.tok0 = s.q0;
  U.kv0 = s.kv0;
  U.off = s.off;
  U.c = U.qlen = s.qlen;
  U.tpc = g.tpc;
  U.kc = 0;
  U.v = U.gt = kt;
  U.k_t0 = kt * kTile;
  U.qa = 0;
  U.rows = kTile;
  if (U.k_t0 >= s.klen || elsewhere) {  // no such key tile, or one whose parts are units
    U.k_t0 = U.k_valid = U.nq = U.items = 0;
    return U;
  }
  const int rem = s.klen - U.k_t0;
  U.k_valid = rem < kTile ? rem : kTile;
  win_query_tiles(g, s, kt, U.qa, U.nq);
  if (U.place >= 0) {
    const int from = part * g.part_tiles;
    const int left = U.nq - from;
    U.qa += from;
    U.nq = left < 0 ? 0 : (left < g.part_tiles ? left : g.part_tiles);
    if (U.nq == 0) U.k_valid = 0;  // a part that the walk does not reach writes nothing
    U.rows = win_part_rows(g, s, kt, U.qa);
  }
  U.items = U.nq * (g.hq / g.hkv);
  return U;
}

// Query tiles that the key tiles with first tokens visit in a sequence of
// `tiles` query tiles, the first at position off.
__host__ __device__ inline int64_t win_first_walks(const CpGeom& g, int tiles, int off) {
  const int64_t keys = win_unit_tiles(off, false) + int64_t(tiles);  // no key tile past the last query's
  const int64_t firsts = (g.sinks + kTile - 1) / kTile, n = firsts < keys ? firsts : keys;
  const int64_t later = n > win_unit_tiles(off, false) ? n - win_unit_tiles(off, false) : 0;  // a query tile less each
  return n * tiles - later * (later - 1) / 2;
}

// Cuts the walks of the tiles that hold first tokens into parts of an ordinary
// tile's work (which is seen by about window/128 + 1 query tiles; at least 8
// tiles, at most kMaxParts parts) when such a walk is over twice that and
// longer than a quarter of what each of a full chip's CTAs has to do in all:
// with many sequences or heads whole walks balance by themselves, and parts
// would only cost workspace. (Parts of twice that size left the last round of
// CTAs uneven: 852 us against 795 us for the kernel at b1 s32768 h32/8 window
// 1024.)
//
// Every sample counts with its own length: taken to be as long as the longest,
// 64 samples of 64 tokens beside one of 32768 kept that one's walk whole, and
// the backward took 3100 us instead of 1680 (h32/8 d128 window 1024).
constexpr int kMaxParts = 64;
constexpr int kWinChipCtas = 152;
__host__ __device__ inline void win_set_parts(CpGeom& g) {
  g.sink_parts = 1;
  g.part_units = g.cut_tiles = 0;
  g.part_tiles = g.tpc > 0 ? g.tpc : 1;
  for (int i = 0; i <= g.nseq; ++i) g.part0[i] = 0;
  if (g.sinks == 0) return;
  const int ordinary = g.window / kTile + 1;
  int tiles = ordinary > 8 ? ordinary : 8;
  if (g.tpc <= 2 * tiles) return;
  const int64_t key_tiles = g.nseq > 0 ? g.tile0[g.nseq] : int64_t(g.b) * win_key_tiles(g);
  int64_t long_walks = 0;
  if (g.nseq > 0)
    for (int i = 0; i < g.nseq; ++i) long_walks += win_first_walks(g, win_sample_tiles(g, i), 0);
  else
    long_walks = g.b * win_first_walks(g, g.tpc, g.kv_s - g.s);
  const int64_t work = g.hkv * (key_tiles * ordinary + long_walks);  // query tiles visited
  if (int64_t(g.tpc) * 4 * kWinChipCtas <= work) return;
  const int least = (g.tpc + kMaxParts - 1) / kMaxParts;
  if (tiles < least) tiles = least;
  // The parts' fp32 dK and dV may take four times the bytes of dk and dv, no
  // more: two parts per key tile. (Only hundreds of first tokens reach it, and
  // two parts of every walk always fit.)
  for (;; tiles += tiles / 8 + 1) {
    g.part_tiles = tiles;
    g.sink_parts = (g.tpc + tiles - 1) / tiles;
    g.cut_tiles = g.sink_parts > 1 ? (g.sinks + kTile - 1) / kTile : 0;
    int64_t parts = int64_t(g.b) * g.cut_tiles * g.sink_parts;  // per KV head
    if (g.nseq > 0) {
      parts = 0;
      for (int i = 0; i < g.nseq; ++i) {
        const int t = win_sample_tiles(g, i);
        g.part0[i] = int(parts);
        parts += int64_t(win_sample_cut(g, t)) * win_parts(g, t);
      }
      g.part0[g.nseq] = int(parts);
    }
    if (parts <= 2 * key_tiles) {
      g.part_units = int(parts * g.hkv);
      return;
    }
  }
}

// The divisors of the decodes above; after win_finish and win_set_parts.
__host__ __device__ inline void win_set_divs(CpGeom& g, bool pairs) {
  const int G = g.hq / g.hkv, T = win_unit_tiles(g.s, pairs), cut = win_cut_tiles(g);
  g.fd_hkv = make_fastdiv(g.hkv);
  g.fd_G = make_fastdiv(G);
  g.fd_tpc = make_fastdiv(g.tpc > 0 ? g.tpc : 1);
  g.fd_per = make_fastdiv(pairs ? G : (G > 1 ? G / 2 : 1));
  g.fd_T = make_fastdiv(T > 0 ? T : 1);
  g.fd_kt = make_fastdiv(win_key_tiles(g) > 0 ? win_key_tiles(g) : 1);
  g.fd_parts = make_fastdiv(g.sink_parts);
  g.fd_cut = make_fastdiv(cut > 0 ? cut : 1);
}

}  // namespace cpattn
