// The keys that the sequences of a group have in common, read once for all of
// their queries.
//
// The query heads that share a KV head, of every member of the group, are the
// rows of one matrix product: |group| G of them against the group's common
// keys, 4 d flops a row and key for 4 d bytes a key. So few rows are HBM-bound,
// and from about 290 on (measured peaks) the tensor cores are the limit; single
// rows' matrix tiles, as in paged_kernel.cuh, would read the keys again for
// each member. The members' own keys and the join are that file's kernels'.
//
// One CTA per run (see SharedPlan): a unit of up to 256 rows and some of its
// key tiles of 128. The warps' roles, TMEM and the online softmax are the
// forward's (fwd_kernel.cuh): two sub-tiles keep the tensor cores busy while
// the other one's softmax runs. Above 128 rows the two are the unit's row
// tiles, and share the key tiles; below, both hold the same rows and take the
// key tiles in turn, so that a unit of few rows also has two softmaxes at once
// and, with one tile of queries, more room for keys on their way; their two
// results are joined at the end in shared memory.
//
// Keys come by TMA, in boxes of as many tokens as page_size and 128 have as
// their common divisor (16 or more), a lane of the producer warp for each of
// a tile's boxes. Boxes past the common keys are not read. Where the last tile
// ends inside a box, what the page holds beyond is masked in the scores, and
// its values are overwritten with zeros in shared memory, so that nothing there,
// infinities and NaN included, reaches a sum.
//
// How long runs are is settled on the device, since the counts live there:
// every CTA adds up the tiles of all groups and takes the shortest length for
// which all runs fit into the CTAs that were launched, so groups of different
// lengths fill the chip evenly. CTA 0 leaves each group's place for the join.
//
// Measured, d128: 1.75 us for two row tiles and a key tile in the steady state
// (1460 TFLOP/s over the chip, as the forward), 3 us to the plan, 3 to 6 more to
// the first scores (queries and first keys of all CTAs come at once), 2 us to
// store. 64 sequences behind 32768 tokens with up to 1024 of their own, h32/8: 66
// us with the own keys and the join (45 us of bytes); 256 behind 16384 with up to
// 2048, h64/8: 242 to 250 us (212).
#pragma once
#include <cuda_bf16.h>

#include "fwd_kernel.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace cpattn {

struct PrefixArgs {
  SharedPlan sh;
  PagedPlace pg;
  const __nv_bfloat16* q;  // [b, hq, D], batch stride q_batch
  int64_t q_batch;
  int hq;
  int box;  // tokens of a box: gcd(page_size, 128)
  int sms;
  float scale_log2;
  unsigned int* status;
  uint32_t producer_waits;  // as PagedArgs::copy_waits, of the producer's for free slots
};

template <int D>
struct PrefixCfg {
  static constexpr int kTileBytes = kTile * D * 2;         // queries, keys or values
  static constexpr int kSlots = D == 128 ? 7 : 12;         // the first (or first two) hold queries
  static constexpr int kOffBar = kSlots * kTileBytes;
  // q_full s_full[2] p_half[2] p_full[2] o_full[2] drain kv_full[] kv_empty[]
  static constexpr int kNumBars = 10 + 2 * kSlots;
  static constexpr int kOffMisc = (kOffBar + kNumBars * 8 + 15) & ~15;
  static constexpr int kSmemBytes = kOffMisc + 64 + 1024;  // + alignment slack
  static constexpr uint32_t kColO = 256;
  static_assert(kSmemBytes <= 232448, "shared memory per block");
  // a sub-tile's results are left where the keys were
  static_assert(kTile * D * 4 <= (kSlots - 2) * kTileBytes, "join");
};

constexpr int kPrefixMinTiles = 2;  // tiles of a run at least (where there are as many)

// A CTA's run.
struct PrefixRun {
  int go;            // 0: nothing to do
  int first, row0;   // first sequence of the group, first row of the unit in the group
  int rows;          // rows of the unit
  int kvh, keys;     // KV head; common keys of the group
  int tile0, tiles;  // key tiles
  int table;         // the sequence whose table names the pages
};

// How many of the CTAs take runs. While they do, the members' own keys are read
// by the other SMs (paged_kernel.cuh runs beside this kernel), so each of the
// two gets the SMs that let both end together: with tp and to the times that
// they would take by themselves on all SMs, and kOwnShare the part of the SMs
// that reads at the chip's full bandwidth, tp / x = to kOwnShare / (1 - x). (64
// sequences behind 32768 tokens with up to 1024 of their own, h32/8 d128: 66 us
// for 0.35 to 0.5, 71 for 0.1 and 0.9; the whole chip first, then the own keys, 72.)
constexpr float kRowTileNs = 875.f;       // of an SM for 128 rows and a key tile, d 64 and 128, as measured
constexpr float kOwnBytesPerNs = 6700.f;  // measured copy bandwidth
constexpr float kOwnShare = 0.4f;
__device__ __forceinline__ float prefix_share(float tile_ns, float own_bytes, int sms) {
  const float tp = tile_ns / sms, to = own_bytes / kOwnBytesPerNs;
  return tp / (tp + to * kOwnShare);
}

// Finds the CTA's run. One whole warp; CTA 0 also writes every group's place.
// (The number of groups is seldom above 32; up to there a lane keeps its group
// in registers.)
__device__ __forceinline__ PrefixRun prefix_plan(const SharedPlan& s, int cta, int sms, float row_tile_ns) {
  const int lane = threadIdx.x & 31;
  PrefixRun r = {};
  struct Group {
    int first, size, keys, tiles, units;
  };
  const auto of = [&](int g) {
    Group x = {};
    if (g < s.groups) {
      shared_group(s, g, x.first, x.size);
      x.keys = shared_count(s, g);
      x.units = (x.size * s.G + kSharedRows - 1) / kSharedRows * s.hkv;
      x.tiles = x.units > 0 ? (x.keys + kTile - 1) / kTile : 0;
    }
    return x;
  };
  // Whether the SMs are shared with the own keys' kernel (units take at most half
  // of them); with more units nobody asks how long the sequences are.
  const bool shares = s.ctas == sms;
  // (the first lengths are on their way while the groups' loads are waited for)
  int head[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) head[k] = shares && lane + 32 * k < s.b ? s.lengths[lane + 32 * k] : 0;
  const Group mine = of(lane);
  float held[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) held[k] = float(head[k]);
  if (shares)
    for (int i = lane + 128; i < s.b; i += 128)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i + 32 * k < s.b) held[k] += float(s.lengths[i + 32 * k]);
  // work of all groups, in tiles and in row tiles; own keys (as if every member shared)
  float total = 0.f, rows = 0.f, own = (held[0] + held[1]) + (held[2] + held[3]);
  unsigned units = 0;
  for (int g0 = 0; g0 < s.groups; g0 += 32) {
    const Group x = g0 == 0 ? mine : of(g0 + lane);
    const float tiles = float(x.tiles) * float(s.hkv);
    total += tiles * float((x.size * s.G + kSharedRows - 1) / kSharedRows);
    rows += tiles * float((x.size * s.G + kTile - 1) / kTile);
    own -= float(x.keys) * float(x.size);
    units += __reduce_add_sync(0xffffffffu, x.tiles > 0 ? unsigned(x.units) : 0u);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, o);
    rows += __shfl_xor_sync(0xffffffffu, rows, o);
    own += __shfl_xor_sync(0xffffffffu, own, o);
  }
  int ctas = s.ctas;
  if (shares) {
    const float own_bytes = fmaxf(own, 0.f) * float(s.hkv) * s.token_bytes;
    ctas = int(prefix_share(rows * row_tile_ns, own_bytes, sms) * float(sms));
    ctas = ctas < int(units) ? int(units) : ctas;
    ctas = ctas < s.ctas ? ctas : s.ctas;
  }
  int len = int(total / float(ctas));
  if (s.groups == 1 && units > 0) {  // the shortest that fits
    const unsigned runs = unsigned(ctas) / units, tiles = unsigned(__shfl_sync(0xffffffffu, mine.tiles, 0));
    len = int((tiles + runs - 1) / runs);
  }
  if (len < kPrefixMinTiles) len = kPrefixMinTiles;
  // there are as many CTAs as units, so this ends: at the latest when no unit is cut
  while (true) {
    unsigned runs = 0;
    for (int g0 = 0; g0 < s.groups; g0 += 32) {
      const Group x = g0 == 0 ? mine : of(g0 + lane);
      const unsigned long long v = (unsigned long long)(unsigned(x.tiles + len - 1) / unsigned(len)) * unsigned(x.units);
      const unsigned most = kSharedMaxCtas;  // more than there are CTAs; 32 of them fit a word
      const unsigned add = __reduce_add_sync(0xffffffffu, v < most ? unsigned(v) : most);
      runs = runs + add < (1u << 31) ? runs + add : (1u << 31);
    }
    if (runs <= unsigned(ctas)) break;
    len += len >= 16 ? len / 16 : 1;
  }
  int base = 0;
  for (int g0 = 0; g0 < s.groups; g0 += 32) {
    const Group x = g0 == 0 ? mine : of(g0 + lane);
    const int runs = int(unsigned(x.tiles + len - 1) / unsigned(len)), count = runs * x.units;
    int up = count;  // inclusive sum over the lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += v;
    }
    const int from = base + up - count;
    if (cta == 0 && g0 + lane < s.groups) s.runs[g0 + lane] = {from, runs};
    const unsigned hit = __ballot_sync(0xffffffffu, cta >= from && cta < from + count);
    if (hit) {
      const int l = __ffs(hit) - 1;
      const auto get = [&](int v) { return __shfl_sync(0xffffffffu, v, l); };
      const int first = get(x.first), size = get(x.size), tiles = get(x.tiles), gruns = get(runs);
      const int local = cta - get(from);
      const int unit = local / gruns, run = local % gruns, row_units = (size * s.G + kSharedRows - 1) / kSharedRows;
      r.first = first;
      r.keys = get(x.keys);
      r.kvh = unit / row_units;
      r.row0 = (unit % row_units) * kSharedRows;
      r.rows = size * s.G - r.row0 < kSharedRows ? size * s.G - r.row0 : kSharedRows;
      const int per = (tiles + gruns - 1) / gruns;  // no run is empty: per <= len
      r.tile0 = run * per;
      r.tiles = tiles - r.tile0 < per ? tiles - r.tile0 : per;
      // The first of the unit's members that holds all of the common tokens names
      // their pages; without one, nobody reads the unit's results. (The whole
      // group's members may be many, and each CTA would look through them.)
      const int end = (r.row0 + r.rows - 1) / s.G + 1;
      for (int m0 = r.row0 / s.G; m0 < end; m0 += 32) {
        const int m = m0 + lane;
        const unsigned full = __ballot_sync(0xffffffffu, m < end && s.lengths[first + m] >= r.keys);
        if (full) {
          r.table = first + m0 + __ffs(full) - 1;
          r.go = 1;
          break;
        }
      }
    }
    base += __shfl_sync(0xffffffffu, up, 31);
  }
  return r;
}

template <int D>
__global__ void __launch_bounds__(kFwdThreads, 1)
    cpattn_prefix_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                         const __grid_constant__ PrefixArgs a) {
  using C = PrefixCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* q_full = bars;
  uint64_t* s_full = bars + 1;
  uint64_t* p_half = bars + 3;
  uint64_t* p_full = bars + 5;
  uint64_t* o_full = bars + 7;
  uint64_t* drain = bars + 9;
  uint64_t* kv_full = bars + 10;
  uint64_t* kv_empty = bars + 10 + C::kSlots;
  PrefixRun* run = reinterpret_cast<PrefixRun*>(smem + C::kOffMisc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc + 48);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 52);
  static_assert(sizeof(PrefixRun) <= 48, "run");

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (warp == 9) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  // Up to here, and the barriers, beside what runs before this call; the own
  // keys' kernel finds that finished.
  chain_wait();
  chain_next();
  if (warp == 0) {
    const PrefixRun r = prefix_plan(a.sh, blockIdx.x, a.sms, kRowTileNs);
    if (lane == 0) *run = r;
  }
  if (warp == 8 && lane == 0) {
    tma_prefetch_desc(&tmk);
    tma_prefetch_desc(&tmv);
    *abort_flag = 0;
    mbar_init(q_full, 8);
    mbar_init(drain, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_half[i], 4);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_full[i], 1);
    }
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  if (!run->go) {
    if (warp == 9) tmem_dealloc(tbase, 512);
    return;
  }

  const int n = run->tiles;
  const bool pair = run->rows > kTile;  // two row tiles, or one whose key tiles the sub-tiles take in turn
  const int q_tiles = pair ? 2 : 1;
  const uint32_t slots = C::kSlots - q_tiles;
  uint8_t* sKV = smem + q_tiles * C::kTileBytes;
  // keys of the run's last tile
  const int tail = run->keys - (run->tile0 + n - 1) * kTile < kTile ? run->keys - (run->tile0 + n - 1) * kTile : kTile;

  if (warp >= 8) {
    reg_dealloc<kFwdOtherRegs>();
    if (warp == 8) {
      // ------------------------------------------------------------ producer
      const int boxes = kTile / a.box;  // of a whole tile; lane: its box
      const int cols = boxes == 1 ? 1 : D / 64;  // copies of a box: a whole tile is one
      const int* table = a.pg.tables + int64_t(run->table) * a.pg.tables_row;
      const int key0 = run->tile0 * kTile + lane * a.box;  // first key of this lane's box in the run's first tile
      const auto page_of = [&](int t) {
        const int key = key0 + t * kTile;
        return t < n && lane < boxes && key < run->keys ? table[unsigned(key) / unsigned(a.pg.page_size)] : 0;
      };
      bool ok = true;
      uint32_t nload = 0, waits = a.producer_waits;
      // Tile t's keys or values into the next slot of the ring, from this lane's page.
      const auto load = [&](const CUtensorMap* map, int t, int page) {
        const uint32_t slot = nload % slots, turn = nload / slots;
        if (turn > 0 && !(waits-- > 0 && mbar_wait_warp(&kv_empty[slot], (turn - 1) & 1, abort_flag, kWaitLimitNs))) {
          *abort_flag = 1;
          return false;
        }
        const int key = key0 + t * kTile;
        const int live = t < n - 1 ? boxes : (tail + a.box - 1) / a.box;  // boxes that hold common keys
        if (lane == 0) mbar_arrive_expect_tx(&kv_full[slot], uint32_t(live) * a.box * (D * 2));
        __syncwarp();
        if (lane < live) {
          page_ok(page, a.pg, a.status);  // (a copy from outside of the pool brings zeros)
          const int at = int(unsigned(key) % unsigned(a.pg.page_size));
          bounds_ok(key < a.sh.cap && at + a.box <= a.pg.page_size, a.status);
          uint8_t* dst = sKV + slot * C::kTileBytes + lane * a.box * 128;
          for (int c = 0; c < cols; ++c)
            tma_load_5d(dst + c * (kTile * 128), map, &kv_full[slot], 0, at, c, run->kvh, page);
        }
        __syncwarp();
        ++nload;
        return true;
      };
      // in the order of the MMA warp: K of the first tile (of the first two, taken in turn), then V(t), K(t + ahead)
      const int ahead = pair ? 1 : 2;
      int pk[2] = {page_of(0), page_of(1)}, pv = pk[0];  // pages of the tiles ahead
      ok = load(&tmk, 0, pk[0]);
      if (ok && !pair && n > 1) ok = load(&tmk, 1, pk[1]);
      int nv = pk[1];               // tile t + 1
      int nn = pair ? nv : page_of(2);  // tile t + ahead
      for (int t = 0; ok && t < n; ++t) {
        const int next = page_of(t + ahead + 1);
        ok = load(&tmv, t, pv);
        if (ok && t + ahead < n) ok = load(&tmk, t + ahead, nn);
        pv = nv;
        nv = pair ? next : nn;
        nn = next;
      }
      if (!ok && lane == 0) atomicOr(a.status, kStatusProducer);
      // every copy in flight lands before the CTA can exit
      bool drained = true;
      for (uint32_t i = nload > slots ? nload - slots : 0; i < nload; ++i)
        drained &= mbar_wait_drain_warp(&kv_full[i % slots], (i / slots) & 1, kWaitLimitNs);
      if (!drained && lane == 0) atomicOr(a.status, kStatusDrain);
    } else if (warp == 9) {
      // ------------------------------------------------------------ MMA issuer
      constexpr uint32_t idS = make_idesc_bf16(kTile, kTile, false, false);
      constexpr uint32_t idO = make_idesc_bf16(kTile, D, false, true);
      const uint64_t dQ = make_sdesc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t dK = make_sdesc_sw128(smem_u32(sKV), 16, 1024);
      const uint64_t dV = make_sdesc_sw128(smem_u32(sKV), 16384, 1024);
      uint32_t ncons = 0;
      bool ok = true;
      const auto take = [&](uint32_t& slot) {
        slot = ncons % slots;
        const uint32_t par = (ncons / slots) & 1;
        ++ncons;
        return ok = mbar_wait_warp(&kv_full[slot], par, abort_flag, kWaitLimitNs);
      };
      const auto issue_S = [&](int sub, uint32_t slot) {
        const uint64_t qb = dQ + ((pair ? sub * C::kTileBytes : 0) >> 4), kb = dK + ((slot * C::kTileBytes) >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk / 4) * (kTile * 128) + (kk % 4) * 32) >> 4;
          umma_ss_w(tbase + sub * kTile, qb + off, kb + off, idS, kk > 0);
        }
        umma_commit_w(&s_full[sub]);
      };
      uint32_t pcnt[2] = {0, 0};
      // O += P V, the first half of the keys as soon as their P is in TMEM
      const auto issue_PV = [&](int sub, uint32_t slot, bool acc) {
        const uint64_t vb = dV + ((slot * C::kTileBytes) >> 4);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          ok = mbar_wait_warp(half ? &p_full[sub] : &p_half[sub], pcnt[sub] & 1, abort_flag, kWaitLimitNs);
          if (!ok) return false;
          tc_fence_after();
#pragma unroll
          for (int q = 0; q < kTile / 32; ++q) {
            const int kk = half * (kTile / 32) + q;
            umma_ts_w(tbase + C::kColO + sub * D, tbase + sub * kTile + kk * 8, vb + ((kk * 2048) >> 4), idO,
                      (acc || kk > 0) ? 1u : 0u);
          }
        }
        ++pcnt[sub];
        return true;
      };
      // The last tile's values past the common keys: zeros instead of what
      // the page (or, past its last box, an earlier tile) holds there.
      const auto clear_tail = [&](uint32_t slot) {
        if (tail == kTile) return;
        uint8_t* v = sKV + slot * C::kTileBytes;
        for (int i = tail * 8 + lane; i < kTile * 8; i += 32)
#pragma unroll
          for (int x = 0; x < D; x += 64)
            *reinterpret_cast<uint4*>(v + (x / 64) * (kTile * 128) + i * 16) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
        __syncwarp();
      };
      uint32_t k, v;
      ok = mbar_wait_warp(q_full, 0, abort_flag, kWaitLimitNs);
      if (ok && pair) {
        if (take(k)) {
          issue_S(0, k);
          issue_S(1, k);
          umma_commit_w(&kv_empty[k]);
        }
        for (int j = 0; ok && j < n; ++j) {
          if (!take(v)) break;
          if (j == n - 1) clear_tail(v);
          if (!issue_PV(0, v, j > 0)) break;
          if (j == n - 1) umma_commit_w(&o_full[0]);
          if (j + 1 < n) {
            if (!take(k)) break;
            issue_S(0, k);
          }
          if (!issue_PV(1, v, j > 0)) break;
          umma_commit_w(&kv_empty[v]);
          if (j == n - 1) umma_commit_w(&o_full[1]);
          if (j + 1 < n) {
            issue_S(1, k);
            umma_commit_w(&kv_empty[k]);
          }
        }
      } else if (ok) {
        for (int sub = 0; sub < 2 && sub < n && take(k); ++sub) {
          issue_S(sub, k);
          umma_commit_w(&kv_empty[k]);
        }
        for (int t = 0; ok && t < n; ++t) {
          const int sub = t & 1;
          if (!take(v)) break;
          if (t == n - 1) clear_tail(v);
          if (!issue_PV(sub, v, t > 1)) break;
          umma_commit_w(&kv_empty[v]);
          if (t + 2 >= n) umma_commit_w(&o_full[sub]);
          if (t + 2 < n) {
            if (!take(k)) break;
            issue_S(sub, k);
            umma_commit_w(&kv_empty[k]);
          }
        }
      }
      if (!ok && lane == 0) atomicOr(a.status, kStatusMma);
      // no MMA may be in flight when TMEM and the shared memory are released
      umma_commit_w(drain);
      if (!mbar_wait_drain_warp(drain, 0, kWaitLimitNs) && lane == 0) atomicOr(a.status, kStatusDrain);
    }
  } else {
    reg_alloc<kFwdSoftmaxRegs>();
    // ------------------------------------------------------------ softmax
    const int sub = warp >> 2;
    const int wq = warp & 3;
    const int row = wq * 32 + lane;
    const int unit_row = (pair ? sub * kTile : 0) + row;  // row within the unit
    // Queries: 16-byte pieces, all on their way at once, swizzled as TMA would
    // (piece p of row r of a 128-byte column block at p ^ (r & 7)); rows past the
    // unit's are zeros.
    {
      constexpr int kPieces = D / 8, kPerStep = 32 / kPieces;
      const int rows_each = pair ? 32 : 16;
      const int r0 = (pair ? wq * 32 : warp * 16) + lane / kPieces;  // this lane's first row of its tile
      const int ur0 = (pair ? sub * kTile : 0) + r0;
      const int p = lane % kPieces;
      const uint32_t dst = smem_u32(smem) + (pair ? sub * C::kTileBytes : 0) + (p / 8) * (kTile * 128);
      int seq = (run->row0 + ur0) / a.sh.G, head = run->row0 + ur0 - seq * a.sh.G;
      const __nv_bfloat16* q0 = a.q + int64_t(run->first) * a.q_batch + int64_t(run->kvh * a.sh.G) * D + p * 8;
      for (int s = 0; s < rows_each; s += kPerStep) {
        const int r = r0 + s;
        const bool valid = ur0 + s < run->rows;
        bounds_ok(!valid || (run->first + seq < a.sh.b && run->kvh * a.sh.G + head < a.hq), a.status);
        cp_async16(dst + r * 128 + (((p % 8) ^ (r & 7)) * 16), valid ? q0 + seq * a.q_batch + head * D : a.q, valid);
        head += kPerStep;
        while (head >= a.sh.G) {
          head -= a.sh.G;
          ++seq;
        }
      }
      cp_async_commit();
      cp_async_wait<0>();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    }
    const uint32_t lane_off = uint32_t(wq * 32) << 16;
    const uint32_t tS = tbase + lane_off + sub * kTile;
    const uint32_t tO = tbase + lane_off + C::kColO + sub * D;
    const float sl2 = a.scale_log2;
    bool ok = true;  // (waits are the whole warp's: TMEM is read and written by all lanes or none)
    float m_used = -INFINITY, l = 0.f;
    const int mine = pair ? n : (n - sub + 1) / 2;  // tiles of this sub-tile
    for (int j = 0; j < mine; ++j) {
      const int t = pair ? j : 2 * j + sub;
      if (!(ok = mbar_wait_warp(&s_full[sub], j & 1, abort_flag, kWaitLimitNs))) break;
      tc_fence_after();
      float s[kTile];
      float m_raw;
      {
        uint32_t r0[32], r1[32], r2[32], r3[32];
        float m4[4];
        tmem_ld32x4_max(tS, tS + 32, tS + 64, tS + 96, r0, r1, r2, r3, m4);
        m_raw = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          s[i] = __uint_as_float(r0[i]);
          s[32 + i] = __uint_as_float(r1[i]);
          s[64 + i] = __uint_as_float(r2[i]);
          s[96 + i] = __uint_as_float(r3[i]);
        }
      }
      if (t == n - 1 && tail < kTile) {
#pragma unroll
        for (int i = 0; i < kTile; ++i)
          if (i >= tail) s[i] = -INFINITY;
        m_raw = row_max(s);
      }
      const float m_new = m_raw * sl2;
      const bool upd = m_new > m_used;
      float alpha = 1.f;
      if (upd) {
        alpha = m_used == -INFINITY ? 0.f : ex2_approx(m_used - m_new);
        m_used = m_new;
      }
      const float neg = m_used == -INFINITY ? 0.f : -m_used;
      const bool rescale = j > 0 && __any_sync(0xffffffffu, upd);
      uint32_t pk[32];
      const uint64_t sl2x2 = f2_pack(sl2, sl2), negx2 = f2_pack(neg, neg);
      uint64_t acc[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = f2_pack(0.f, 0.f);
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
#pragma unroll
        for (int q = 0; q < kTile / 4; ++q) {
          const int i = hh * (kTile / 4) + q;
          float x0, x1;
          f2_unpack(f2_fma(f2_pack(s[2 * i], s[2 * i + 1]), sl2x2, negx2), x0, x1);
          const float e0 = ex2_approx(x0), e1 = ex2_approx(x1);
          acc[i & 3] = f2_add(acc[i & 3], f2_pack(e0, e1));
          pk[q] = pack_bf16x2(e0, e1);
        }
        if (hh == 0 && rescale) {  // P V of the sub-tile's last tile was complete before S was signalled
#pragma unroll
          for (int c0 = 0; c0 < D; c0 += 32) {
            uint32_t r[32];
            tmem_ld32(tO + c0, r);
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
            tmem_st32_nowait(tO + c0, r);
          }
        }
        tmem_st32(tS + hh * 32, pk);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(hh == 0 ? &p_half[sub] : &p_full[sub]);
      }
      float a0, a1;
      f2_unpack(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])), a0, a1);
      l = l * alpha + (a0 + a1);
    }
    // ---- epilogue: O / l as it is, and its log-sum-exp. Two sub-tiles of the
    // same rows are joined first: sub-tile 1 leaves its O where the keys were,
    // once no product reads them any more (chunk c of 16 bytes of row r at
    // c ^ r, modulo the row's chunks: no two rows meet in a bank), and its m and l
    // where the queries were.
    constexpr int kChunks = D / 4;
    const auto spot = [&](int c) {
      return reinterpret_cast<float4*>(sKV) + row * kChunks + (c ^ (row & (kChunks - 1)));
    };
    float2* sML = reinterpret_cast<float2*>(smem);
    if (ok && mine > 0) ok = mbar_wait_warp(&o_full[sub], 0, abort_flag, kWaitLimitNs);
    if (!pair) {
      if (ok && n > 1) ok = mbar_wait_warp(&o_full[1 - sub], 0, abort_flag, kWaitLimitNs);
      tc_fence_after();
      if (sub == 1 && ok && mine > 0) {  // (with one tile the queries may still be read)
#pragma unroll
        for (int c0 = 0; c0 < D; c0 += 32) {
          uint32_t r[32];
          tmem_ld32(tO + c0, r);
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *spot((c0 + i) / 4) = make_float4(__uint_as_float(r[i]), __uint_as_float(r[i + 1]),
                                              __uint_as_float(r[i + 2]), __uint_as_float(r[i + 3]));
        }
        sML[row] = make_float2(m_used, l);
      }
      // every softmax warp comes here, whether or not a role gave up
      asm volatile("bar.sync 1, 256;" ::: "memory");
    }
    tc_fence_after();
    if (__all_sync(0xffffffffu, ok && !*abort_flag) && (pair || sub == 0)) {
      float w0 = 1.f, w1 = 0.f;
      const bool other = !pair && n > 1;
      if (other) {
        const float2 o = sML[row];
        const float m = fmaxf(m_used, o.x);
        const float base = m == -INFINITY ? 0.f : m;
        w0 = ex2_approx(m_used - base);
        w1 = ex2_approx(o.x - base);
        l = l * w0 + o.y * w1;
        m_used = m;
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      w0 *= inv;
      w1 *= inv;
      const int64_t out = int64_t(blockIdx.x) * a.sh.part_rows + unit_row;
      const bool store = unit_row < run->rows && bounds_ok(unit_row < a.sh.part_rows && blockIdx.x < a.sh.ctas, a.status);
#pragma unroll
      for (int c0 = 0; c0 < D; c0 += 32) {
        uint32_t r[32];
        tmem_ld32(tO + c0, r);
        float x[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(r[i]) * w0;
        if (other) {
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const float4 y = *spot((c0 + i) / 4);
            x[i] = fmaf(y.x, w1, x[i]);
            x[i + 1] = fmaf(y.y, w1, x[i + 1]);
            x[i + 2] = fmaf(y.z, w1, x[i + 2]);
            x[i + 3] = fmaf(y.w, w1, x[i + 3]);
          }
        }
        // whole 32-byte sectors
        if (store)
#pragma unroll
          for (int i = 0; i < 32; i += 8) store_sector(a.sh.part_o + out * D + c0 + i, x + i);
      }
      if (store) a.sh.part_lse[out] = l == 0.f ? -INFINITY : m_used + log2f(l);
    }
    if (!ok && lane == 0) atomicOr(a.status, kStatusSoftmax);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

}  // namespace cpattn
