// The keys that the sequences of a group have in common, read once for all of
// their queries.
//
// The query heads that share a KV head, of every member of the group, are the
// rows of one matrix product: |group| G of them against the group's common
// keys, 4 d flops a row and key for 4 d bytes a key. So few rows are HBM-bound,
// and from about 290 on (measured peaks) the tensor cores are the limit; single
// rows' matrix tiles, as in decode_kernel.cuh, would read the keys again for
// each member. The members' own keys and the join are that kernel's.
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
// Keys come by TMA, a box per page and 64 features (page_size and 128 have a
// common divisor of 16 or more tokens), each lane of the producer warp one
// page's boxes. Boxes past the common keys are not read. Where the last tile
// ends inside a box, what the page holds beyond is masked in the scores, and
// its values are overwritten with zeros in shared memory, so that nothing there,
// infinities and NaN included, reaches a sum.
//
// How long runs are is settled on the device, since the counts live there:
// every CTA adds up the tiles of all groups and takes the shortest length for
// which all runs fit into the CTAs that were launched, so groups of different
// lengths fill the chip evenly. CTA 0 leaves each group's place for the join.
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
  float scale_log2;
  unsigned int* status;
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
  // the results of both sub-tiles are staged where the keys were
  static_assert(2 * kTile * D * 4 <= (kSlots - 2) * kTileBytes, "staging");
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

// Finds the CTA's run. One whole warp; CTA 0 also writes every group's place.
__device__ __forceinline__ PrefixRun prefix_plan(const SharedPlan& s, int cta) {
  const int lane = threadIdx.x & 31;
  PrefixRun r = {};
  const auto of = [&](int g, int& tiles, int& units) {
    tiles = units = 0;
    if (g >= s.groups) return;
    int first, size;
    shared_group(s, g, first, size);
    tiles = (shared_count(s, g) + kTile - 1) / kTile;
    units = shared_units(s, size) * s.hkv;
    if (units == 0) tiles = 0;
  };
  const auto sum = [](int64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  };
  int64_t total = 0;
  for (int g0 = 0; g0 < s.groups; g0 += 32) {
    int tiles, units;
    of(g0 + lane, tiles, units);
    total += sum(int64_t(tiles) * units);
  }
  int64_t len = (total + s.ctas - 1) / s.ctas;
  if (len < kPrefixMinTiles) len = kPrefixMinTiles;
  // units take at most half of the CTAs, so this ends: at the latest when no unit is cut
  while (true) {
    int64_t runs = 0;
    for (int g0 = 0; g0 < s.groups; g0 += 32) {
      int tiles, units;
      of(g0 + lane, tiles, units);
      runs += sum(((tiles + len - 1) / len) * units);
    }
    if (runs <= s.ctas) break;
    len += len >= 16 ? len / 16 : 1;
  }
  int base = 0;
  for (int g0 = 0; g0 < s.groups; g0 += 32) {
    const int g = g0 + lane;
    int tiles, units;
    of(g, tiles, units);
    const int runs = int((tiles + len - 1) / len), mine = runs * units;
    int up = mine;  // inclusive sum over the lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += v;
    }
    const int from = base + up - mine;
    if (cta == 0 && g < s.groups) s.runs[g] = {from, runs};
    const unsigned hit = __ballot_sync(0xffffffffu, cta >= from && cta < from + mine);
    if (hit) {
      const int l = __ffs(hit) - 1;
      const int gg = g0 + l;
      const int gruns = __shfl_sync(0xffffffffu, runs, l), gtiles = __shfl_sync(0xffffffffu, tiles, l);
      const int local = cta - __shfl_sync(0xffffffffu, from, l);
      int first, size;
      shared_group(s, gg, first, size);
      const int unit = local / gruns, run = local % gruns, row_units = shared_units(s, size);
      r.first = first;
      r.kvh = unit / row_units;
      r.row0 = (unit % row_units) * kSharedRows;
      r.rows = size * s.G - r.row0 < kSharedRows ? size * s.G - r.row0 : kSharedRows;
      r.keys = shared_count(s, gg);
      const int per = (gtiles + gruns - 1) / gruns;  // no run is empty: per <= len
      r.tile0 = run * per;
      r.tiles = gtiles - r.tile0 < per ? gtiles - r.tile0 : per;
      // the first member that holds all of the common tokens names their pages
      for (int m0 = 0; m0 < size; m0 += 32) {
        const int m = m0 + lane;
        const unsigned held = __ballot_sync(0xffffffffu, m < size && s.lengths[first + m] >= r.keys);
        if (held) {
          r.table = first + m0 + __ffs(held) - 1;
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
  chain_next();
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
  if (warp == 0) {
    const PrefixRun r = prefix_plan(a.sh, blockIdx.x);
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
  __syncthreads();
  if (!run->go) return;
  if (warp == 9) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;

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
      const int* table = a.pg.tables + int64_t(run->table) * a.pg.tables_row;
      const int key0 = run->tile0 * kTile + lane * a.box;  // first key of this lane's box in the run's first tile
      const auto page_of = [&](int t) {
        const int key = key0 + t * kTile;
        return t < n && lane < boxes && key < run->keys ? table[unsigned(key) / unsigned(a.pg.page_size)] : 0;
      };
      bool ok = true;
      uint32_t nload = 0;
      // Tile t's keys or values into the next slot of the ring, from this lane's page.
      const auto load = [&](const CUtensorMap* map, int t, int page) {
        const uint32_t slot = nload % slots, turn = nload / slots;
        if (turn > 0 && !mbar_wait_warp(&kv_empty[slot], (turn - 1) & 1, abort_flag, kWaitLimitNs)) return false;
        const int key = key0 + t * kTile;
        const int live = t < n - 1 ? boxes : (tail + a.box - 1) / a.box;  // boxes that hold common keys
        if (lane == 0) mbar_arrive_expect_tx(&kv_full[slot], uint32_t(live) * a.box * (D * 2));
        __syncwarp();
        if (lane < live) {
          page_ok(page, a.pg, a.status);  // (a copy from outside of the pool brings zeros)
          const int at = int(unsigned(key) % unsigned(a.pg.page_size));
          bounds_ok(key < a.sh.cap && at + a.box <= a.pg.page_size, a.status);
          uint8_t* dst = sKV + slot * C::kTileBytes + lane * a.box * 128;
#pragma unroll
          for (int x = 0; x < D; x += 64)
            tma_load_4d(dst + (x / 64) * (kTile * 128), map, &kv_full[slot], x, run->kvh, at, page);
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
    // Queries: 16-byte pieces, swizzled as TMA would (piece p of row r of a 128-byte
    // column block at p ^ (r & 7)); rows past the unit's are zeros.
    {
      constexpr int kPieces = D / 8, kPerStep = 32 / kPieces;
      const int rows_each = pair ? 32 : 16;
      const int r0 = pair ? wq * 32 : warp * 16;  // rows of this warp in its tile
      uint8_t* dst = smem + (pair ? sub * C::kTileBytes : 0);
      const int p = lane % kPieces;
#pragma unroll 8
      for (int s = 0; s < rows_each; s += kPerStep) {
        const int r = r0 + s + lane / kPieces;
        const int ur = (pair ? sub * kTile : 0) + r;
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (ur < run->rows) {
          const int gr = run->row0 + ur, seq = gr / a.sh.G, head = gr - seq * a.sh.G;
          bounds_ok(run->first + seq < a.sh.b && run->kvh * a.sh.G + head < a.hq, a.status);
          x = *reinterpret_cast<const uint4*>(a.q + int64_t(run->first + seq) * a.q_batch +
                                              int64_t(run->kvh * a.sh.G + head) * D + p * 8);
        }
        *reinterpret_cast<uint4*>(dst + (p / 8) * (kTile * 128) + r * 128 + (((p % 8) ^ (r & 7)) * 16)) = x;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    }
    const uint32_t lane_off = uint32_t(wq * 32) << 16;
    const uint32_t tS = tbase + lane_off + sub * kTile;
    const uint32_t tO = tbase + lane_off + C::kColO + sub * D;
    const float sl2 = a.scale_log2;
    bool ok = true;
    float m_used = -INFINITY, l = 0.f;
    const int mine = pair ? n : (n - sub + 1) / 2;  // tiles of this sub-tile
    for (int j = 0; j < mine; ++j) {
      const int t = pair ? j : 2 * j + sub;
      if (!(ok = mbar_wait_bounded(&s_full[sub], j & 1, abort_flag, kWaitLimitNs))) break;
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
    // ---- epilogue. Results are staged where the keys were, once no product
    // reads them any more: chunk c of 16 bytes of row r at c ^ r (modulo the
    // row's chunks), so that neither rows nor chunks meet in a bank.
    constexpr int kChunks = D / 4;
    for (int i = 0; ok && i < 2; ++i)
      if (i < n || pair) ok = mbar_wait_bounded(&o_full[i], 0, abort_flag, kWaitLimitNs);
    tc_fence_after();
    const auto spot = [&](int tile, int r, int c) {
      return reinterpret_cast<float4*>(sKV) + (tile * kTile + r) * kChunks + (c ^ (r & (kChunks - 1)));
    };
    float2* sML = reinterpret_cast<float2*>(smem);  // where the queries were: m and l of sub-tile 1's rows
    if (!pair) {
      if (sub == 1 && ok) {
        if (mine > 0) {
#pragma unroll
          for (int c0 = 0; c0 < D; c0 += 32) {
            uint32_t r[32];
            tmem_ld32(tO + c0, r);
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *spot(1, row, (c0 + i) / 4) = make_float4(__uint_as_float(r[i]), __uint_as_float(r[i + 1]),
                                                        __uint_as_float(r[i + 2]), __uint_as_float(r[i + 3]));
          }
        }
        sML[row] = make_float2(m_used, l);
      }
      // every softmax warp comes here, whether or not a role gave up
      asm volatile("bar.sync 1, 256;" ::: "memory");
    }
    if (ok && !*abort_flag && (pair || sub == 0)) {
      float w0 = 1.f, w1 = 0.f;
      if (!pair) {
        const float2 o = sML[row];
        const float m = fmaxf(m_used, o.x);
        const float base = m == -INFINITY ? 0.f : m;
        w0 = ex2_approx(m_used - base);
        w1 = ex2_approx(o.x - base);
        l = l * w0 + o.y * w1;
        m_used = m;
      }
      const bool other = !pair && n > 1;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      w0 *= inv;
      w1 *= inv;
#pragma unroll
      for (int c0 = 0; c0 < D; c0 += 32) {
        uint32_t r[32];
        tmem_ld32(tO + c0, r);
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          float4 x = make_float4(__uint_as_float(r[i]) * w0, __uint_as_float(r[i + 1]) * w0,
                                 __uint_as_float(r[i + 2]) * w0, __uint_as_float(r[i + 3]) * w0);
          if (other) {
            const float4 y = *spot(1, row, (c0 + i) / 4);
            x.x = fmaf(y.x, w1, x.x);
            x.y = fmaf(y.y, w1, x.y);
            x.z = fmaf(y.z, w1, x.z);
            x.w = fmaf(y.w, w1, x.w);
          }
          *spot(sub, row, (c0 + i) / 4) = x;
        }
      }
      __syncwarp();
      // whole lines: the warp's rows one (d = 64: two) at a time
      const int64_t out = int64_t(blockIdx.x) * a.sh.part_rows;
      const int u0 = (pair ? sub * kTile : 0) + wq * 32;
#pragma unroll 4
      for (int i = lane; i < 32 * kChunks; i += 32) {
        const int r = i / kChunks, c = i % kChunks;
        if (u0 + r < run->rows && bounds_ok(u0 + r < a.sh.part_rows && blockIdx.x < a.sh.ctas, a.status))
          reinterpret_cast<float4*>(a.sh.part_o)[(out + u0 + r) * kChunks + c] = *spot(sub, wq * 32 + r, c);
      }
      if (unit_row < run->rows && unit_row < a.sh.part_rows)
        a.sh.part_lse[out + unit_row] = l == 0.f ? -INFINITY : m_used + log2f(l);
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
