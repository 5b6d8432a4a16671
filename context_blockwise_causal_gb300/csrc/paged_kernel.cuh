// Single-token attention over a cache in pages (paged.cuh), whole or with a
// sliding window and visible first tokens; and the same over the keys that a
// sequence does not share with its group (prefix_kernel.cuh), with the join of
// the two.
//
// Mathematics, tiles and joins are those of decode_kernel.cuh; what differs is
// how keys come. What is visible is cut into rounds of 64 keys, each starting at
// a whole 64 of the sequence's own numbering, 16 keys for each of the four
// warps that compute. A warp of its own asks the copy engine for them: a box of
// 32 or 16 tokens (the page size is a multiple of it) and all features for a
// lane, whose page it has looked up a round ahead. Asking is not cheap, some tens
// of cycles a box: when every warp asked for its own 16 keys in boxes of 64
// features, that took longer than the products (0.47 of 0.9 us for 16 keys, and
// 16 sequences of 32K to 64K keys took 491 us).
// The first and last keys of what is visible are masked inside their blocks:
// scores by the mask, and values, whose product with a weight of zero would
// still be NaN if they are not finite, by zeros written over them.
//
// P enters its product in two bf16 pieces, the rounded value and what the rounding
// left, for whole sequences: their products have time to spare. Relative L2
// of O 1.66e-3 to 1.68e-3, its own rounding and no more, with one piece
// 2.0e-3 to 2.2e-3; it costs 0.2 to 1.5 % with 8 heads or fewer to a KV head (one
// sequence of 8192 keys 11.3 -> 11.45 us, 16 of 32K to 64K keys 469 -> 471), 2 to 4 %
// with 16 (120 of 1000 to 2000 keys, d 64, 15.8 -> 16.45). Where common keys are
// computed, here and in prefix_kernel.cuh, P is rounded to one piece, as by the other
// attention kernels (2.1e-3 to 2.3e-3): units of many rows have no such time
// (32 rows behind 8192 keys 17.5 -> 18.6 us). Sums, maxima and joins are fp32.
//
// HBM-bound where there are sequences enough: 16 of 32K to 64K keys, h64/8 d128,
// 471 us (reads at 1.02 of the measured copy bandwidth, which counts writes
// too), 64 with a window of 4096, h32/8, pages of 16, 157 us (1.03). A few short
// ones are bound by what waits for one another: length, table, first copy, some
// rounds of 0.5 us, the joins (one sequence of 8192 keys, h32/8, 11.5 us, 9.0 where the
// keys lie in L2; 37 of 1464 to 2928, 2 KV heads of 64, 12.6).
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "decode_kernel.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace cpattn {

constexpr unsigned int kStatusCopies = 1u << 4;  // copies of a paged decode did not arrive in time
constexpr int kPagedThreads = (kDecWarps + 1) * 32;

struct PagedArgs {
  DecodeArgs d;  // k and v are not used (the copies' descriptors name the pools)
  PagedPlace pg;
  SharedPlan sh;    // kOwn, kBoth
  int common_ctas;  // kBoth
  int join_warps;   // of the join kernel, to a row
  int box;          // tokens of a copy: gcd(page_size, 32)
  uint32_t copy_waits;  // the copying warp gives up at the wait for a free stage after so many (kAllWaits: never)
};

constexpr int kPagedRound = kDecWarps * kDecBlock;  // keys of a round

template <int D>
struct PagedCfg {
  static constexpr int kTileBytes = kPagedRound * D * 2;  // keys or values of a round
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kStages = 3;
  // (d = 64 with six stages and two CTAs an SM: 64 sequences of 4096 to 8192 keys, 8 KV heads, 132 us instead of
  // 125; 37 of 1464 to 2928, 2 KV heads, 12.5 either way.)
  // barriers (full and empty per stage) and the flag come first, the ring (1024-byte aligned) behind them
  static constexpr int kOffFlag = 2 * kStages * 8;
  static constexpr int kOffRing = 1024;
  static constexpr int kSmemBytes = kOffRing + kStages * kStageBytes + 1024;  // + alignment slack
  // the join of the warps reuses the ring, kJoinBytes for each: O and pairs, as in DecodeCfg, and the CTA's result
  static constexpr int kResult = 16 * D * 4 + 16 * 8;
  static constexpr int kJoinBytes = kStages * kStageBytes / kDecWarps;
  static_assert(kResult + 16 * D * 4 + 16 * 4 <= kJoinBytes, "join buffers");
  static_assert(paged_per_sm(D, 8) * (kSmemBytes + 1024) <= 228 * 1024, "shared memory of an SM");
};

// An 8x8 matrix of 16-bit elements, turned over (as ldmatrix lays them out).
__device__ __forceinline__ uint32_t turn_8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// A warp's part of a unit of up to 8 kT rows (query heads of one KV head).
// decode_kernel.cuh has them as the rows of the matrix tiles, which come in
// sixteens; here they are the columns, which come in eights: S^T = K Q^T and
// O^T = V^T P^T, so that 8 heads or fewer take half of the products,
// exponentials and registers. Lane, for each tile of 8: rows 2 c4 and 2 c4 + 1;
// of S^T keys g4 and g4 + 8, of O^T features g4 and g4 + 8 of each 16.
template <int D, int kT>
struct DecodeCols {
  static constexpr int kSteps = D / 16;
  uint32_t qf[kT][kSteps][2];
  float acc[kT][kSteps][4];
  float m[kT][2], l[kT][2];  // l: this lane's keys

  // row(r): the queries of row r, or nullptr past the unit's rows
  template <class R>
  __device__ __forceinline__ void load(R row) {
    const int lane = threadIdx.x & 31, g4 = lane >> 2, c4 = lane & 3;
#pragma unroll
    for (int t = 0; t < kT; ++t) {
      const __nv_bfloat16* q = row(8 * t + g4);
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
#pragma unroll
        for (int e = 0; e < 2; ++e) qf[t][s][e] = q ? *reinterpret_cast<const uint32_t*>(q + s * 16 + e * 8 + 2 * c4) : 0u;
        acc[t][s][0] = acc[t][s][1] = acc[t][s][2] = acc[t][s][3] = 0.f;
      }
      m[t][0] = m[t][1] = -INFINITY;
      l[t][0] = l[t][1] = 0.f;
    }
  }

  // One block of 16 keys, those in [from, to) of it visible. kat(r, p), vat(r, p):
  // shared-memory address of 16-byte piece p of key r. kPieces: bf16 pieces that P has
  // in its product.
  template <int kPieces, class K, class V>
  __device__ __forceinline__ void block(K kat, V vat, int from, int to, float scale_log2) {
    const int lane = threadIdx.x & 31, g4 = lane >> 2;
    // two chains of products for each tile, which are added: half as long
    float sa[kT][4], sb[kT][4];
#pragma unroll
    for (int t = 0; t < kT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) sa[t][e] = sb[t][e] = 0.f;
    {
      const int r = (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        uint32_t kb[4];
        ldmatrix4(kat(r, 2 * s + (lane >> 4)), kb);
#pragma unroll
        for (int t = 0; t < kT; ++t) mma_16x8x16(s & 1 ? sb[t] : sa[t], kb, qf[t][s][0], qf[t][s][1]);
      }
    }
    float alpha[kT][2];
    uint32_t p0[kPieces][kT], p1[kPieces][kT];
    bool moved = false;
#pragma unroll
    for (int t = 0; t < kT; ++t) {
      float x[4];  // [key g4, g4 + 8][row]
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int key = g4 + (e >> 1) * 8;
        x[e] = key >= from && key < to ? (sa[t][e] + sb[t][e]) * scale_log2 : -INFINITY;
      }
      float mx[2] = {fmaxf(x[0], x[2]), fmaxf(x[1], x[3])};
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], o));
        mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], o));
      }
      moved |= mx[0] > m[t][0] || mx[1] > m[t][1];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float mn = fmaxf(m[t][h], mx[h]);
        const float base = mn == -INFINITY ? 0.f : mn;
        alpha[t][h] = ex2_approx(m[t][h] - base);
        m[t][h] = mn;
        x[h] = ex2_approx(x[h] - base);
        x[2 + h] = ex2_approx(x[2 + h] - base);
        l[t][h] = l[t][h] * alpha[t][h] + (x[h] + x[2 + h]);
      }
#pragma unroll
      for (int c = 0; c < kPieces; ++c) {
        const uint32_t lo = pack_bf16x2(x[0], x[1]), hi = pack_bf16x2(x[2], x[3]);
        p0[c][t] = turn_8x8(lo);
        p1[c][t] = turn_8x8(hi);
        x[0] -= __uint_as_float(lo << 16);  // exact
        x[1] -= __uint_as_float(lo & 0xffff0000u);
        x[2] -= __uint_as_float(hi << 16);
        x[3] -= __uint_as_float(hi & 0xffff0000u);
      }
    }
    if (__any_sync(0xffffffffu, moved)) {  // seldom, after a few blocks
#pragma unroll
      for (int t = 0; t < kT; ++t)
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          acc[t][s][0] *= alpha[t][0];
          acc[t][s][1] *= alpha[t][1];
          acc[t][s][2] *= alpha[t][0];
          acc[t][s][3] *= alpha[t][1];
        }
    }
    {
      const int r = (lane & 7) + (lane >> 4) * 8;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        uint32_t vb[4];
        ldmatrix4_trans(vat(r, 2 * s + ((lane >> 3) & 1)), vb);
#pragma unroll
        for (int t = 0; t < kT; ++t)
#pragma unroll
          for (int c = 0; c < kPieces; ++c) mma_16x8x16(acc[t][s], vb, p0[c][t], p1[c][t]);
      }
    }
  }

  // For the join of the CTA's warps: O [16][D], then m[16] and l[16], at jo.
  __device__ __forceinline__ void store(float* jo) {
    const int lane = threadIdx.x & 31, g4 = lane >> 2, c4 = lane & 3;
#pragma unroll
    for (int t = 0; t < kT; ++t) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        l[t][0] += __shfl_xor_sync(0xffffffffu, l[t][0], o);
        l[t][1] += __shfl_xor_sync(0xffffffffu, l[t][1], o);
      }
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e) jo[(8 * t + 2 * c4 + (e & 1)) * D + s * 16 + g4 + (e >> 1) * 8] = acc[t][s][e];
      if (g4 == 0) {
        float* jm = jo + 16 * D;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          jm[8 * t + 2 * c4 + h] = m[t][h];
          jm[16 + 8 * t + 2 * c4 + h] = l[t][h];
        }
      }
    }
  }
};

// What a launch computes: whole sequences; the own keys of sequences whose
// common ones the prefix kernel takes; or both, common keys in its first CTAs.
enum class PagedKind { kWhole, kOwn, kBoth };

// kT: rows of a unit in eights.
template <int D, PagedKind kKind, int kT>
__global__ void __launch_bounds__(kPagedThreads, paged_per_sm(D, 8 * kT))
    cpattn_decode_paged_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                               const __grid_constant__ PagedArgs pa) {
  constexpr bool kParts = kKind != PagedKind::kWhole;  // results go to the join kernel
  constexpr int kRows = 8 * kT, kPieces = kParts ? 1 : 2;
  const DecodeArgs& a = pa.d;
  using C = PagedCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem);
  uint64_t* empty = full + C::kStages;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffFlag);
  if (threadIdx.x == 0) *abort_flag = 0;
  if (threadIdx.x < 2 * C::kStages) {
    mbar_init(&full[threadIdx.x], threadIdx.x < C::kStages ? 1 : kDecWarps);
    fence_mbar_init();
  }
  __syncthreads();
  smem += C::kOffRing;
  // Up to here beside what runs before this call; a kernel behind this one finds
  // that finished. (The own keys' kernel is behind the prefix kernel, which has waited.)
  if constexpr (kKind != PagedKind::kOwn) chain_wait();
  if (kParts || a.nsplit > kDecMaxCluster) chain_next();
  // unit: (sequence or group, KV head, kRows of its rows), then the run of keys
  const bool common = kKind == PagedKind::kBoth && int(blockIdx.x) < pa.common_ctas;
  const int nsplit = common ? pa.sh.fixed_runs : a.nsplit, row_groups = common ? pa.sh.fixed_units : a.row_groups;
  int x = blockIdx.x - (kKind == PagedKind::kBoth && !common ? pa.common_ctas : 0);
  const int split = x % nsplit;
  x /= nsplit;
  const int unit = x;
  const int row0 = x % row_groups * kRows;  // first row of the unit
  x /= row_groups;
  const int kvh = x % a.hkv;
  const int bi = x / a.hkv;  // (of common keys: the group)
  int rows, n, lo = 0, ns = 0;
  int first = bi;  // sequence of row 0
  int named = bi;  // sequence whose table names the pages
  if (common) {
    int size;
    shared_group(pa.sh, bi, first, size);
    n = shared_count(pa.sh, bi);
    rows = size * a.G - row0;
    // the first member that holds all of the common tokens (there are no more than 32)
    const unsigned full_members = __ballot_sync(0xffffffffu, lane < size && a.lengths[first + lane] >= n);
    if (!full_members || rows <= 0) rows = n = 0;
    named = first + (full_members ? __ffs(full_members) - 1 : 0);
  } else {
    rows = a.G - row0;
    n = a.lengths[bi];
    n = n < 0 ? 0 : (n > a.cap ? a.cap : n);
    if constexpr (kParts) {
      lo = shared_seq(pa.sh, bi, n).keys;  // those before it are the group's
    } else {
      lo = a.window > 0 && n > a.window ? n - a.window : 0;  // first key of the window
      ns = a.sinks < lo ? a.sinks : lo;
    }
  }
  rows = rows < kRows ? rows : kRows;
  // rounds that hold visible keys: the first tokens', then the window's
  const int sink_rounds = (ns + kPagedRound - 1) / kPagedRound, lo_round = lo / kPagedRound;
  const int all = sink_rounds + (n > lo ? (n + kPagedRound - 1) / kPagedRound - lo_round : 0);
  // this CTA's run
  const int per = (all + nsplit - 1) / nsplit;
  const int64_t begin64 = int64_t(split) * per;
  const int begin = begin64 < all ? int(begin64) : all;
  const int rounds = all - begin < per ? all - begin : per;
  // Round t of the run: its first key, and the keys [from, to) of it that are seen.
  const auto place = [&](int t, int& from, int& to) {
    const int v = begin + t;
    const bool early = v < sink_rounds;
    const int key0 = (early ? v : lo_round + (v - sink_rounds)) * kPagedRound;
    from = early || lo < key0 ? 0 : lo - key0;
    to = (early ? ns : n) - key0;
    return key0;
  };
  DecodeCols<D, kT> part;
  if (warp == kDecWarps) {
    // ------------------------------------------------------------ copies
    // lane: its box of the keys or of the values
    const int boxes = kPagedRound / pa.box, box = lane % boxes;
    const bool mine = lane < 2 * boxes, values = lane >= boxes;
    const int box_bytes = pa.box * (D * 2);
    const int* table = pa.pg.tables + int64_t(named) * pa.pg.tables_row;
    const CUtensorMap* map = values ? &tmv : &tmk;
    uint8_t* dst = smem + (values ? C::kTileBytes : 0) + box * box_bytes;
    // whether this lane's box of a round holds visible keys, its slot in its page, and the page
    const auto look = [&](int t, int& slot, int& page) {
      if (!mine || t >= rounds) return false;
      int from, to;
      const int key0 = place(t, from, to) + box * pa.box;
      if (to <= box * pa.box || from >= (box + 1) * pa.box) return false;
      const int column = int(unsigned(key0) / unsigned(pa.pg.page_size));
      slot = key0 - column * pa.pg.page_size;
      bounds_ok(key0 >= 0 && key0 < a.cap && slot + pa.box <= pa.pg.page_size && kvh < a.hkv, a.status);
      page = table[column];
      return true;
    };
    int slot = 0, page = 0;
    bool on = look(0, slot, page);
    bool ok = true;
    int t = 0, stage = 0;
    uint32_t turn = 0;  // of the ring
    uint32_t waits = pa.copy_waits;
    for (; t < rounds; ++t) {
      int next_slot = 0, next_page = 0;
      const bool next_on = look(t + 1, next_slot, next_page);
      if (turn > 0) {
        ok = waits-- > 0 && mbar_wait_warp_lean(&empty[stage], (turn - 1) & 1, abort_flag, kWaitLimitNs);
        if (!ok) {
          *abort_flag = 1;
          break;
        }
      }
      if (on) page_ok(page, pa.pg, a.status);  // (a copy from outside of the pool brings zeros)
      const int count = __popc(__ballot_sync(0xffffffffu, on));
      if (lane == 0) mbar_arrive_expect_tx(&full[stage], uint32_t(count * box_bytes));
      __syncwarp();
      if (on) tma_load_5d(dst + stage * C::kStageBytes, map, &full[stage], 0, slot, 0, kvh, page);
      on = next_on;
      slot = next_slot;
      page = next_page;
      if (++stage == C::kStages) {
        stage = 0;
        ++turn;
      }
    }
    // what was asked for arrives before the shared memory is used otherwise, whoever gave up
    for (int u = t > C::kStages ? t - C::kStages : 0; u < t; ++u)
      ok &= mbar_wait_drain_warp(&full[u % C::kStages], (u / C::kStages) & 1, kWaitLimitNs);
    if (!ok && lane == 0) atomicOr(a.status, kStatusCopies);
  } else {
    // ------------------------------------------------------------ products
    part.load([&](int r) -> const __nv_bfloat16* {
      if (r >= rows) return nullptr;
      int seq = first, head = row0 + r;
      if (common) {
        seq += head / a.G;
        head %= a.G;
      }
      bounds_ok(seq < a.b && kvh * a.G + head < a.hq, a.status);
      return a.q + int64_t(seq) * a.q_batch + int64_t(kvh * a.G + head) * D;
    });
    // this warp's 16 keys of a round: in a box, whose features come 64 at a time
    const int half_bytes = pa.box * 128;
    const int mine = (warp * kDecBlock / pa.box) * pa.box * (D * 2) + (warp * kDecBlock % pa.box) * 128;
    int stage = 0;
    uint32_t turn = 0;
    for (int t = 0; t < rounds; ++t) {
      if (!mbar_wait_warp_lean(&full[stage], turn & 1, abort_flag, kWaitLimitNs)) {
        if (lane == 0) atomicOr(a.status, kStatusCopies);
        break;
      }
      uint8_t* sk = smem + stage * C::kStageBytes + mine;
      int from, to;
      place(t, from, to);
      from -= warp * kDecBlock;
      to -= warp * kDecBlock;
      if (from < kDecBlock && to > 0) {
        if (from > 0 || to < kDecBlock) {
          uint8_t* sv = sk + C::kTileBytes;
          for (int x = lane; x < kDecBlock * 8; x += 32)
            if (x / 8 < from || x / 8 >= to)
#pragma unroll
              for (int f = 0; f < D / 64; ++f)
                *reinterpret_cast<uint4*>(sv + f * half_bytes + x * 16) = make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_smem();  // before the copy that takes the stage next
          __syncwarp();
        }
        const auto at = [half_bytes](uint32_t tile) {
          return [tile, half_bytes](int r, int p) {
            return tile + (p / 8) * half_bytes + r * 128 + (((p % 8) ^ (r & 7)) * 16);
          };
        };
        const uint32_t tile = smem_u32(sk);
        part.template block<kPieces>(at(tile), at(tile + C::kTileBytes), from, to, a.scale_log2);
        __syncwarp();  // all lanes have read the stage
      }
      if (lane == 0) mbar_arrive(&empty[stage]);
      if (++stage == C::kStages) {
        stage = 0;
        ++turn;
      }
    }
  }
  __syncthreads();  // the ring is idle: the join reuses it
  if (warp < kDecWarps) part.store(reinterpret_cast<float*>(smem + warp * C::kJoinBytes));
  __syncthreads();
  // The warps' results are joined by weights, formed once for each row.
  const auto of = [&](int w) { return reinterpret_cast<float*>(smem + w * C::kJoinBytes); };
  if (threadIdx.x < rows) {
    const int r = threadIdx.x;
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) mm = fmaxf(mm, of(w)[16 * D + r]);
    const float base = mm == -INFINITY ? 0.f : mm;
    float f[kDecWarps], ll = 0.f;
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) {
      f[w] = ex2_approx(of(w)[16 * D + r] - base);
      ll = fmaf(f[w], of(w)[16 * D + 16 + r], ll);
    }
    const float inv = ll == 0.f ? 0.f : 1.f / ll;
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) of(w)[16 * D + r] = f[w] * inv;
    of(0)[16 * D + 16 + r] = ll == 0.f ? -INFINITY : mm + log2f(ll);
  }
  __syncthreads();
  const int64_t out0 = int64_t(bi) * a.hq + kvh * a.G + row0;  // (not of common keys)
  for (int i = threadIdx.x; i < rows * (D / 4); i += kPagedThreads) {
    const int r = i / (D / 4), c = (i % (D / 4)) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) {
      const float f = of(w)[16 * D + r];
      const float4 y = *reinterpret_cast<const float4*>(of(w) + r * D + c);
      v.x = fmaf(f, y.x, v.x);
      v.y = fmaf(f, y.y, v.y);
      v.z = fmaf(f, y.z, v.z);
      v.w = fmaf(f, y.w, v.w);
    }
    const float l2 = of(0)[16 * D + 16 + r];
    if (!bounds_ok(common ? r < pa.sh.part_rows && unit * nsplit + split < pa.common_ctas : bi < a.b && row0 + r < a.G,
                   a.status))
      continue;
    if (kParts || a.nsplit > kDecMaxCluster) {  // to the join kernel
      const int64_t at = common ? (int64_t(unit) * nsplit + split) * pa.sh.part_rows + r : (out0 + r) * a.nsplit + split;
      *reinterpret_cast<float4*>((common ? pa.sh.part_o : a.part_o) + at * D + c) = v;
      if (c == 0) (common ? pa.sh.part_lse : a.part_lse)[at] = l2;
    } else if (a.nsplit > 1) {  // to the cluster
      float* res = reinterpret_cast<float*>(smem + C::kResult);
      *reinterpret_cast<float4*>(res + r * D + c) = v;
      if (c == 0) res[16 * D + r] = l2;
    } else {
      *reinterpret_cast<uint2*>(a.o + (out0 + r) * D + c) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
      if (c == 0) a.lse[out0 + r] = l2 * kLn2;
    }
  }
  if (!kParts && a.nsplit > 1 && a.nsplit <= kDecMaxCluster) {
    // the cluster's CTAs are the runs of one unit: each joins its share of the features
    cluster_sync();
    for (int i = split * kPagedThreads + threadIdx.x; i < rows * (D / 2); i += a.nsplit * kPagedThreads) {
      const int r = i / (D / 2), c = (i % (D / 2)) * 2;
      const DecodeResult v = decode_join_cluster<D>(smem_u32(smem) + C::kResult, a.nsplit, r, c);
      *reinterpret_cast<uint32_t*>(a.o + (out0 + r) * D + c) = pack_bf16x2(v.o0, v.o1);
      if (c == 0) a.lse[out0 + r] = v.l2 * kLn2;
    }
    cluster_sync();  // no CTA leaves while another still reads its results
  }
  // This kernel is over only when the prefix kernel is, beside which it may run: the join waits for this one.
  if (kKind == PagedKind::kOwn && blockIdx.x == gridDim.x - 1) chain_wait();
}

// Joins the results of a row's own keys (or of all its keys) and of its group's, kWarps warps to a row
// (sequence, query head). Results are numbered, own ones first; warp w takes w, w + kWarps
// and so on, a batch at a time, whose values are on their way before their
// weights are formed. With up to 8 results a warp does by itself; more of them
// for four warps (30 results of 128 rows: 6 us by one warp, whose loads wait for
// one another, 2.5 by four).
template <int D, int kWarps>
__global__ void __launch_bounds__(128) cpattn_shared_join_kernel(const __grid_constant__ PagedArgs pa) {
  const DecodeArgs& a = pa.d;
  constexpr int kPer = D / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = int64_t(blockIdx.x) * (4 / kWarps) + warp / kWarps;
  const bool live = row < int64_t(a.b) * a.hq;
  if (kWarps == 1 && !live) return;
  const int bi = live ? int(row / a.hq) : 0, h = live ? int(row - int64_t(bi) * a.hq) : 0;
  const int kvh = h / a.G;
  SharedSeq mate = {};
  if (pa.sh.groups > 0) {  // (0: whole sequences)
    int n = a.lengths[bi];
    n = n < 0 ? 0 : (n > a.cap ? a.cap : n);
    mate = shared_seq(pa.sh, bi, n);
  }
  chain_wait();
  int64_t at = 0;
  if (mate.keys > 0) {
    shared_runs(pa.sh, mate);
    at = shared_at(pa.sh, mate, kvh, h - kvh * a.G);
    if (!bounds_ok(at + int64_t(mate.at.runs - 1) * pa.sh.part_rows < int64_t(pa.sh.ctas) * pa.sh.part_rows, a.status))
      mate.keys = 0;
  }
  const int count = a.nsplit + (mate.keys > 0 ? mate.at.runs : 0);
  const auto place = [&](int i, const float*& l2) {  // of result i: its values (this lane's)
    const bool own = i < a.nsplit;
    const int64_t x = own ? row * a.nsplit + i : at + int64_t(i - a.nsplit) * pa.sh.part_rows;
    l2 = (own ? a.part_lse : pa.sh.part_lse) + x;
    return (own ? a.part_o : pa.sh.part_o) + x * D + lane * kPer;
  };
  float m = -INFINITY, l = 0.f, o[kPer] = {};
  for (int i0 = warp % kWarps; i0 < count; i0 += kWarps * kJoinBatch) {
    float v[kJoinBatch][kPer], l2[kJoinBatch];
#pragma unroll
    for (int k = 0; k < kJoinBatch; ++k) {
      const int i = i0 + k * kWarps;
      l2[k] = -INFINITY;
#pragma unroll
      for (int e = 0; e < kPer; ++e) v[k][e] = 0.f;
      if (i < count) {
        const float* pl;
        const float* p = place(i, pl);
        l2[k] = __ldcg(pl);
        if constexpr (kPer == 4) {
          const float4 f = __ldcg(reinterpret_cast<const float4*>(p));
          v[k][0] = f.x, v[k][1] = f.y, v[k][2] = f.z, v[k][3] = f.w;
        } else {
          const float2 f = __ldcg(reinterpret_cast<const float2*>(p));
          v[k][0] = f.x, v[k][1] = f.y;
        }
      }
    }
    float mm = m;
#pragma unroll
    for (int k = 0; k < kJoinBatch; ++k) mm = fmaxf(mm, l2[k]);
    const float base = mm == -INFINITY ? 0.f : mm;
    const float old = ex2_approx(m - base);
    m = mm;
    l *= old;
#pragma unroll
    for (int e = 0; e < kPer; ++e) o[e] *= old;
#pragma unroll
    for (int k = 0; k < kJoinBatch; ++k) {
      const float w = ex2_approx(l2[k] - base);
      l += w;
#pragma unroll
      for (int e = 0; e < kPer; ++e) o[e] = fmaf(w, v[k][e], o[e]);
    }
  }
  if constexpr (kWarps > 1) {
    __shared__ float sm[kWarps], sl[kWarps];
    __shared__ float so[kWarps][32][kPer];
    if (lane == 0) {
      sm[warp] = m;
      sl[warp] = l;
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e) so[warp][lane][e] = o[e];
    __syncthreads();
    if (warp > 0 || !live) return;
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      const float mm = fmaxf(m, sm[w]), base = mm == -INFINITY ? 0.f : mm;
      const float f0 = ex2_approx(m - base), f1 = ex2_approx(sm[w] - base);
      m = mm;
      l = l * f0 + sl[w] * f1;
#pragma unroll
      for (int e = 0; e < kPer; ++e) o[e] = o[e] * f0 + so[w][lane][e] * f1;
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int i = 0; i < kPer; i += 2)
    *reinterpret_cast<uint32_t*>(a.o + row * D + lane * kPer + i) = pack_bf16x2(o[i] * inv, o[i + 1] * inv);
  if (lane == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

}  // namespace cpattn
