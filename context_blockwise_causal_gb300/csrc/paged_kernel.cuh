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
#pragma once
#include <cuda_bf16.h>

#include <cstdint>
#include <type_traits>

#include "decode_kernel.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace cpattn {

constexpr unsigned int kStatusCopies = 1u << 4;  // copies of a paged decode did not arrive in time
constexpr int kPagedThreads = (kDecWarps + 1) * 32;

struct PagedArgs {
  DecodeArgs d;  // k and v are not used (the copies' descriptors name the pools)
  PagedPlace pg;
  SharedPlan sh;  // kOwn
  float* own_o;   // kOwn: [b, hq, D] normalised
  float* own_lse; // [b, hq], base 2
  int box;  // tokens of a copy: gcd(page_size, 32)
};

constexpr int kPagedRound = kDecWarps * kDecBlock;  // keys of a round

template <int D>
struct PagedCfg {
  static constexpr int kTileBytes = kPagedRound * D * 2;  // keys or values of a round
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kStages = 3;
  // CTAs that fit an SM with 8 heads to a unit. (d = 64 with six stages and two of
  // them: 37 sequences of up to 2928 keys, 2 KV heads, 12.4 us instead of 10.7; 64 of
  // 8192, 8 KV heads, 135 instead of 120.)
  static constexpr int kPerSm = D == 128 ? 2 : 4;
  // barriers (full and empty per stage) and the flag come first, the ring (1024-byte aligned) behind them
  static constexpr int kOffFlag = 2 * kStages * 8;
  static constexpr int kOffRing = 1024;
  static constexpr int kSmemBytes = kOffRing + kStages * kStageBytes + 1024;  // + alignment slack
  // the join of the warps reuses the ring, kJoinBytes for each: O and pairs, as in DecodeCfg, and the CTA's result
  static constexpr int kResult = 16 * D * 4 + 16 * 8;
  static constexpr int kJoinBytes = kStages * kStageBytes / kDecWarps;
  static_assert(kResult + 16 * D * 4 + 16 * 4 <= kJoinBytes, "join buffers");
};

// An 8x8 matrix of 16-bit elements, turned over (as ldmatrix lays them out).
__device__ __forceinline__ uint32_t turn_8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// A warp's part of a unit of up to 8 query heads. Where decode_kernel.cuh has
// the heads as the rows of the matrix tiles, which come in sixteens, here they
// are the columns, which come in eights: S^T = K Q^T and O^T = V^T P^T, half of
// the products, exponentials and registers. Lane: heads 2 c4 and 2 c4 + 1; of S^T
// keys g4 and g4 + 8, of O^T features g4 and g4 + 8 of each 16.
template <int D>
struct DecodeCols {
  static constexpr int kHeads = 8, kSteps = D / 16;
  uint32_t qf[kSteps][2];
  float acc[kSteps][4];
  float m[2], l[2];  // l: this lane's keys

  __device__ __forceinline__ void load(const __nv_bfloat16* qp, int rows) {
    const int lane = threadIdx.x & 31, g4 = lane >> 2, c4 = lane & 3;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
        qf[s][e] = g4 < rows ? *reinterpret_cast<const uint32_t*>(qp + int64_t(g4) * D + s * 16 + e * 8 + 2 * c4) : 0u;
      acc[s][0] = acc[s][1] = acc[s][2] = acc[s][3] = 0.f;
    }
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
  }

  // As DecodeRows::block.
  template <class K, class V>
  __device__ __forceinline__ void block(K kat, V vat, int from, int to, float scale_log2) {
    const int lane = threadIdx.x & 31, g4 = lane >> 2;
    // two chains of products, which are added: half as long
    float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
    {
      const int r = (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        uint32_t kb[4];
        ldmatrix4(kat(r, 2 * s + (lane >> 4)), kb);
        mma_16x8x16(s & 1 ? s1 : s0, kb, qf[s][0], qf[s][1]);
      }
    }
    float x[4];  // [key g4, g4 + 8][head]
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int key = g4 + (e >> 1) * 8;
      x[e] = key >= from && key < to ? (s0[e] + s1[e]) * scale_log2 : -INFINITY;
    }
    float mx[2] = {fmaxf(x[0], x[2]), fmaxf(x[1], x[3])}, alpha[2];
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], o));
      mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], o));
    }
    const bool moved = mx[0] > m[0] || mx[1] > m[1];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float mn = fmaxf(m[h], mx[h]);
      const float base = mn == -INFINITY ? 0.f : mn;
      alpha[h] = ex2_approx(m[h] - base);
      m[h] = mn;
      x[h] = ex2_approx(x[h] - base);
      x[2 + h] = ex2_approx(x[2 + h] - base);
      l[h] = l[h] * alpha[h] + (x[h] + x[2 + h]);
    }
    const uint32_t p0 = turn_8x8(pack_bf16x2(x[0], x[1])), p1 = turn_8x8(pack_bf16x2(x[2], x[3]));
    if (__any_sync(0xffffffffu, moved)) {  // seldom, after a few blocks
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        acc[s][0] *= alpha[0];
        acc[s][1] *= alpha[1];
        acc[s][2] *= alpha[0];
        acc[s][3] *= alpha[1];
      }
    }
    {
      const int r = (lane & 7) + (lane >> 4) * 8;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        uint32_t vb[4];
        ldmatrix4_trans(vat(r, 2 * s + ((lane >> 3) & 1)), vb);
        mma_16x8x16(acc[s], vb, p0, p1);
      }
    }
  }

  // As DecodeRows::store (8 rows of the 16).
  __device__ __forceinline__ void store(float* jo) {
    const int lane = threadIdx.x & 31, g4 = lane >> 2, c4 = lane & 3;
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      l[0] += __shfl_xor_sync(0xffffffffu, l[0], o);
      l[1] += __shfl_xor_sync(0xffffffffu, l[1], o);
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int e = 0; e < 4; ++e) jo[(2 * c4 + (e & 1)) * D + s * 16 + g4 + (e >> 1) * 8] = acc[s][e];
    if (g4 == 0) {
      float* jm = jo + 16 * D;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        jm[2 * c4 + h] = m[h];
        jm[16 + 2 * c4 + h] = l[h];
      }
    }
  }
};

// kHeads: query heads of a unit, 8 (DecodeCols) or 16 (DecodeRows).
template <int D, bool kOwn, int kHeads>
__global__ void __launch_bounds__(kPagedThreads, kHeads == 8 ? PagedCfg<D>::kPerSm : 2)
    cpattn_decode_paged_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                               const __grid_constant__ PagedArgs pa) {
  const DecodeArgs& a = pa.d;
  if (kOwn || a.nsplit > kDecMaxCluster) chain_next();
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
  // unit: (batch, KV head, group of kHeads query heads), then the run of keys
  int x = blockIdx.x;
  const int split = x % a.nsplit;
  x /= a.nsplit;
  const int rg = x % a.row_groups;
  x /= a.row_groups;
  const int kvh = x % a.hkv;
  const int bi = x / a.hkv;
  const int rows = a.G - rg * kHeads < kHeads ? a.G - rg * kHeads : kHeads;  // query heads of this CTA
  const int h0 = kvh * a.G + rg * kHeads;

  int n = a.lengths[bi];
  n = n < 0 ? 0 : (n > a.cap ? a.cap : n);
  int lo = a.window > 0 && n > a.window ? n - a.window : 0;  // first key of the window
  if constexpr (kOwn) lo = shared_seq(pa.sh, bi, n).keys;    // those before it are the prefix kernel's
  const int ns = kOwn ? 0 : (a.sinks < lo ? a.sinks : lo);
  // rounds that hold visible keys: the first tokens', then the window's
  const int sink_rounds = (ns + kPagedRound - 1) / kPagedRound, lo_round = lo / kPagedRound;
  const int all = sink_rounds + (n > lo ? (n + kPagedRound - 1) / kPagedRound - lo_round : 0);
  // this CTA's run
  const int per = (all + a.nsplit - 1) / a.nsplit;
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
  std::conditional_t<kHeads == 8, DecodeCols<D>, DecodeRows<D>> part;
  if (warp == kDecWarps) {
    // ------------------------------------------------------------ copies
    // lane: its box of the keys or of the values
    const int boxes = kPagedRound / pa.box, box = lane % boxes;
    const bool mine = lane < 2 * boxes, values = lane >= boxes;
    const int box_bytes = pa.box * (D * 2);
    const int* table = pa.pg.tables + int64_t(bi) * pa.pg.tables_row;
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
    for (; t < rounds; ++t) {
      int next_slot = 0, next_page = 0;
      const bool next_on = look(t + 1, next_slot, next_page);
      if (turn > 0 && !(ok = mbar_wait_warp_lean(&empty[stage], (turn - 1) & 1, abort_flag, kWaitLimitNs))) break;
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
    if (!ok) {  // gave up: what was asked for arrives before the shared memory is used otherwise
      if (lane == 0) atomicOr(a.status, kStatusCopies);
      for (int u = t > C::kStages ? t - C::kStages : 0; u < t; ++u)
        mbar_wait_drain_warp(&full[u % C::kStages], (u / C::kStages) & 1, kWaitLimitNs);
    }
  } else {
    // ------------------------------------------------------------ products
    part.load(a.q + int64_t(bi) * a.q_batch + int64_t(h0) * D, rows);
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
        part.block(at(tile), at(tile + C::kTileBytes), from, to, a.scale_log2);
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
  const auto put = [&](int64_t row, int c, const DecodeResult& r) {
    if constexpr (kOwn) {
      *reinterpret_cast<float2*>(pa.own_o + row * D + c) = make_float2(r.o0, r.o1);
      if (c == 0) pa.own_lse[row] = r.l2;
    } else {
      *reinterpret_cast<uint32_t*>(a.o + row * D + c) = pack_bf16x2(r.o0, r.o1);
      if (c == 0) a.lse[row] = r.l2 * kLn2;
    }
  };
  for (int i = threadIdx.x; i < rows * (D / 2); i += kPagedThreads) {
    const int r = i / (D / 2), c = (i % (D / 2)) * 2;
    const DecodeResult v = decode_join_warps<D>(smem, C::kJoinBytes, r, c);
    const int64_t row = int64_t(bi) * a.hq + h0 + r;
    if (!bounds_ok(bi < a.b && h0 + r < a.hq, a.status)) continue;
    if (a.nsplit == 1) {
      put(row, c, v);
    } else if (a.nsplit <= kDecMaxCluster) {
      float* res = reinterpret_cast<float*>(smem + C::kResult);
      *reinterpret_cast<float2*>(res + r * D + c) = make_float2(v.o0, v.o1);
      if (c == 0) res[16 * D + r] = v.l2;
    } else {
      const int64_t pr = row * a.nsplit + split;
      *reinterpret_cast<float2*>(a.part_o + pr * D + c) = make_float2(v.o0, v.o1);
      if (c == 0) a.part_lse[pr] = v.l2;
    }
  }
  if (a.nsplit > 1 && a.nsplit <= kDecMaxCluster) {
    // the cluster's CTAs are the runs of one unit: each joins its share of the features
    cluster_sync();
    for (int i = split * kPagedThreads + threadIdx.x; i < rows * (D / 2); i += a.nsplit * kPagedThreads) {
      const int r = i / (D / 2), c = (i % (D / 2)) * 2;
      put(int64_t(bi) * a.hq + h0 + r, c, decode_join_cluster<D>(smem_u32(smem) + C::kResult, a.nsplit, r, c));
    }
    cluster_sync();  // no CTA leaves while another still reads its results
  }
  // This kernel is over only when the prefix kernel is, beside which it may run: the join waits for this one.
  if (kOwn && blockIdx.x == gridDim.x - 1) chain_wait();
}

// Joins a row's own keys and its group's: one warp per (sequence, query head).
template <int D>
__global__ void __launch_bounds__(128) cpattn_shared_join_kernel(const __grid_constant__ PagedArgs pa) {
  const DecodeArgs& a = pa.d;
  constexpr int kPer = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t row = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (row >= int64_t(a.b) * a.hq) return;
  const int bi = int(row / a.hq), h = int(row - int64_t(bi) * a.hq);
  const int kvh = h / a.G;
  int n = a.lengths[bi];
  n = n < 0 ? 0 : (n > a.cap ? a.cap : n);
  SharedSeq mate = shared_seq(pa.sh, bi, n);
  chain_wait();
  const float own = __ldcg(pa.own_lse + row);
  float o[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) o[i] = __ldcg(pa.own_o + row * D + lane * kPer + i);
  int64_t at = 0;
  if (mate.keys > 0) {
    shared_runs(pa.sh, mate);
    at = shared_at(pa.sh, mate, kvh, h - kvh * a.G);
    if (!bounds_ok(at + int64_t(mate.at.runs - 1) * pa.sh.part_rows < int64_t(pa.sh.ctas) * pa.sh.part_rows, a.status)) return;
  }
  const float* pl = pa.sh.part_lse + at;
  const float* po = pa.sh.part_o + at * D + lane * kPer;
  const int64_t step = pa.sh.part_rows;
  float mm = own;
  for (int s = lane; s < mate.at.runs; s += 32) mm = fmaxf(mm, __ldcg(pl + s * step));
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, x));
  const float base = mm == -INFINITY ? 0.f : mm;
  float ll = ex2_approx(own - base);
#pragma unroll
  for (int i = 0; i < kPer; ++i) o[i] *= ll;
  for (int s0 = 0; s0 < mate.at.runs; s0 += 32) {
    const float mine = s0 + lane < mate.at.runs ? ex2_approx(__ldcg(pl + (s0 + lane) * step) - base) : 0.f;
    const int count = mate.at.runs - s0 < 32 ? mate.at.runs - s0 : 32;
#pragma unroll 8
    for (int s = 0; s < count; ++s) {
      const float w = __shfl_sync(0xffffffffu, mine, s);
      const float* p = po + (s0 + s) * step * D;
      float v[kPer];
      if constexpr (kPer == 4) {
        const float4 f = __ldcg(reinterpret_cast<const float4*>(p));
        v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
      } else {
        const float2 f = __ldcg(reinterpret_cast<const float2*>(p));
        v[0] = f.x, v[1] = f.y;
      }
      ll += w;
#pragma unroll
      for (int i = 0; i < kPer; ++i) o[i] = fmaf(w, v[i], o[i]);
    }
  }
  const float inv = ll == 0.f ? 0.f : 1.f / ll;
#pragma unroll
  for (int i = 0; i < kPer; i += 2)
    *reinterpret_cast<uint32_t*>(a.o + row * D + lane * kPer + i) = pack_bf16x2(o[i] * inv, o[i + 1] * inv);
  if (lane == 0) a.lse[row] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
}

}  // namespace cpattn
