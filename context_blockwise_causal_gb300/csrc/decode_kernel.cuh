// Attention of one new token per sequence over a K/V cache, whole or with a
// sliding window and visible first tokens.
//
// A sequence of n tokens (the new one included) sees the keys
//     [0, min(sinks, n - window))  and  [max(0, n - window), n)
// (window 0: all of [0, n)); o = softmax(scale q K^T) V over them, and their
// log-sum-exp. n = 0 gives o = 0 and L = -inf.
//
// HBM-bound: the visible K and V are read once, 4 d bytes per key and KV head
// for 4 d G flops (G query heads share a KV head), and nothing else counts.
// The G queries of a KV head are the rows of one 16-row matrix tile, so the
// matrix unit does the products whatever G is and the cache is read once for
// all of them; with fewer than 16 rows of queries an M = 128 tcgen05 tile
// would add shared-memory staging of P for nothing, the warp-level m16n8k16
// instruction takes both operands from registers and keeps up with the loads.
//
// The visible keys (numbered without the gap between first tokens and window)
// are cut into nsplit runs, one CTA each, and a run into 16-key blocks dealt
// to the CTA's warps in turn. Every warp keeps its own ring of blocks in
// shared memory, filled by 16-byte asynchronous copies two blocks ahead, and
// its own running maximum, sum and O, so warps never wait for one another
// until the end. Keys past the run are never read: their slots are filled
// with zeros and their scores masked, whatever the cache holds there. Warps
// and then runs are joined through their log-sum-exp in a fixed order. Up to
// 8 runs are the CTAs of one cluster, which read one another's results from
// shared memory: one launch and no workspace. More runs (a few very long
// sequences) go through device memory and a second kernel.
//
// Measured, d128: 64 sequences of up to 16384 tokens, h32/8, window 4096: 154
// us; 16 of up to 65537, h64/8, whole: 447 to 488 us (both at the measured copy
// bandwidth and a few percent above it, as reads alone may be); one sequence,
// h32/8, window 1024: 6.9 us, a launch and three rounds of loads.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "ptx.cuh"

namespace cpattn {

constexpr int kDecWarps = 4;
constexpr int kDecStages = 3;
constexpr int kDecBlock = 16;  // keys per block
constexpr int kDecMaxCluster = 8;  // the portable cluster size
constexpr int kDecMaxSplit = 64;

struct DecodeArgs {
  const __nv_bfloat16* q;  // [b, hq, D], batch stride q_batch
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const int* lengths;      // [b] device
  __nv_bfloat16* o;        // [b, hq, D]
  float* lse;              // [b, hq]
  float* part_o;           // nsplit > kDecMaxCluster: [b, hq, nsplit, D] normalised
  float* part_lse;         // [b, hq, nsplit], base-2
  int64_t q_batch;
  int64_t k_batch, k_token, k_head, v_batch, v_token, v_head;  // elements
  int b, hq, hkv, G, cap, window, sinks;
  int row_groups;  // groups of 16 query heads per KV head
  int nsplit;
  float scale_log2;
  unsigned int* status;
};

template <int D>
struct DecodeCfg {
  static constexpr int kTileBytes = kDecBlock * D * 2;        // K or V of a block
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kWarpBytes = kDecStages * kStageBytes;
  static constexpr int kSmemBytes = kDecWarps * kWarpBytes;
  // the join of the warps reuses the rings: 16 x D fp32 and 16 pairs per
  // warp; in warp 0's, behind it, the CTA's result for the cluster's join
  static constexpr int kResult = 16 * D * 4 + 16 * 8;
  static_assert(kResult + 16 * D * 4 + 16 * 4 <= kWarpBytes, "join buffers");
};

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// D (16x8 fp32) += A (16x16 bf16) B (16x8 bf16)
__device__ __forceinline__ void mma_16x8x16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A shared-memory address of CTA `rank` of the cluster, and loads through it.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float cluster_ld(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float2 cluster_ld2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
// All threads of the cluster's CTAs (a hardware barrier: they run together).
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

template <int D>
__global__ void __launch_bounds__(kDecWarps * 32) cpattn_decode_kernel(const DecodeArgs a) {
  if (a.nsplit > kDecMaxCluster) chain_next();
  using C = DecodeCfg<D>;
  constexpr int kPieces = D / 8;          // 16-byte pieces of a row
  constexpr int kSteps = D / 16;          // 16-feature steps
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g4 = lane >> 2, c4 = lane & 3;
  // unit: (batch, KV head, group of 16 query rows), then the run of keys
  int x = blockIdx.x;
  const int split = x % a.nsplit;
  x /= a.nsplit;
  const int rg = x % a.row_groups;
  x /= a.row_groups;
  const int kvh = x % a.hkv;
  const int bi = x / a.hkv;
  const int rows = a.G - rg * 16 < 16 ? a.G - rg * 16 : 16;  // query heads of this CTA
  const int h0 = kvh * a.G + rg * 16;

  int n = a.lengths[bi];
  n = n < 0 ? 0 : (n > a.cap ? a.cap : n);
  const int lo = a.window > 0 && n > a.window ? n - a.window : 0;  // first key of the window
  const int ns = a.sinks < lo ? a.sinks : lo;
  const int nk = ns + (n - lo);  // visible keys
  // this CTA's run: whole rounds of the warps' blocks
  constexpr int kRound = kDecWarps * kDecBlock;
  const int per = ((nk + a.nsplit - 1) / a.nsplit + kRound - 1) / kRound * kRound;
  const int64_t begin64 = int64_t(split) * per;
  const int begin = begin64 < nk ? int(begin64) : nk;
  const int end = nk - begin < per ? nk : begin + per;
  const int blocks = (end - begin + kDecBlock - 1) / kDecBlock;
  const int mine = blocks > warp ? (blocks - warp + kDecWarps - 1) / kDecWarps : 0;  // blocks of this warp

  const __nv_bfloat16* kp = a.k + int64_t(bi) * a.k_batch + int64_t(kvh) * a.k_head;
  const __nv_bfloat16* vp = a.v + int64_t(bi) * a.v_batch + int64_t(kvh) * a.v_head;
  const uint32_t ring = smem_u32(smem) + warp * C::kWarpBytes;

  // Copies block i of this warp into its stage: lane -> piece lane % kPieces
  // of row lane / kPieces (+ 32 / kPieces per step); piece p of row r sits at
  // p ^ (r & 7), so ldmatrix's eight rows fall into different banks.
  auto load = [&](int i) {
    const int v0 = begin + (warp + i * kDecWarps) * kDecBlock;
    const uint32_t dst = ring + (i % kDecStages) * C::kStageBytes;
    constexpr int kRowsPerStep = 32 / kPieces;
    const int p = lane % kPieces;
#pragma unroll
    for (int s = 0; s < kDecBlock / kRowsPerStep; ++s) {
      const int r = s * kRowsPerStep + lane / kPieces;
      const int vis = v0 + r;
      const bool valid = vis < end;
      int key = vis < ns ? vis : lo + (vis - ns);
      if (!valid) key = 0;
      bounds_ok(key >= 0 && key < a.cap, a.status);
      const uint32_t off = uint32_t(r * D * 2 + ((p ^ (r & 7)) * 16));
      cp_async16(dst + off, kp + int64_t(key) * a.k_token + p * 8, valid);
      cp_async16(dst + C::kTileBytes + off, vp + int64_t(key) * a.v_token + p * 8, valid);
    }
  };
  // (a group is committed even when there is nothing left to load, so that
  // the wait counts blocks)
#pragma unroll
  for (int i = 0; i < kDecStages - 1; ++i) {
    if (i < mine) load(i);
    cp_async_commit();
  }

  // Q fragments (A operand): rows g4 and g4 + 8; rows past the group's heads are zero
  uint32_t qf[kSteps][4];
  {
    const __nv_bfloat16* qp = a.q + int64_t(bi) * a.q_batch + int64_t(h0) * D;
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = g4 + (e & 1) * 8, c = s * 16 + (e >> 1) * 8 + 2 * c4;
        qf[s][e] = r < rows ? *reinterpret_cast<const uint32_t*>(qp + int64_t(r) * D + c) : 0u;
      }
  }
  float acc[D / 8][4];
#pragma unroll
  for (int i = 0; i < D / 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // rows g4, g4 + 8 (l: this thread's columns)

  for (int i = 0; i < mine; ++i) {
    cp_async_wait<kDecStages - 2>();
    __syncwarp();  // every lane's copies of block i have landed; stage (i - 1) has been read by all
    if (i + kDecStages - 1 < mine) load(i + kDecStages - 1);
    cp_async_commit();
    const uint32_t sk = ring + (i % kDecStages) * C::kStageBytes, sv = sk + C::kTileBytes;
    // S = Q K^T: two 8-key column tiles. ldmatrix: lanes 0-7 and 8-15 address
    // keys 0-7 at features +0 and +8, lanes 16-31 keys 8-15.
    float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
    {
      const int r = (lane & 7) + ((lane >> 4) << 3);
      const uint32_t row = sk + r * D * 2;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int p = 2 * s + ((lane >> 3) & 1);
        uint32_t kb[4];
        ldmatrix4(row + ((p ^ (r & 7)) * 16), kb);
        mma_16x8x16(s0, qf[s], kb[0], kb[1]);
        mma_16x8x16(s1, qf[s], kb[2], kb[3]);
      }
    }
    // columns 2*c4, +1 (s0: keys 0-7, s1: keys 8-15); [0], [1]: row g4, [2], [3]: row g4 + 8
    const int left = end - (begin + (warp + i * kDecWarps) * kDecBlock);
    float sc[8] = {s0[0], s0[1], s1[0], s1[1], s0[2], s0[3], s1[2], s1[3]};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int col = 2 * c4 + (e & 1) + ((e >> 1) & 1) * 8;
      sc[e] = col < left ? sc[e] * a.scale_log2 : -INFINITY;
    }
    float alpha[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float mx = fmaxf(fmaxf(sc[4 * r], sc[4 * r + 1]), fmaxf(sc[4 * r + 2], sc[4 * r + 3]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float mn = fmaxf(m[r], mx);
      const float base = mn == -INFINITY ? 0.f : mn;
      alpha[r] = ex2_approx(m[r] - base);
      m[r] = mn;
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sc[4 * r + e] = ex2_approx(sc[4 * r + e] - base);
        sum += sc[4 * r + e];
      }
      l[r] = l[r] * alpha[r] + sum;
    }
    const uint32_t pf[4] = {pack_bf16x2(sc[0], sc[1]), pack_bf16x2(sc[4], sc[5]), pack_bf16x2(sc[2], sc[3]),
                            pack_bf16x2(sc[6], sc[7])};
    // O = alpha O + P V: V rows (keys) through transposing loads; lanes 0-15
    // address the 16 keys at features +0, lanes 16-31 at +8
    {
      const int r = lane & 15;
      const uint32_t row = sv + r * D * 2;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int p = 2 * s + (lane >> 4);
        uint32_t vb[4];
        ldmatrix4_trans(row + ((p ^ (r & 7)) * 16), vb);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          float(&c)[4] = acc[2 * s + t];
          c[0] *= alpha[0];
          c[1] *= alpha[0];
          c[2] *= alpha[1];
          c[3] *= alpha[1];
          mma_16x8x16(c, pf, vb[2 * t], vb[2 * t + 1]);
        }
      }
    }
    __syncwarp();  // all lanes have read the stage before the next turn refills it
  }
  cp_async_wait<0>();
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
  }
  __syncthreads();  // the rings are idle: reuse them for the join
  float* jo = reinterpret_cast<float*>(smem + warp * C::kWarpBytes);  // [16][D], then m[16], l[16]
  float* jm = jo + 16 * D;
#pragma unroll
  for (int t = 0; t < D / 8; ++t) {
    *reinterpret_cast<float2*>(jo + g4 * D + t * 8 + 2 * c4) = make_float2(acc[t][0], acc[t][1]);
    *reinterpret_cast<float2*>(jo + (g4 + 8) * D + t * 8 + 2 * c4) = make_float2(acc[t][2], acc[t][3]);
  }
  if (c4 == 0) {
    jm[g4] = m[0];
    jm[g4 + 8] = m[1];
    jm[16 + g4] = l[0];
    jm[16 + g4 + 8] = l[1];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < rows * (D / 2); i += kDecWarps * 32) {
    const int r = i / (D / 2), c = (i % (D / 2)) * 2;
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w)
      mm = fmaxf(mm, reinterpret_cast<const float*>(smem + w * C::kWarpBytes)[16 * D + r]);
    const float base = mm == -INFINITY ? 0.f : mm;
    float ll = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) {
      const float* p = reinterpret_cast<const float*>(smem + w * C::kWarpBytes);
      const float f = ex2_approx(p[16 * D + r] - base);
      ll = fmaf(f, p[16 * D + 16 + r], ll);
      o0 = fmaf(f, p[r * D + c], o0);
      o1 = fmaf(f, p[r * D + c + 1], o1);
    }
    const float inv = ll == 0.f ? 0.f : 1.f / ll;
    const int64_t row = int64_t(bi) * a.hq + h0 + r;
    const float l2 = ll == 0.f ? -INFINITY : mm + log2f(ll);
    if (!bounds_ok(bi < a.b && h0 + r < a.hq, a.status)) continue;
    if (a.nsplit == 1) {
      *reinterpret_cast<uint32_t*>(a.o + row * D + c) = pack_bf16x2(o0 * inv, o1 * inv);
      if (c == 0) a.lse[row] = l2 * 0.69314718055994530942f;
    } else if (a.nsplit <= kDecMaxCluster) {
      float* res = reinterpret_cast<float*>(smem + C::kResult);
      *reinterpret_cast<float2*>(res + r * D + c) = make_float2(o0 * inv, o1 * inv);
      if (c == 0) res[16 * D + r] = l2;
    } else {
      const int64_t pr = row * a.nsplit + split;
      *reinterpret_cast<float2*>(a.part_o + pr * D + c) = make_float2(o0 * inv, o1 * inv);
      if (c == 0) a.part_lse[pr] = l2;
    }
  }
  if (a.nsplit == 1 || a.nsplit > kDecMaxCluster) return;
  // The cluster's CTAs are the runs of one unit, in order: each joins its
  // share of the unit's features.
  cluster_sync();
  const uint32_t res = smem_u32(smem) + C::kResult;
  for (int i = split * kDecWarps * 32 + threadIdx.x; i < rows * (D / 2); i += a.nsplit * kDecWarps * 32) {
    const int r = i / (D / 2), c = (i % (D / 2)) * 2;
    float mm = -INFINITY;
#pragma unroll 4
    for (int s = 0; s < a.nsplit; ++s) mm = fmaxf(mm, cluster_ld(cluster_addr(res + (16 * D + r) * 4, s)));
    const float base = mm == -INFINITY ? 0.f : mm;
    float ll = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll 4
    for (int s = 0; s < a.nsplit; ++s) {
      const float w = ex2_approx(cluster_ld(cluster_addr(res + (16 * D + r) * 4, s)) - base);
      const float2 o = cluster_ld2(cluster_addr(res + (r * D + c) * 4, s));
      ll += w;
      o0 = fmaf(w, o.x, o0);
      o1 = fmaf(w, o.y, o1);
    }
    const float inv = ll == 0.f ? 0.f : 1.f / ll;
    const int64_t row = int64_t(bi) * a.hq + h0 + r;
    *reinterpret_cast<uint32_t*>(a.o + row * D + c) = pack_bf16x2(o0 * inv, o1 * inv);
    if (c == 0) a.lse[row] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * 0.69314718055994530942f;
  }
  cluster_sync();  // no CTA leaves while another still reads its results
}

// Joins the runs of a row: one warp per (sequence, query head).
template <int D>
__global__ void __launch_bounds__(128) cpattn_decode_join_kernel(const DecodeArgs a) {
  chain_wait();
  const int lane = threadIdx.x & 31;
  const int64_t row = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (row >= int64_t(a.b) * a.hq) return;
  const float* pl = a.part_lse + row * a.nsplit;
  // a lane's runs: lane and lane + 32 (nsplit <= 64)
  const float l0 = lane < a.nsplit ? pl[lane] : -INFINITY, l1 = lane + 32 < a.nsplit ? pl[lane + 32] : -INFINITY;
  float mm = fmaxf(l0, l1);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
  const float base = mm == -INFINITY ? 0.f : mm;
  const float w0 = ex2_approx(l0 - base), w1 = ex2_approx(l1 - base);
  float ll = w0 + w1;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ll += __shfl_xor_sync(0xffffffffu, ll, o);
  constexpr int kPer = D / 32;
  float acc[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
#pragma unroll 8
  for (int s = 0; s < a.nsplit; ++s) {
    const float w = __shfl_sync(0xffffffffu, s < 32 ? w0 : w1, s & 31);
    const float* p = a.part_o + (row * a.nsplit + s) * D + lane * kPer;
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[i] = fmaf(w, p[i], acc[i]);
  }
  const float inv = ll == 0.f ? 0.f : 1.f / ll;
#pragma unroll
  for (int i = 0; i < kPer; i += 2)
    *reinterpret_cast<uint32_t*>(a.o + row * D + lane * kPer + i) = pack_bf16x2(acc[i] * inv, acc[i + 1] * inv);
  if (lane == 0) a.lse[row] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * 0.69314718055994530942f;
}

}  // namespace cpattn
