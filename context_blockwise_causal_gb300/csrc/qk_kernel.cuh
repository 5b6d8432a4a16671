// Queries and keys on their way into attention: rotary positions in their
// general form, alone or behind an RMS norm of each head, forward and
// backward. One kernel template serves all of them.
//
// Rotation of the first rot features of a head: pair i (half layout: features
// i and i + rot/2; interleaved: 2i and 2i + 1) turns by theta = pos * f_i,
//   y_a = m (x_a cos theta - x_b sin theta),
//   y_b = m (x_a sin theta + x_b cos theta);
// features from rot on pass unchanged. The gradient turns back (theta -> -theta).
//
// Norm of a head row x of d features with weight w:
//   r = 1 / sqrt(mean(x^2) + eps),  xh = x r,  y = R(xh * w).
// Backward, with t = R^T dy:  dw = sum over rows of t * xh,
//   dx = r (t w - xh mean(t w * xh)).
// Everything between the load and the store is fp32; the output is rounded once.
//
// Angle: positions reach 10^5 and beyond, where an fp32 product has lost the
// phase. The host gives each pair's turns per position as a 64-bit fraction of
// a turn (rope_turns.h), so pos * fraction modulo 2^64 is the phase, within
// |pos| 2^-64 turns, by integer multiplication, without this chip's slow fp64.
// The upper 32 bits, signed, are the phase in [-1/2, 1/2) turn, which sincospi
// takes.
//
// HBM-bound: each feature is read once and written once (backward: read twice,
// written once); 2 or 3 flops a byte. A row takes D/16 threads, each holding
// two 16-byte pieces placed so that both features of a pair are in one thread,
// whatever the layout: a warp forms its token's cosines and sines once (see
// QkTurns) for all of its heads. A warp takes the heads of one token
// (or, when tokens are few, some of them, so that single tokens spread over
// the chip); rows of several tokens and heads are in flight at once. Measured
// at 32K tokens, d128: rotation alone of 40 heads 103 us (0.97 of the measured
// copy bandwidth), with the norms of 32 + 8 heads 105 us, the backward 160 us
// (0.94); one token of 40 heads takes 2.3 us, a launch.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "ptx.cuh"
#include "qk_rows.cuh"

namespace cpattn {

// The norm weights of both tensors as fp32 in shared memory (registers hold
// the rows in flight instead).
template <int D>
__device__ __forceinline__ void qk_stage_weights(const QkArgs& a, float (&w)[2][D]) {
  for (int i = threadIdx.x; i < 2 * D; i += kQkThreads) {
    const void* p = a.t[i / D].w;
    w[i / D][i % D] = a.w_fp32 ? static_cast<const float*>(p)[i % D]
                               : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i % D]);
  }
  __syncthreads();
}
__device__ __forceinline__ void qk_weights(const float* w, const QkLane& l, float (&out)[16]) {
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    const float4 v = *reinterpret_cast<const float4*>(w + (i < 8 ? l.fa + i : l.fb + i - 8));
    out[i] = v.x; out[i + 1] = v.y; out[i + 2] = v.z; out[i + 3] = v.w;
  }
}

// Sum over the lanes of a row (kT of them, neighbours in the warp).
template <int kT>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = kT / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// ---------------------------------------------------------------- forward
// One unit of a warp: some heads of one token. The heads of both tensors
// count as one run, queries first, so the keys' rows are addressed from the
// queries' head 0.
template <int D, bool kNorm>
struct QkUnit {
  int bi, tok, h0, h1, hq;
  const __nv_bfloat16* xq;
  const __nv_bfloat16* xk;
  __device__ __forceinline__ void set(const QkArgs& a, int64_t idx) {
    const int64_t bt = idx / a.split;
    const int part = int(idx - bt * a.split);
    hq = a.t[0].h;
    const int heads = hq + (kNorm ? a.t[1].h : 0);
    bi = int(bt / a.n);
    tok = int(bt - int64_t(bi) * a.n);
    h0 = part * a.heads_per;
    h1 = h0 + a.heads_per < heads ? h0 + a.heads_per : heads;
    xq = a.t[0].x + int64_t(bi) * a.t[0].x_batch + int64_t(tok) * a.t[0].x_token;
    xk = xq;
    if constexpr (kNorm)
      xk = a.t[1].x + int64_t(bi) * a.t[1].x_batch + int64_t(tok) * a.t[1].x_token - int64_t(hq) * D;
  }
  __device__ __forceinline__ void fetch(int hh, const QkLane& l, uint4& va, uint4& vb) const {
    va = vb = make_uint4(0u, 0u, 0u, 0u);
    if (hh < h1) {
      const __nv_bfloat16* x = (hh < hq ? xq : xk) + hh * D;  // below 2^31 (kQkMaxFeatures in qk_api.cu)
      va = *reinterpret_cast<const uint4*>(x + l.fa);
      vb = *reinterpret_cast<const uint4*>(x + l.fb);
    }
  }
};

// A warp's rows are loaded one group ahead of the one it works on, across
// units too, so that loads are in flight while cosines are formed.
template <int D, bool kNorm, bool kInter>
__global__ void __launch_bounds__(kQkThreads, 2) cpattn_qk_fwd_kernel(const __grid_constant__ QkArgs a) {
  constexpr int kT = D / 16, kRows = 32 / kT, kU = 2, kGroup = kRows * kU;
  __shared__ __align__(16) float w[kNorm ? 2 : 1][D];
  if constexpr (kNorm) qk_stage_weights<D>(a, w);
  const int lane = threadIdx.x & 31;
  const QkLane l = qk_lane<D, kInter>(lane % kT, a.rot);
  const int sub = lane / kT;
  const QkTurns<D> turns(a, l, sub);
  const int64_t units = int64_t(a.b) * a.n * a.split;
  const int64_t step = int64_t(gridDim.x) * (kQkThreads / 32);
  int64_t idx = int64_t(blockIdx.x) * (kQkThreads / 32) + (threadIdx.x >> 5);
  if (idx >= units) return;
  QkUnit<D, kNorm> U;
  U.set(a, idx);
  uint4 va[kU], vb[kU], na[kU], nb[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) U.fetch(U.h0 + u * kRows + sub, l, va[u], vb[u]);
  while (true) {
    const int bi = U.bi, tok = U.tok, h1 = U.h1, hq = U.hq;
    __nv_bfloat16* yq = a.t[0].y + int64_t(bi) * a.t[0].y_batch + int64_t(tok) * a.t[0].y_token;
    __nv_bfloat16* yk = yq;
    if constexpr (kNorm) yk = a.t[1].y + int64_t(bi) * a.t[1].y_batch + int64_t(tok) * a.t[1].y_token - int64_t(hq) * D;
    float cs[8], sn[8];
    turns.cos_sin(a, qk_position(a, bi, tok), cs, sn);
    idx += step;
    for (int h = U.h0, last; ; h += kGroup) {
      last = h + kGroup >= h1;
      if (!last) {
#pragma unroll
        for (int u = 0; u < kU; ++u) U.fetch(h + kGroup + u * kRows + sub, l, na[u], nb[u]);
      } else if (idx < units) {
        U.set(a, idx);
#pragma unroll
        for (int u = 0; u < kU; ++u) U.fetch(U.h0 + u * kRows + sub, l, na[u], nb[u]);
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int hh = h + u * kRows + sub;
        if (h + u * kRows >= h1) break;  // uniform in the warp
        float f[16];
        bf16x8_to_f32(va[u], f);
        bf16x8_to_f32(vb[u], f + 8);
        if constexpr (kNorm) {
          float ss = 0.f, wr[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) ss = fmaf(f[i], f[i], ss);
          ss = row_sum<kT>(ss);
          const float r = rsqrtf(ss * (1.0f / D) + a.eps);
          qk_weights(w[hh < hq ? 0 : 1], l, wr);
#pragma unroll
          for (int i = 0; i < 16; ++i) f[i] *= r * wr[i];
        }
        qk_rotate<kInter>(f, l, cs, sn);
        if (hh < h1 && bounds_ok(bi < a.b && tok < a.n && hh < hq + (kNorm ? a.t[1].h : 0), a.status)) {
          __nv_bfloat16* y = (hh < hq ? yq : yk) + hh * D;
          *reinterpret_cast<uint4*>(y + l.fa) = f32_to_bf16x8(f);
          *reinterpret_cast<uint4*>(y + l.fb) = f32_to_bf16x8(f + 8);
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        va[u] = na[u];
        vb[u] = nb[u];
      }
      if (last) break;
    }
    if (idx >= units) break;
  }
}

// ---------------------------------------------------------------- backward
// dx of every row and, per CTA, the sum over its rows of t * xh. The first
// q_ctas CTAs take the queries, the others the keys, so that a thread keeps
// one set of 16 sums over all its rows; they are added across the CTA in a
// fixed order at the end and across CTAs by cpattn_qk_dw_kernel: no atomics,
// the same bits every time. A thread's pieces of the next three groups of rows
// are on their way into its own slots of shared memory while it works on one
// (held in registers one group ahead, as in the forward, the 16 warps an SM has
// room for do not keep enough bytes in flight: 178 us against 163 at 32K
// tokens, 32 + 8 heads).
constexpr int kQkBwdStages = 4;
constexpr int kQkBwdSmem = kQkBwdStages * kQkThreads * 4 * 16;

template <int D, bool kInter>
__global__ void __launch_bounds__(kQkThreads, 2) cpattn_qk_bwd_kernel(const __grid_constant__ QkArgs a) {
  chain_next();
  constexpr int kT = D / 16, kRows = 32 / kT, kWarps = kQkThreads / 32;
  __shared__ __align__(16) float w[2][D];
  __shared__ float red[kWarps][D];
  extern __shared__ __align__(16) uint8_t ring[];  // [stage][piece][thread] 16 bytes
  qk_stage_weights<D>(a, w);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const QkLane l = qk_lane<D, kInter>(lane % kT, a.rot);
  const int sub = lane / kT;
  const QkTurns<D> turns(a, l, sub);
  const bool is_q = int(blockIdx.x) < a.q_ctas;
  const QkTensor& t = a.t[is_q ? 0 : 1];
  const float* wt = w[is_q ? 0 : 1];
  const int cta = is_q ? blockIdx.x : blockIdx.x - a.q_ctas;
  const int ctas = is_q ? a.q_ctas : gridDim.x - a.q_ctas;
  float dw[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) dw[i] = 0.f;
  const int64_t tokens = int64_t(a.b) * a.n, step = int64_t(ctas) * kWarps;
  // the group of rows to be loaded next: heads h .. of token pt
  int64_t pt = int64_t(cta) * kWarps + warp;
  int ph = 0;
  const __nv_bfloat16* px = nullptr;
  const __nv_bfloat16* pdy = nullptr;
  auto rows_of = [&](int64_t at) {
    const int bi = int(at / a.n), tok = int(at - int64_t(bi) * a.n);
    px = t.x + int64_t(bi) * t.x_batch + int64_t(tok) * t.x_token;
    pdy = t.dy + int64_t(bi) * t.dy_batch + int64_t(tok) * t.dy_token;
  };
  const uint32_t slot = smem_u32(ring) + threadIdx.x * 16;
  auto load = [&](int stage) {  // a group is committed even when nothing is left
    if (pt < tokens) {
      const int hh = ph + sub;
      const bool on = hh < t.h;
      const int64_t o = on ? int64_t(hh) * D : 0;
      const uint32_t dst = slot + stage * (kQkThreads * 64);
      cp_async16(dst, px + o + l.fa, on);
      cp_async16(dst + kQkThreads * 16, px + o + l.fb, on);
      cp_async16(dst + kQkThreads * 32, pdy + o + l.fa, on);
      cp_async16(dst + kQkThreads * 48, pdy + o + l.fb, on);
      ph += kRows;
      if (ph >= t.h) {
        ph = 0;
        pt += step;
        if (pt < tokens) rows_of(pt);
      }
    }
    cp_async_commit();
  };
  int64_t bt = pt;
  if (pt < tokens) rows_of(pt);
#pragma unroll
  for (int s = 0; s < kQkBwdStages - 1; ++s) load(s);
  int stage = 0;
  for (; bt < tokens; bt += step) {
    const int bi = int(bt / a.n), tok = int(bt - int64_t(bi) * a.n);
    __nv_bfloat16* y = t.y + int64_t(bi) * t.y_batch + int64_t(tok) * t.y_token;
    float cs[8], sn[8];
    turns.cos_sin(a, qk_position(a, bi, tok), cs, sn);
    for (int h = 0; h < t.h; h += kRows) {
      const int hh = h + sub;
      cp_async_wait<kQkBwdStages - 2>();
      float f[16], g[16];
      {
        const uint4* v = reinterpret_cast<const uint4*>(ring + stage * (kQkThreads * 64)) + threadIdx.x;
        bf16x8_to_f32(v[0], f);
        bf16x8_to_f32(v[kQkThreads], f + 8);
        bf16x8_to_f32(v[2 * kQkThreads], g);
        bf16x8_to_f32(v[3 * kQkThreads], g + 8);
      }
      load((stage + kQkBwdStages - 1) % kQkBwdStages);
      stage = (stage + 1) % kQkBwdStages;
      qk_rotate<kInter>(g, l, cs, sn);  // a.inverse: turns back
      float ss = 0.f, gx = 0.f, wr[16];
      qk_weights(wt, l, wr);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        ss = fmaf(f[i], f[i], ss);
        gx = fmaf(g[i] * wr[i], f[i], gx);
      }
      ss = row_sum<kT>(ss);
      gx = row_sum<kT>(gx);
      const float r = rsqrtf(ss * (1.0f / D) + a.eps);
      const float c = gx * r * r * (1.0f / D);  // mean(t * w * xh) * r
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        dw[i] = fmaf(g[i], f[i] * r, dw[i]);  // a lane past the last head adds zero
        f[i] = r * (g[i] * wr[i] - f[i] * c);
      }
      if (hh < t.h && bounds_ok(bi < a.b && tok < a.n, a.status)) {
        *reinterpret_cast<uint4*>(y + hh * D + l.fa) = f32_to_bf16x8(f);
        *reinterpret_cast<uint4*>(y + hh * D + l.fb) = f32_to_bf16x8(f + 8);
      }
    }
  }
  cp_async_wait<0>();
  // the warp's rows, then the CTA's warps
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float s = dw[i];
#pragma unroll
    for (int o = kT; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (sub == 0) red[warp][(i < 8 ? l.fa + i : l.fb + i - 8)] = s;
  }
  __syncthreads();
  for (int c = threadIdx.x; c < D; c += kQkThreads) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) s += red[i][c];
    a.partial[int64_t(blockIdx.x) * D + c] = s;
  }
}

// Adds the CTAs' sums: D / 8 CTAs for the queries' and as many for the keys',
// 256 threads = 8 features x 32 strips of CTAs. A few hundred KB at most: bound by its launch.
__global__ void __launch_bounds__(256) cpattn_qk_dw_kernel(const float* partial, int q_ctas, int ctas, int d,
                                                           float* dwq, float* dwk) {
  chain_wait();
  __shared__ float red[32][8];
  const bool keys = int(blockIdx.x) >= d / 8;
  const int c = (blockIdx.x - (keys ? d / 8 : 0)) * 8 + (threadIdx.x & 7), strip = threadIdx.x >> 3;
  const int lo = keys ? q_ctas : 0, hi = keys ? ctas : q_ctas;
  float v = 0.f;
  for (int i = lo + strip; i < hi; i += 32) v += partial[int64_t(i) * d + c];
  red[strip][threadIdx.x & 7] = v;
  __syncthreads();
  if (threadIdx.x < 8) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += red[i][threadIdx.x];
    (keys ? dwk : dwq)[c] = s;
  }
}

}  // namespace cpattn
