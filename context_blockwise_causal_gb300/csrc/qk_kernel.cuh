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
// a turn, so pos * fraction modulo 2^64 is the phase itself, exact to 2^-64 *
// pos turns, by integer multiplication, without this chip's slow fp64. The upper 32 bits, signed, are the
// phase in [-1/2, 1/2) turn, which sincospi takes.
//
// HBM-bound: each feature is read once and written once (backward: read twice,
// written once); 2 or 3 flops a byte. A row takes D/16 threads, each holding
// two 16-byte pieces placed so that both features of a pair are in one thread,
// whatever the layout: cosines and sines are formed once per thread and token
// and used for all of the warp's heads. A warp takes the heads of one token
// (or, when tokens are few, some of them, so that single tokens spread over
// the chip); rows of several tokens and heads are in flight at once.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "ptx.cuh"
#include "rope_kernel.cuh"

namespace cpattn {

constexpr int kQkThreads = 256;
constexpr int kQkMaxPairs = 64;

// One of the tensors of a call: rows [b, n, h, D], features and heads
// contiguous, strides in elements.
struct QkTensor {
  const __nv_bfloat16* x;
  const __nv_bfloat16* dy;  // backward: gradient of the output
  __nv_bfloat16* y;         // output, or dx in the backward
  const void* w;            // norm weight [D], fp32 or bf16
  int h;
  int64_t x_batch, x_token, dy_batch, dy_token, y_batch, y_token;
};

struct QkArgs {
  QkTensor t[2];  // queries and keys (rope alone: only t[0])
  int b, n;
  // positions (rope_position), or explicit ones
  int s, cp, rank;
  const int* cu_seqlens;
  int nseq;
  const int* positions;
  int64_t pos_batch;  // elements between batch elements' positions (0: shared)
  int rot;            // rotated features (a multiple of 16)
  int inverse;
  int w_fp32;
  float magnitude, eps;
  int split, heads_per;  // warps per token, heads of each (forward)
  float* partial;        // backward: [CTAs][D] sums of t * xh
  int q_ctas;            // backward: CTAs that take t[0]; the others take t[1]
  unsigned int* status;  // checked builds
  uint64_t turns[kQkMaxPairs];  // turns per position of each pair, times 2^64
};

__device__ __forceinline__ void bf16x8_to_f32(const uint4& v, float* f) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 f32_to_bf16x8(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// A thread's place in a row: the features of its two 16-byte pieces, whether
// each is rotated, and the first pair of each.
struct QkLane {
  int fa, fb;
  bool ra, rb;
  int pa, pb;
};
template <int D, bool kInter>
__device__ __forceinline__ QkLane qk_lane(int j, int rot) {
  constexpr int kT = D / 16;
  QkLane l;
  if (kInter) {  // pieces j and j + kT: four pairs each
    l.fa = 8 * j;
    l.fb = 8 * (j + kT);
    l.ra = l.fa < rot;
    l.rb = l.fb < rot;
    l.pa = l.fa / 2;
    l.pb = l.fb / 2;
  } else {  // rotated: pieces j and j + rot/16 hold the two features of eight pairs
    const int half = rot / 16;
    l.ra = l.rb = j < half;
    l.fa = l.ra ? 8 * j : rot + 8 * (j - half);
    l.fb = l.ra ? 8 * (j + half) : rot + 8 * (j - half + (kT - half));
    l.pa = 8 * j;
    l.pb = 8 * j + 4;
  }
  return l;
}

// Rotates a thread's 16 features (f[0..7] from the first piece). cs, sn:
// those of its eight pairs.
template <bool kInter>
__device__ __forceinline__ void qk_rotate(float (&f)[16], const QkLane& l, const float (&cs)[8], const float (&sn)[8]) {
  if (kInter) {
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      if (p < 4 ? l.ra : l.rb) {
        const float a = f[2 * p], b = f[2 * p + 1];
        f[2 * p] = a * cs[p] - b * sn[p];
        f[2 * p + 1] = a * sn[p] + b * cs[p];
      }
    }
  } else if (l.ra) {
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const float a = f[p], b = f[8 + p];
      f[p] = a * cs[p] - b * sn[p];
      f[8 + p] = a * sn[p] + b * cs[p];
    }
  }
}

// Cosines and sines, times the magnitude, of a thread's eight pairs.
__device__ __forceinline__ void qk_cos_sin(const QkArgs& a, const QkLane& l, int pos, float (&cs)[8], float (&sn)[8]) {
  const float sign = a.inverse ? -a.magnitude : a.magnitude;
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const bool on = p < 4 ? l.ra : l.rb;
    const uint64_t ph = uint64_t(int64_t(pos)) * a.turns[on ? (p < 4 ? l.pa + p : l.pb + p - 4) : 0];
    sincospif(float(int32_t(ph >> 32)) * 4.656612873077393e-10f, &sn[p], &cs[p]);  // 2^-31 half turns
    sn[p] *= sign;
    cs[p] *= a.magnitude;
  }
}

__device__ __forceinline__ int qk_position(const QkArgs& a, int bi, int tok) {
  return a.positions ? a.positions[int64_t(bi) * a.pos_batch + tok] : rope_position(a, tok);
}

__device__ __forceinline__ void qk_weights(const void* w, int fp32, const QkLane& l, float (&out)[16]) {
  if (fp32) {
    const float* p = static_cast<const float*>(w);
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const float4 v = *reinterpret_cast<const float4*>(p + (i < 8 ? l.fa + i : l.fb + i - 8));
      out[i] = v.x; out[i + 1] = v.y; out[i + 2] = v.z; out[i + 3] = v.w;
    }
  } else {
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(w);
    bf16x8_to_f32(*reinterpret_cast<const uint4*>(p + l.fa), out);
    bf16x8_to_f32(*reinterpret_cast<const uint4*>(p + l.fb), out + 8);
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
// Heads [h0, h1) of one token of tensor t, kRows rows of the warp at a time
// and kU such groups in flight.
template <int D, bool kNorm, bool kInter>
__device__ __forceinline__ void qk_token(const QkArgs& a, const QkTensor& t, int bi, int tok, int h0, int h1, int sub,
                                         const QkLane& l, const float (&cs)[8], const float (&sn)[8]) {
  constexpr int kT = D / 16, kRows = 32 / kT, kU = 4;
  const __nv_bfloat16* x = t.x + int64_t(bi) * t.x_batch + int64_t(tok) * t.x_token;
  __nv_bfloat16* y = t.y + int64_t(bi) * t.y_batch + int64_t(tok) * t.y_token;
  [[maybe_unused]] float w[16];
  if constexpr (kNorm) qk_weights(t.w, a.w_fp32, l, w);
  for (int h = h0; h < h1; h += kRows * kU) {
    uint4 va[kU], vb[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int hh = h + u * kRows + sub;
      if (hh < h1) {
        va[u] = *reinterpret_cast<const uint4*>(x + hh * D + l.fa);
        vb[u] = *reinterpret_cast<const uint4*>(x + hh * D + l.fb);
      } else {
        va[u] = vb[u] = make_uint4(0u, 0u, 0u, 0u);
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int hh = h + u * kRows + sub;
      if (h + u * kRows >= h1) break;  // uniform in the warp
      float f[16];
      bf16x8_to_f32(va[u], f);
      bf16x8_to_f32(vb[u], f + 8);
      if constexpr (kNorm) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) ss = fmaf(f[i], f[i], ss);
        ss = row_sum<kT>(ss);
        const float r = rsqrtf(ss * (1.0f / D) + a.eps);
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] *= r * w[i];
      }
      qk_rotate<kInter>(f, l, cs, sn);
      if (hh < h1 && bounds_ok(bi < a.b && tok < a.n && hh < t.h, a.status)) {
        *reinterpret_cast<uint4*>(y + hh * D + l.fa) = f32_to_bf16x8(f);
        *reinterpret_cast<uint4*>(y + hh * D + l.fb) = f32_to_bf16x8(f + 8);
      }
    }
  }
}

template <int D, bool kNorm, bool kInter>
__global__ void __launch_bounds__(kQkThreads) cpattn_qk_fwd_kernel(const __grid_constant__ QkArgs a) {
  constexpr int kT = D / 16;
  const int lane = threadIdx.x & 31;
  const QkLane l = qk_lane<D, kInter>(lane % kT, a.rot);
  const int sub = lane / kT;
  const int64_t units = int64_t(a.b) * a.n * a.split;
  const int64_t step = int64_t(gridDim.x) * (kQkThreads / 32);
  for (int64_t idx = int64_t(blockIdx.x) * (kQkThreads / 32) + (threadIdx.x >> 5); idx < units; idx += step) {
    const int64_t bt = idx / a.split;
    const int part = int(idx - bt * a.split);
    const int bi = int(bt / a.n), tok = int(bt - int64_t(bi) * a.n);
    float cs[8], sn[8];
    qk_cos_sin(a, l, qk_position(a, bi, tok), cs, sn);
    const int h0 = part * a.heads_per, h1 = h0 + a.heads_per, hq = a.t[0].h;
    if (h0 < hq) qk_token<D, kNorm, kInter>(a, a.t[0], bi, tok, h0, h1 < hq ? h1 : hq, sub, l, cs, sn);
    if (kNorm && h1 > hq) {
      const int k1 = h1 - hq < a.t[1].h ? h1 - hq : a.t[1].h;
      qk_token<D, kNorm, kInter>(a, a.t[1], bi, tok, h0 > hq ? h0 - hq : 0, k1, sub, l, cs, sn);
    }
  }
}

// ---------------------------------------------------------------- backward
// dx of every row and, per CTA, the sum over its rows of t * xh. The first
// q_ctas CTAs take the queries, the others the keys, in proportion to their
// rows, so that a thread keeps one set of 16 sums over all its rows; they are
// added across the CTA in a fixed order at the end and across CTAs by
// cpattn_qk_dw_kernel: no atomics, the same bits every time.
template <int D, bool kInter>
__global__ void __launch_bounds__(kQkThreads, 2) cpattn_qk_bwd_kernel(const __grid_constant__ QkArgs a) {
  constexpr int kT = D / 16, kRows = 32 / kT, kWarps = kQkThreads / 32, kU = 2;
  __shared__ float red[kWarps][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const QkLane l = qk_lane<D, kInter>(lane % kT, a.rot);
  const int sub = lane / kT;
  const bool is_q = int(blockIdx.x) < a.q_ctas;
  const QkTensor& t = a.t[is_q ? 0 : 1];
  const int cta = is_q ? blockIdx.x : blockIdx.x - a.q_ctas;
  const int ctas = is_q ? a.q_ctas : gridDim.x - a.q_ctas;
  float w[16], dw[16];
  qk_weights(t.w, a.w_fp32, l, w);
#pragma unroll
  for (int i = 0; i < 16; ++i) dw[i] = 0.f;
  const int64_t tokens = int64_t(a.b) * a.n;
  for (int64_t bt = int64_t(cta) * kWarps + warp; bt < tokens; bt += int64_t(ctas) * kWarps) {
    const int bi = int(bt / a.n), tok = int(bt - int64_t(bi) * a.n);
    float cs[8], sn[8];
    qk_cos_sin(a, l, qk_position(a, bi, tok), cs, sn);
    const __nv_bfloat16* x = t.x + int64_t(bi) * t.x_batch + int64_t(tok) * t.x_token;
    const __nv_bfloat16* dy = t.dy + int64_t(bi) * t.dy_batch + int64_t(tok) * t.dy_token;
    __nv_bfloat16* y = t.y + int64_t(bi) * t.y_batch + int64_t(tok) * t.y_token;
    for (int h = 0; h < t.h; h += kRows * kU) {
      uint4 xa[kU], xb[kU], ga[kU], gb[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int hh = h + u * kRows + sub;
        if (hh < t.h) {
          xa[u] = *reinterpret_cast<const uint4*>(x + hh * D + l.fa);
          xb[u] = *reinterpret_cast<const uint4*>(x + hh * D + l.fb);
          ga[u] = *reinterpret_cast<const uint4*>(dy + hh * D + l.fa);
          gb[u] = *reinterpret_cast<const uint4*>(dy + hh * D + l.fb);
        } else {
          xa[u] = xb[u] = ga[u] = gb[u] = make_uint4(0u, 0u, 0u, 0u);
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int hh = h + u * kRows + sub;
        if (h + u * kRows >= t.h) break;  // uniform in the warp
        float f[16], g[16];
        bf16x8_to_f32(xa[u], f);
        bf16x8_to_f32(xb[u], f + 8);
        bf16x8_to_f32(ga[u], g);
        bf16x8_to_f32(gb[u], g + 8);
        qk_rotate<kInter>(g, l, cs, sn);  // a.inverse: turns back
        float ss = 0.f, gx = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          ss = fmaf(f[i], f[i], ss);
          gx = fmaf(g[i] * w[i], f[i], gx);
        }
        ss = row_sum<kT>(ss);
        gx = row_sum<kT>(gx);
        const float r = rsqrtf(ss * (1.0f / D) + a.eps);
        const float c = gx * r * r * (1.0f / D);  // mean(t w * xh) * r
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          dw[i] = fmaf(g[i], f[i] * r, dw[i]);  // a lane past the last head adds zero
          f[i] = r * (g[i] * w[i] - f[i] * c);
        }
        if (hh < t.h && bounds_ok(bi < a.b && tok < a.n, a.status)) {
          *reinterpret_cast<uint4*>(y + hh * D + l.fa) = f32_to_bf16x8(f);
          *reinterpret_cast<uint4*>(y + hh * D + l.fb) = f32_to_bf16x8(f + 8);
        }
      }
    }
  }
  // the warp's rows, then the CTA's warps
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float v = dw[i];
#pragma unroll
    for (int o = kT; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (sub == 0) red[warp][(i < 8 ? l.fa + i : l.fb + i - 8)] = v;
  }
  __syncthreads();
  for (int c = threadIdx.x; c < D; c += kQkThreads) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) v += red[i][c];
    a.partial[int64_t(blockIdx.x) * D + c] = v;
  }
}

// Adds the CTAs' sums: grid (D / 8, 2), 256 threads = 8 features x 32 strips
// of CTAs. A few hundred KB at most: bound by its launch.
__global__ void __launch_bounds__(256) cpattn_qk_dw_kernel(const float* partial, int q_ctas, int ctas, int d,
                                                           float* dwq, float* dwk) {
  __shared__ float red[32][8];
  const int c = blockIdx.x * 8 + (threadIdx.x & 7), strip = threadIdx.x >> 3;
  const int lo = blockIdx.y ? q_ctas : 0, hi = blockIdx.y ? ctas : q_ctas;
  float v = 0.f;
  for (int i = lo + strip; i < hi; i += 32) v += partial[int64_t(i) * d + c];
  red[strip][threadIdx.x & 7] = v;
  __syncthreads();
  if (threadIdx.x < 8) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += red[i][threadIdx.x];
    (blockIdx.y ? dwk : dwq)[c] = s;
  }
}

}  // namespace cpattn
