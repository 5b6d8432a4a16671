// Rows of heads on their way through a rotation: a thread's place in a row,
// the cosines of its pairs and the rotation itself (the mathematics stands in
// qk_kernel.cuh).
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

// Cosines and sines, times the magnitude, of a thread's eight pairs. The
// threads at one place of a warp's 512/D rows need the same ones, so each of
// them forms 1/(512/D) of them, of pairs that stay its own, and they exchange
// (a whole warp works on one token). All eight formed by each: 5331 tokens of
// 6 + 2 heads of 64 took 6.3 us forward and 11.9 backward, with this 5.2 and
// 9.5; with 40 heads there is no difference.
template <int D>
struct QkTurns {
  static constexpr int kT = D / 16, kRows = 32 / kT, kOwn = 8 / kRows;
  uint64_t own[kOwn];  // turns of pairs sub, sub + kRows, ...
  __device__ __forceinline__ QkTurns(const QkArgs& a, const QkLane& l, int sub) {
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const int p = sub + i * kRows;
      const bool on = p < 4 ? l.ra : l.rb;
      own[i] = a.turns[on ? (p < 4 ? l.pa + p : l.pb + p - 4) : 0];
    }
  }
  __device__ __forceinline__ void cos_sin(const QkArgs& a, int pos, float (&cs)[8], float (&sn)[8]) const {
    const float sign = a.inverse ? -a.magnitude : a.magnitude;
    float c[kOwn], s[kOwn];
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const uint64_t ph = uint64_t(int64_t(pos)) * own[i];
      sincospif(float(int32_t(ph >> 32)) * 4.656612873077393e-10f, &s[i], &c[i]);  // 2^-31 half turns
      s[i] *= sign;
      c[i] *= a.magnitude;
    }
    const int j = threadIdx.x & (kT - 1);
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      cs[p] = __shfl_sync(0xffffffffu, c[p / kRows], (p % kRows) * kT + j);
      sn[p] = __shfl_sync(0xffffffffu, s[p / kRows], (p % kRows) * kT + j);
    }
  }
};

__device__ __forceinline__ int qk_position(const QkArgs& a, int bi, int tok) {
  return a.positions ? a.positions[int64_t(bi) * a.pos_batch + tok] : rope_position(a, tok);
}

}  // namespace cpattn
