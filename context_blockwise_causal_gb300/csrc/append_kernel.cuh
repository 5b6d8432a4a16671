// New tokens' keys and values into the pages of their sequences, the keys (and
// the queries beside them) rotated to their positions on the way.
//
// Token j of the m new ones of a sequence that then holds n is its token
// p = n - m + j: key R_p k and value v go to slot p % page_size of page
// tables[p / page_size], the query becomes R_p q. Rotation as in qk_kernel.cuh,
// whose threads' places, cosines and phases are used here.
//
// HBM-bound: every row is read once and written once; single tokens cost a
// launch. A token's heads, queries, keys and values in one run, stay with one
// warp, or spread over several when tokens are few; the warp looks up where its
// token goes once and loads its next rows, of its next token too, while it
// works on these. Measured in captured graphs, caches cold: one token of 32 + 8 + 8
// heads of 128 takes 2.7 us, 128 sequences' tokens 4.1 (2.9 where they lie in L2), 5331
// tokens of 6 + 2 + 2 heads of 64 in seven chunks 8.0 (6.7; 2 us of copying; the rest
// is the launch and loads that wait for one another: offsets, length, page), 32768
// tokens 125.5 us, 0.96 of the measured copy bandwidth.
// Looking up several tokens at once, a lane each, is no faster (6.9 and 128 us: a
// warp's tokens then have to follow one another).
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "paged.cuh"
#include "qk_rows.cuh"

namespace cpattn {

struct AppendArgs {
  QkArgs qk;  // t[0]: queries and their output; t[1].x: keys; positions, rotation (rot 0: none), split
  const __nv_bfloat16* v;
  int64_t v_batch, v_row;  // of the new values
  __nv_bfloat16* k_pool;
  __nv_bfloat16* v_pool;
  PagedPlace pg;
  int64_t k_token, k_head, v_token, v_head;
  const int* lengths;  // [seqs]
  const int* cu;       // [seqs + 1] offsets of the sequences' new tokens (b == 1), or nullptr: n each
  int seqs, cap;
};

// Last i with cu[i] <= tok, -1 if there is none: 32 places at a time (a whole warp).
__device__ __forceinline__ int append_seq(const int* cu, int count, int tok) {
  int lo = 0, len = count;  // the number of entries <= tok lies in [lo, lo + len]
  while (len > 0) {
    const int step = (len + 31) / 32;
    const int i = lo + ((threadIdx.x & 31) + 1) * step - 1;
    const unsigned le = __ballot_sync(0xffffffffu, i < lo + len && cu[i] <= tok);
    const int whole = __popc(le);
    const int rest = len - whole * step < step - 1 ? len - whole * step : step - 1;
    lo += whole * step;
    len = rest;
  }
  return lo - 1;
}

// One unit of a warp: some heads of one token.
template <int D>
struct AppendUnit {
  int h0, h1, pos;
  bool live, kept;  // the token belongs to a sequence; it has a slot
  const __nv_bfloat16* xq;
  const __nv_bfloat16* xk;  // these two so that head hh of the run is at + hh * D
  const __nv_bfloat16* xv;
  __nv_bfloat16* yq;
  __nv_bfloat16* yk;
  __nv_bfloat16* yv;
  __device__ __forceinline__ void set(const AppendArgs& a, int64_t idx) {
    const QkArgs& qk = a.qk;
    const int hq = qk.t[0].h, hkv = qk.t[1].h, heads = hq + 2 * hkv;
    const int64_t bt = idx / qk.split;
    const int part = int(idx - bt * qk.split);
    const int bi = int(bt / qk.n), tok = int(bt - int64_t(bi) * qk.n);
    h0 = part * qk.heads_per;
    h1 = h0 + qk.heads_per < heads ? h0 + qk.heads_per : heads;
    int seq = bi, back = qk.n - tok;  // tokens from this one to the sequence's last
    live = true;
    if (a.cu) {
      seq = append_seq(a.cu, a.seqs + 1, tok);
      live = seq >= 0 && seq < a.seqs;
      if (!live) seq = 0;
      back = a.cu[seq + 1] - tok;
    }
    const int64_t place64 = int64_t(a.lengths[seq]) - back;
    kept = live && place64 >= 0 && place64 < a.cap;
    const int place = int(place64);
    const int in_page = kept ? int(unsigned(place) / unsigned(a.pg.page_size)) : 0;
    int page = kept ? a.pg.tables[int64_t(seq) * a.pg.tables_row + in_page] : 0;
    if (kept && !page_ok(page, a.pg, qk.status)) {
      kept = false;
      page = 0;
    }
    const int slot = kept ? place - in_page * a.pg.page_size : 0;
    pos = qk.positions ? qk.positions[int64_t(bi) * qk.pos_batch + tok] : place;
    xq = qk.t[0].x + int64_t(bi) * qk.t[0].x_batch + int64_t(tok) * qk.t[0].x_token;
    xk = qk.t[1].x + int64_t(bi) * qk.t[1].x_batch + int64_t(tok) * qk.t[1].x_token - int64_t(hq) * D;
    xv = a.v + int64_t(bi) * a.v_batch + int64_t(tok) * a.v_row - int64_t(hq + hkv) * D;
    yq = qk.t[0].y + int64_t(bi) * qk.t[0].y_batch + int64_t(tok) * qk.t[0].y_token;
    yk = a.k_pool + page * a.pg.k_page + slot * a.k_token;
    yv = a.v_pool + page * a.pg.v_page + slot * a.v_token;
  }
  __device__ __forceinline__ void fetch(const AppendArgs& a, int hh, const QkLane& l, uint4& va, uint4& vb) const {
    va = vb = make_uint4(0u, 0u, 0u, 0u);
    if (live && hh < h1) {
      const int hq = a.qk.t[0].h;
      const __nv_bfloat16* x = (hh < hq ? xq : hh < hq + a.qk.t[1].h ? xk : xv) + hh * D;  // below 2^31
      va = *reinterpret_cast<const uint4*>(x + l.fa);
      vb = *reinterpret_cast<const uint4*>(x + l.fb);
    }
  }
};

template <int D, bool kInter>
__global__ void __launch_bounds__(kQkThreads, 2) cpattn_append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int kT = D / 16, kRows = 32 / kT, kU = 2, kGroup = kRows * kU;
  const int lane = threadIdx.x & 31;
  const QkLane l = qk_lane<D, kInter>(lane % kT, a.qk.rot);
  const int sub = lane / kT;
  const QkTurns<D> turns(a.qk, l, sub);
  const int hq = a.qk.t[0].h, hr = hq + a.qk.t[1].h;  // the first hr heads of the run turn
  const int64_t units = int64_t(a.qk.b) * a.qk.n * a.qk.split;
  const int64_t step = int64_t(gridDim.x) * (kQkThreads / 32);
  int64_t idx = int64_t(blockIdx.x) * (kQkThreads / 32) + (threadIdx.x >> 5);
  chain_wait();  // up to here beside what runs before this call
  if (idx >= units) return;
  AppendUnit<D> U;
  U.set(a, idx);
  uint4 va[kU], vb[kU], na[kU], nb[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) U.fetch(a, U.h0 + u * kRows + sub, l, va[u], vb[u]);
  while (true) {
    const AppendUnit<D> W = U;
    float cs[8], sn[8];
    const bool turn = a.qk.rot > 0 && W.h0 < hr;
    if (turn) turns.cos_sin(a.qk, W.pos, cs, sn);
    idx += step;
    for (int h = W.h0, last; ; h += kGroup) {
      last = h + kGroup >= W.h1;
      if (!last) {
#pragma unroll
        for (int u = 0; u < kU; ++u) U.fetch(a, h + kGroup + u * kRows + sub, l, na[u], nb[u]);
      } else if (idx < units) {
        U.set(a, idx);
#pragma unroll
        for (int u = 0; u < kU; ++u) U.fetch(a, U.h0 + u * kRows + sub, l, na[u], nb[u]);
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int hh = h + u * kRows + sub;
        uint4 xa = va[u], xb = vb[u];
        if (turn && hh < hr) {
          float f[16];
          bf16x8_to_f32(xa, f);
          bf16x8_to_f32(xb, f + 8);
          qk_rotate<kInter>(f, l, cs, sn);
          // a piece that passes keeps its bits, whatever they mean
          if (l.ra) xa = f32_to_bf16x8(f);
          if (l.rb) xb = f32_to_bf16x8(f + 8);
        }
        if (hh < W.h1 && W.live && (hh < hq || W.kept)) {
          __nv_bfloat16* y = hh < hq ? W.yq + hh * D
                                     : hh < hr ? W.yk + int64_t(hh - hq) * a.k_head : W.yv + int64_t(hh - hr) * a.v_head;
          *reinterpret_cast<uint4*>(y + l.fa) = xa;
          *reinterpret_cast<uint4*>(y + l.fb) = xb;
        }
        va[u] = na[u];
        vb[u] = nb[u];
      }
      if (last) break;
    }
    if (idx >= units) return;
  }
}

}  // namespace cpattn
