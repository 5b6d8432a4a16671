// C-ABI entry points of sliding-window attention (include/cpattn.h): argument
// checks, geometry, tensor maps and launches of the forward and backward
// kernels in their window form (win_schedule.cuh).
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/cpattn.h"
#include "api_common.h"
#include "bwd_kernel.cuh"
#include "fwd_kernel.cuh"
#include "tmap.h"

using namespace cpattn;

namespace {

struct WinShape {
  int b, sq, skv, hq, hkv, d, window, sinks;
};

bool pairs_of(const WinShape& w) { return (w.hq / w.hkv) % 2 != 0; }

int check_shape(const WinShape& w) {
  if (w.b < 1 || w.sq < 1 || w.skv < w.sq || w.hq < 1 || w.hkv < 1) return CPATTN_ERR_INVALID_ARG;
  if ((w.d != 64 && w.d != 128) || w.hq % w.hkv != 0) return CPATTN_ERR_INVALID_ARG;
  if (w.window < 1 || w.sinks < 0) return CPATTN_ERR_INVALID_ARG;
  // rows, tile-padded rows and work units are 32-bit
  const int64_t lim = int64_t(1) << 31;
  if (w.skv > (1 << 30) || int64_t(w.b) * w.skv >= lim) return CPATTN_ERR_INVALID_ARG;
  if (int64_t(w.b) * w.hq * ((w.skv + kTile - 1) / kTile) >= lim / 2) return CPATTN_ERR_INVALID_ARG;
  return CPATTN_OK;
}

// Geometry of a uniform batch, or of packed samples (cu: nseq + 1 offsets).
CpGeom win_geom(const WinShape& w, const int* cu, int nseq, bool pairs) {
  CpGeom g;
  g.b = w.b;
  g.s = w.sq;
  g.kv_s = w.skv;
  g.hq = w.hq;
  g.hkv = w.hkv;
  g.cp = 1;
  g.causal = 1;
  g.c = w.sq;
  g.npairs = (w.hq + 1) / 2;
  // a window or a count of first tokens beyond the sequence is the whole of it
  g.window = w.window < w.skv ? w.window : w.skv;
  g.sinks = w.sinks < w.skv ? w.sinks : w.skv;
  g.nseq = nseq;
  for (int i = 0; i <= nseq && cu; ++i) g.cu[i] = cu[i];
  win_finish(g, pairs);
  win_set_parts(g);
  win_set_divs(g, pairs);
  return g;
}

template <int D, bool kTP>
int launch_fwd(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const FwdArgs& args,
               DeviceInfo* di, cudaStream_t st) {
  constexpr int kRing = fwd_ring<D>(false);
  using C = FwdCfg<D, kRing>;
  auto kernel = cpattn_fwd_kernel<D, false, kRing, kTP, false, true>;
  std::atomic<bool>& done = di->win_fwd_attr[(D == 128 ? 2 : 0) + (kTP ? 1 : 0)];
  if (!done.load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes) != cudaSuccess)
      return CPATTN_ERR_CUDA;
    // the in-kernel register split assumes exactly kFwdLaunchRegs at launch
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, kernel) != cudaSuccess) return CPATTN_ERR_CUDA;
    if (fa.numRegs != kFwdLaunchRegs) return CPATTN_ERR_LAUNCH_FAILED;
    done.store(true, std::memory_order_release);
  }
  const int grid = persistent_grid(di, win_fwd_units(args.g, kTP));
  kernel<<<grid, kFwdThreads, C::kSmemBytes, st>>>(tq, tk, tv, args);
  return cudaGetLastError() == cudaSuccess ? CPATTN_OK : CPATTN_ERR_LAUNCH_FAILED;
}

// cu == nullptr: a uniform batch. Otherwise packed samples, w.b == 1 and
// w.sq == w.skv == the packed rows of these samples; lse_stride is the row
// stride of lse (the whole packed total).
int fwd_window(const void* q, const void* k, const void* v, void* o, float* lse, const WinShape& w, const int* cu,
               int nseq, int64_t lse_stride, double scale, void* stream) {
  DeviceInfo* di = nullptr;
  int rc = device_info(&di);
  if (rc) return rc;
  const uint64_t q_rows = uint64_t(w.b) * w.sq, kv_rows = uint64_t(w.b) * w.skv;
  CUtensorMap tq, tk, tv;
  if (!encode_bf16_rows_heads_d(&tq, q, q_rows, w.hq, w.d, kTile) ||
      !encode_bf16_rows_heads_d(&tk, k, kv_rows, w.hkv, w.d, kTile) ||
      !encode_bf16_rows_heads_d(&tv, v, kv_rows, w.hkv, w.d, kTile))
    return CPATTN_ERR_CUDA;
  const bool pairs = pairs_of(w);
  FwdArgs args;
  args.g = win_geom(w, cu, nseq, pairs);
  args.o = static_cast<__nv_bfloat16*>(o);
  args.lse = lse;
  args.lse_stride = lse_stride;
  args.q_rows = int64_t(q_rows);
  args.kv_rows = int64_t(kv_rows);
  args.lse_len = int64_t(w.b) * w.hq * lse_stride;
  args.o_part = nullptr;
  args.step = -1;
  args.scale_log2 = float(1.4426950408889634 * scale);
  args.status = di->status;
  args.producer_limit_ns = kWaitLimitNs;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (w.d == 128) return pairs ? launch_fwd<128, true>(tq, tk, tv, args, di, st) : launch_fwd<128, false>(tq, tk, tv, args, di, st);
  return pairs ? launch_fwd<64, true>(tq, tk, tv, args, di, st) : launch_fwd<64, false>(tq, tk, tv, args, di, st);
}

struct WinBwdLayout {
  size_t dvec, part_dk, part_dv, total;
  int ntp;
  int64_t vec_len, part_len;
};

WinBwdLayout bwd_layout(const CpGeom& g, int d) {
  WinBwdLayout L;
  L.ntp = g.tpc * kTile;
  L.vec_len = int64_t(num_seqs(g)) * g.hq * L.ntp;
  L.part_len = int64_t(g.part_units) * kTile * d;
  L.dvec = align256(size_t(L.vec_len) * 4);
  L.part_dk = L.dvec + align256(size_t(L.vec_len) * 4);
  L.part_dv = L.part_dk + align256(size_t(L.part_len) * 4);
  L.total = L.part_dv + align256(size_t(L.part_len) * 4);
  return L;
}

template <int D>
int launch_bwd(const CUtensorMap* maps, const BwdArgs& args, DeviceInfo* di, cudaStream_t st) {
  auto dkdv = cpattn_bwd_dkdv_kernel<D, false, true>;
  auto dqk = cpattn_bwd_dq_kernel<D, false, true>;
  std::atomic<bool>& done = di->win_bwd_attr[D == 128 ? 1 : 0];
  if (!done.load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(dkdv, cudaFuncAttributeMaxDynamicSharedMemorySize, DkdvCfg<D>::kSmemBytes) != cudaSuccess ||
        cudaFuncSetAttribute(dqk, cudaFuncAttributeMaxDynamicSharedMemorySize, DqCfg<D, true>::kSmemBytes) != cudaSuccess)
      return CPATTN_ERR_CUDA;
    done.store(true, std::memory_order_release);
  }
  const CpGeom& g = args.g;
  // dQ first: it forms the row vectors that dK/dV reads
  dqk<<<persistent_grid(di, win_dq_units(g)), kBwdThreads, DqCfg<D, true>::kSmemBytes, st>>>(maps[0], maps[1], maps[2],
                                                                                       maps[3], args);
  dkdv<<<persistent_grid(di, win_dkdv_units(g)), kBwdThreads, DkdvCfg<D>::kSmemBytes, st>>>(maps[0], maps[1], maps[2],
                                                                                            maps[3], args);
  const int64_t per = win_join_ctas(g);
  if (g.part_units > 0 && g.nseq > 0) {
    JoinArgs join{args, {}};
    win_set_cuts(g, join.cuts);
    const int64_t tiles = int64_t(g.hkv) * join.cuts.first[g.nseq];
    cpattn_window_join_kernel<D, true><<<unsigned(tiles * per), kJoinWarps * 32, 0, st>>>(join);
  } else if (g.part_units > 0) {
    const int64_t tiles = int64_t(g.b) * g.hkv * win_cut_tiles(g);
    cpattn_window_join_kernel<D, false><<<unsigned(tiles * per), kJoinWarps * 32, 0, st>>>(args);
  }
  return cudaGetLastError() == cudaSuccess ? CPATTN_OK : CPATTN_ERR_LAUNCH_FAILED;
}

int bwd_window(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dout, void* dq,
               void* dk, void* dv, void* workspace, size_t workspace_bytes, const WinShape& w, const int* cu, int nseq,
               int64_t lse_stride, double scale, void* stream) {
  BwdArgs args;
  args.g = win_geom(w, cu, nseq, false);
  // units of dK/dV: packed key tiles are the packed query tiles
  if (win_dkdv_units(args.g) >= (int64_t(1) << 31)) return CPATTN_ERR_INVALID_ARG;
  const WinBwdLayout L = bwd_layout(args.g, w.d);
  if (workspace_bytes < L.total) return CPATTN_ERR_WORKSPACE_TOO_SMALL;
  DeviceInfo* di = nullptr;
  int rc = device_info(&di);
  if (rc) return rc;
  const uint64_t q_rows = uint64_t(w.b) * w.sq, kv_rows = uint64_t(w.b) * w.skv;
  CUtensorMap maps[4];
  if (!encode_bf16_rows_heads_d(&maps[0], q, q_rows, w.hq, w.d, kTile) ||
      !encode_bf16_rows_heads_d(&maps[1], k, kv_rows, w.hkv, w.d, kTile) ||
      !encode_bf16_rows_heads_d(&maps[2], v, kv_rows, w.hkv, w.d, kTile) ||
      !encode_bf16_rows_heads_d(&maps[3], dout, q_rows, w.hq, w.d, kTile))
    return CPATTN_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  args.ntp = L.ntp;
  args.o = static_cast<const __nv_bfloat16*>(o);
  args.dout = static_cast<const __nv_bfloat16*>(dout);
  args.lse = lse;
  args.lse_stride = lse_stride;
  args.q_rows = int64_t(q_rows);
  args.kv_rows = int64_t(kv_rows);
  args.lse_len = int64_t(w.b) * w.hq * lse_stride;
  args.vec_len = L.vec_len;
  args.lvec = reinterpret_cast<float*>(ws);
  args.dvec = reinterpret_cast<float*>(ws + L.dvec);
  args.part_dk = reinterpret_cast<float*>(ws + L.part_dk);
  args.part_dv = reinterpret_cast<float*>(ws + L.part_dv);
  args.part_len = L.part_len;
  args.dq = static_cast<__nv_bfloat16*>(dq);
  args.dk = static_cast<__nv_bfloat16*>(dk);
  args.dv = static_cast<__nv_bfloat16*>(dv);
  args.scale = float(scale);
  args.scale_log2 = float(1.4426950408889634 * scale);
  args.status = di->status;
  args.producer_limit_ns = kWaitLimitNs;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return w.d == 128 ? launch_bwd<128>(maps, args, di, st) : launch_bwd<64>(maps, args, di, st);
}

int scale_of(float scale, int d, double* out) {
  if (!(scale == 0.f || valid_scale(scale))) return CPATTN_ERR_INVALID_ARG;
  *out = scale == 0.f ? default_scale(d) : double(scale);
  return CPATTN_OK;
}

// Sample offsets: 0 = cu[0] <= ... <= cu[nseq]; the total, or an error code.
int64_t check_cu(const int* cu, int nseq) {
  if (!cu) return CPATTN_ERR_NULL_PTR;
  if (nseq < 1 || cu[0] != 0) return CPATTN_ERR_INVALID_ARG;
  for (int i = 0; i < nseq; ++i)
    if (cu[i + 1] < cu[i]) return CPATTN_ERR_INVALID_ARG;
  return cu[nseq];
}

// Calls f(first row, rows, offsets from that row, samples) for consecutive
// groups of up to kMaxSeqs samples (their offsets travel as kernel
// parameters), skipping groups without rows.
template <class F>
int for_groups(const int* cu, int nseq, F f) {
  for (int first = 0; first < nseq; first += kMaxSeqs) {
    const int n = nseq - first < kMaxSeqs ? nseq - first : kMaxSeqs;
    int local[kMaxSeqs + 1];
    for (int i = 0; i <= n; ++i) local[i] = cu[first + i] - cu[first];
    if (local[n] == 0) continue;
    const int rc = f(cu[first], local[n], local, n);
    if (rc) return rc;
  }
  return CPATTN_OK;
}

}  // namespace

extern "C" int cpattn_fwd_window(const void* q, const void* k, const void* v, void* o, float* lse, int b, int sq,
                                 int skv, int hq, int hkv, int d, int window, int sinks, float scale, void* stream) {
  if (!q || !k || !v || !o || !lse) return CPATTN_ERR_NULL_PTR;
  const WinShape w{b, sq, skv, hq, hkv, d, window, sinks};
  int rc = check_shape(w);
  if (rc) return rc;
  double sc = 0.0;
  if ((rc = scale_of(scale, d, &sc))) return rc;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse)) return CPATTN_ERR_MISALIGNED;
  return fwd_window(q, k, v, o, lse, w, nullptr, 0, sq, sc, stream);
}

extern "C" int cpattn_fwd_window_varlen(const void* q, const void* k, const void* v, void* o, float* lse,
                                        const int* cu_seqlens, int nseq, int hq, int hkv, int d, int window, int sinks,
                                        float scale, void* stream) {
  const int64_t total = check_cu(cu_seqlens, nseq);
  if (total < 0) return int(total);
  const int rows = total > 0 ? int(total) : 1;
  int rc = check_shape(WinShape{1, rows, rows, hq, hkv, d, window, sinks});
  if (rc) return rc;
  double sc = 0.0;
  if ((rc = scale_of(scale, d, &sc))) return rc;
  if (total == 0) return CPATTN_OK;
  if (!q || !k || !v || !o || !lse) return CPATTN_ERR_NULL_PTR;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse)) return CPATTN_ERR_MISALIGNED;
  return for_groups(cu_seqlens, nseq, [&](int start, int len, const int* cu, int n) {
    const size_t qo = size_t(start) * hq * d * 2, ko = size_t(start) * hkv * d * 2;
    return fwd_window(static_cast<const uint8_t*>(q) + qo, static_cast<const uint8_t*>(k) + ko,
                      static_cast<const uint8_t*>(v) + ko, static_cast<uint8_t*>(o) + qo, lse + start,
                      WinShape{1, len, len, hq, hkv, d, window, sinks}, cu, n, total, sc, stream);
  });
}

extern "C" size_t cpattn_bwd_window_workspace_bytes(int b, int sq, int skv, int hq, int hkv, int d, int window,
                                                    int sinks) {
  const WinShape w{b, sq, skv, hq, hkv, d, window, sinks};
  if (check_shape(w)) return 0;
  return bwd_layout(win_geom(w, nullptr, 0, false), d).total;
}

extern "C" int cpattn_bwd_window(const void* q, const void* k, const void* v, const void* o, const float* lse,
                                 const void* dout, void* dq, void* dk, void* dv, void* workspace,
                                 size_t workspace_bytes, int b, int sq, int skv, int hq, int hkv, int d, int window,
                                 int sinks, float scale, void* stream) {
  if (!q || !k || !v || !o || !lse || !dout || !dq || !dk || !dv || !workspace) return CPATTN_ERR_NULL_PTR;
  const WinShape w{b, sq, skv, hq, hkv, d, window, sinks};
  int rc = check_shape(w);
  if (rc) return rc;
  double sc = 0.0;
  if ((rc = scale_of(scale, d, &sc))) return rc;
  for (const void* p : {q, k, v, o, static_cast<const void*>(lse), dout, static_cast<const void*>(dq),
                        static_cast<const void*>(dk), static_cast<const void*>(dv), static_cast<const void*>(workspace)})
    if (!aligned16(p)) return CPATTN_ERR_MISALIGNED;
  return bwd_window(q, k, v, o, lse, dout, dq, dk, dv, workspace, workspace_bytes, w, nullptr, 0, sq, sc, stream);
}

extern "C" size_t cpattn_bwd_window_varlen_workspace_bytes(const int* cu_seqlens, int nseq, int hq, int hkv, int d,
                                                           int window, int sinks) {
  const int64_t total = check_cu(cu_seqlens, nseq);
  if (total < 0) return 0;
  const int rows = total > 0 ? int(total) : 1;
  if (check_shape(WinShape{1, rows, rows, hq, hkv, d, window, sinks})) return 0;
  size_t need = 16;  // the groups share the workspace: the largest one's
  for_groups(cu_seqlens, nseq, [&](int, int len, const int* cu, int n) {
    const size_t t = bwd_layout(win_geom(WinShape{1, len, len, hq, hkv, d, window, sinks}, cu, n, false), d).total;
    need = t > need ? t : need;
    return int(CPATTN_OK);
  });
  return need;
}

extern "C" int cpattn_bwd_window_varlen(const void* q, const void* k, const void* v, const void* o, const float* lse,
                                        const void* dout, void* dq, void* dk, void* dv, void* workspace,
                                        size_t workspace_bytes, const int* cu_seqlens, int nseq, int hq, int hkv, int d,
                                        int window, int sinks, float scale, void* stream) {
  const int64_t total = check_cu(cu_seqlens, nseq);
  if (total < 0) return int(total);
  const int rows = total > 0 ? int(total) : 1;
  int rc = check_shape(WinShape{1, rows, rows, hq, hkv, d, window, sinks});
  if (rc) return rc;
  double sc = 0.0;
  if ((rc = scale_of(scale, d, &sc))) return rc;
  if (total == 0) return CPATTN_OK;
  if (!q || !k || !v || !o || !lse || !dout || !dq || !dk || !dv || !workspace) return CPATTN_ERR_NULL_PTR;
  for (const void* p : {q, k, v, o, static_cast<const void*>(lse), dout, static_cast<const void*>(dq),
                        static_cast<const void*>(dk), static_cast<const void*>(dv), static_cast<const void*>(workspace)})
    if (!aligned16(p)) return CPATTN_ERR_MISALIGNED;
  if (workspace_bytes < cpattn_bwd_window_varlen_workspace_bytes(cu_seqlens, nseq, hq, hkv, d, window, sinks))
    return CPATTN_ERR_WORKSPACE_TOO_SMALL;  // before the first group's kernels
  return for_groups(cu_seqlens, nseq, [&](int start, int len, const int* cu, int n) {
    const size_t qo = size_t(start) * hq * d * 2, ko = size_t(start) * hkv * d * 2;
    return bwd_window(static_cast<const uint8_t*>(q) + qo, static_cast<const uint8_t*>(k) + ko,
                      static_cast<const uint8_t*>(v) + ko, static_cast<const uint8_t*>(o) + qo, lse + start,
                      static_cast<const uint8_t*>(dout) + qo, static_cast<uint8_t*>(dq) + qo,
                      static_cast<uint8_t*>(dk) + ko, static_cast<uint8_t*>(dv) + ko, workspace, workspace_bytes,
                      WinShape{1, len, len, hq, hkv, d, window, sinks}, cu, n, total, sc, stream);
  });
}
