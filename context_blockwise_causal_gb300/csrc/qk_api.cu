// C-ABI entry points of the rotary positions' general form and of the q/k
// norms with the rotation (include/cpattn.h): checks, frequencies, launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/cpattn.h"
#include "api_common.h"
#include "qk_host.h"
#include "qk_kernel.cuh"

using namespace cpattn;

namespace {

constexpr double kTwoPi = 6.283185307179586476925;

template <int D, bool kNorm, bool kInter>
int launch_fwd(QkArgs& a, DeviceInfo* di, cudaStream_t st) {
  constexpr int kRows = 32 / (D / 16), kWarps = kQkThreads / 32;
  const int heads = a.t[0].h + (kNorm ? a.t[1].h : 0);
  const int groups = (heads + kRows - 1) / kRows;
  const int64_t tokens = int64_t(a.b) * a.n;
  // A token's heads stay with one warp (one set of cosines) unless that leaves
  // fewer than eight warps per SM; then they spread over more warps.
  const int64_t want = (int64_t(di->num_sms) * 8 + tokens - 1) / tokens;
  const int split = want < groups ? int(want) : groups;
  a.heads_per = (groups + split - 1) / split * kRows;
  a.split = (heads + a.heads_per - 1) / a.heads_per;
  const int64_t ctas = (tokens * a.split + kWarps - 1) / kWarps, most = int64_t(di->num_sms) * 2;  // resident at once
  cpattn_qk_fwd_kernel<D, kNorm, kInter><<<int(ctas < most ? ctas : most), kQkThreads, 0, st>>>(a);
  return launched(cudaGetLastError());
}

template <bool kNorm>
int dispatch_fwd(QkArgs& a, int d, int layout, DeviceInfo* di, cudaStream_t st) {
  if (layout == CPATTN_ROPE_INTERLEAVED)
    return d == 128 ? launch_fwd<128, kNorm, true>(a, di, st) : launch_fwd<64, kNorm, true>(a, di, st);
  return d == 128 ? launch_fwd<128, kNorm, false>(a, di, st) : launch_fwd<64, kNorm, false>(a, di, st);
}

// CTAs of the backward at most (the workspace holds one row of sums for each).
constexpr int kQkBwdMaxCtas = 512;

template <int D>
int launch_bwd(QkArgs& a, int layout, float* dwq, float* dwk, DeviceInfo* di, cudaStream_t st) {
  const int64_t tokens = int64_t(a.b) * a.n, per = kQkThreads / 32;
  int64_t most = int64_t(di->num_sms) * 2;  // resident at once
  if (most > kQkBwdMaxCtas) most = kQkBwdMaxCtas;
  // A token costs its rows and, for its cosines, about as much as kCosRows
  // groups of rows a warp works on at once.
  constexpr int kRows = 32 / (D / 16), kCosRows = 1;
  const int64_t cq = (a.t[0].h + kRows - 1) / kRows + kCosRows, ck = (a.t[1].h + kRows - 1) / kRows + kCosRows;
  int64_t kc = (most * ck + (cq + ck) / 2) / (cq + ck);
  kc = kc < 1 ? 1 : (kc > most - 1 ? most - 1 : kc);
  const int64_t need = (tokens + per - 1) / per;
  const int64_t qc = most - kc < need ? most - kc : need;
  if (kc > need) kc = need;
  a.q_ctas = int(qc);
  const int ctas = int(qc + kc);
  auto kernel = layout == CPATTN_ROPE_INTERLEAVED ? cpattn_qk_bwd_kernel<D, true> : cpattn_qk_bwd_kernel<D, false>;
  std::atomic<bool>& done = di->qk_bwd_attr[(D == 128 ? 2 : 0) + (layout == CPATTN_ROPE_INTERLEAVED ? 1 : 0)];
  if (!done.load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kQkBwdSmem) != cudaSuccess)
      return CPATTN_ERR_CUDA;
    done.store(true, std::memory_order_release);
  }
  kernel<<<ctas, kQkThreads, kQkBwdSmem, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) e = launch_chained(cpattn_qk_dw_kernel, D / 4, 256, st, a.partial, a.q_ctas, ctas, D, dwq, dwk);
  return launched(e);
}

}  // namespace

extern "C" int cpattn_rope_frequencies(int rot_dim, double base, int scaling, double factor, double original_len,
                                       double low, double high, double* inv_freq) {
  if (!inv_freq) return CPATTN_ERR_NULL_PTR;
  if (rot_dim < 2 || rot_dim % 2 != 0 || !(base > 1.0) || !std::isfinite(base)) return CPATTN_ERR_INVALID_ARG;
  if (scaling < CPATTN_ROPE_UNSCALED || scaling > CPATTN_ROPE_BY_INDEX) return CPATTN_ERR_INVALID_ARG;
  if (scaling != CPATTN_ROPE_UNSCALED && !(factor >= 1.0 && std::isfinite(factor))) return CPATTN_ERR_INVALID_ARG;
  const bool parts = scaling == CPATTN_ROPE_BY_TURNS || scaling == CPATTN_ROPE_BY_INDEX;
  if (parts && !(original_len > 0.0 && low > 0.0 && high > low && std::isfinite(high) && std::isfinite(original_len)))
    return CPATTN_ERR_INVALID_ARG;
  if (scaling == CPATTN_ROPE_BASE && rot_dim < 4) return CPATTN_ERR_INVALID_ARG;
  if (scaling == CPATTN_ROPE_BASE) base *= std::pow(factor, double(rot_dim) / (rot_dim - 2));
  // by index: the (fractional) pair that turns t times over original_len
  const auto index_of = [&](double t) { return rot_dim * std::log(original_len / (t * kTwoPi)) / (2.0 * std::log(base)); };
  double first = 0.0, last = 0.0;
  if (scaling == CPATTN_ROPE_BY_INDEX) {
    first = std::floor(index_of(high));
    last = std::ceil(index_of(low));
    first = first < 0.0 ? 0.0 : first;
    last = last > rot_dim - 1.0 ? rot_dim - 1.0 : last;
    if (!(last > first)) last = first + 1.0e-3;
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / rot_dim);
    double keep = 1.0;  // share of the frequency that is not divided by the factor
    if (scaling == CPATTN_ROPE_LINEAR) keep = 0.0;
    if (scaling == CPATTN_ROPE_BY_TURNS) keep = (original_len * f / kTwoPi - low) / (high - low);
    if (scaling == CPATTN_ROPE_BY_INDEX) keep = 1.0 - (i - first) / (last - first);
    keep = keep < 0.0 ? 0.0 : (keep > 1.0 ? 1.0 : keep);
    inv_freq[i] = keep == 1.0 ? f : f * keep + f * (1.0 - keep) / factor;
  }
  return CPATTN_OK;
}

extern "C" int cpattn_rope_ex(const cpattn_rows* x, const cpattn_rows* y, int b, int n, int h, int d,
                              const cpattn_rotary* rotary, int inverse, void* stream) {
  QkArgs a;
  int rc = fill_rotary(rotary, b, n, d, inverse, &a);
  if (rc) return rc;
  if ((rc = check_rows(x, b, n, h, d, false)) || (rc = check_rows(y, b, n, h, d, true))) return rc;
  DeviceInfo* di = nullptr;
  if ((rc = device_info(&di))) return rc;
  set_tensor(&a.t[0], x, nullptr, y, nullptr, h);
  a.t[1] = a.t[0];
  a.eps = 0.f;
  a.w_fp32 = 0;
  a.partial = nullptr;
  a.q_ctas = 0;
  a.status = di->status;
  return dispatch_fwd<false>(a, d, rotary->layout, di, static_cast<cudaStream_t>(stream));
}

extern "C" int cpattn_qk_norm_rope(const cpattn_rows* q, const cpattn_rows* k, const void* q_weight,
                                   const void* k_weight, int weight_fp32, float eps, const cpattn_rows* q_out,
                                   const cpattn_rows* k_out, int b, int n, int hq, int hkv, int d,
                                   const cpattn_rotary* rotary, void* stream) {
  QkArgs a;
  int rc = fill_rotary(rotary, b, n, d, 0, &a);
  if (rc) return rc;
  if (!(eps >= 0.f && eps <= 3.0e38f)) return CPATTN_ERR_INVALID_ARG;
  if (!q_weight || !k_weight) return CPATTN_ERR_NULL_PTR;
  if ((rc = check_rows(q, b, n, hq, d, false)) || (rc = check_rows(k, b, n, hkv, d, false)) ||
      (rc = check_rows(q_out, b, n, hq, d, true)) || (rc = check_rows(k_out, b, n, hkv, d, true)))
    return rc;
  if ((int64_t(hq) + hkv) * d >= kQkMaxFeatures) return CPATTN_ERR_INVALID_ARG;
  if (!aligned16(q_weight) || !aligned16(k_weight)) return CPATTN_ERR_MISALIGNED;
  DeviceInfo* di = nullptr;
  if ((rc = device_info(&di))) return rc;
  set_tensor(&a.t[0], q, nullptr, q_out, q_weight, hq);
  set_tensor(&a.t[1], k, nullptr, k_out, k_weight, hkv);
  a.eps = eps;
  a.w_fp32 = weight_fp32 ? 1 : 0;
  a.partial = nullptr;
  a.q_ctas = 0;
  a.status = di->status;
  return dispatch_fwd<true>(a, d, rotary->layout, di, static_cast<cudaStream_t>(stream));
}

extern "C" size_t cpattn_qk_norm_rope_bwd_workspace_bytes(int d) {
  return d == 64 || d == 128 ? size_t(kQkBwdMaxCtas) * d * 4 : 0;
}

extern "C" int cpattn_qk_norm_rope_bwd(const cpattn_rows* q, const cpattn_rows* k, const void* q_weight,
                                       const void* k_weight, int weight_fp32, float eps, const cpattn_rows* dq_out,
                                       const cpattn_rows* dk_out, const cpattn_rows* dq, const cpattn_rows* dk,
                                       float* dq_weight, float* dk_weight, void* workspace, size_t workspace_bytes,
                                       int b, int n, int hq, int hkv, int d, const cpattn_rotary* rotary,
                                       void* stream) {
  QkArgs a;
  int rc = fill_rotary(rotary, b, n, d, 1, &a);
  if (rc) return rc;
  if (!(eps >= 0.f && eps <= 3.0e38f)) return CPATTN_ERR_INVALID_ARG;
  if (!q_weight || !k_weight || !dq_weight || !dk_weight || !workspace) return CPATTN_ERR_NULL_PTR;
  if ((rc = check_rows(q, b, n, hq, d, false)) || (rc = check_rows(k, b, n, hkv, d, false)) ||
      (rc = check_rows(dq_out, b, n, hq, d, false)) || (rc = check_rows(dk_out, b, n, hkv, d, false)) ||
      (rc = check_rows(dq, b, n, hq, d, true)) || (rc = check_rows(dk, b, n, hkv, d, true)))
    return rc;
  if ((int64_t(hq) + hkv) * d >= kQkMaxFeatures) return CPATTN_ERR_INVALID_ARG;
  if (!aligned16(q_weight) || !aligned16(k_weight) || !aligned16(workspace) || !aligned4(dq_weight) ||
      !aligned4(dk_weight))
    return CPATTN_ERR_MISALIGNED;
  if (workspace_bytes < cpattn_qk_norm_rope_bwd_workspace_bytes(d)) return CPATTN_ERR_WORKSPACE_TOO_SMALL;
  DeviceInfo* di = nullptr;
  if ((rc = device_info(&di))) return rc;
  set_tensor(&a.t[0], q, dq_out, dq, q_weight, hq);
  set_tensor(&a.t[1], k, dk_out, dk, k_weight, hkv);
  a.eps = eps;
  a.w_fp32 = weight_fp32 ? 1 : 0;
  a.split = 1;
  a.heads_per = 0;
  a.partial = static_cast<float*>(workspace);
  a.status = di->status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return d == 128 ? launch_bwd<128>(a, rotary->layout, dq_weight, dk_weight, di, st)
                  : launch_bwd<64>(a, rotary->layout, dq_weight, dk_weight, di, st);
}
