// What the library's translation units share on the host: per-device state
// and the checks that every entry point makes.
#pragma once
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <utility>

#include "../../include/cpattn.h"
#include "align.h"

namespace cpattn {

constexpr int kMaxDevices = 64;

struct DeviceInfo {
  bool init = false;
  bool sm103 = false;
  int num_sms = 0;
  unsigned int* status = nullptr;
  // kernel attributes already set, per kernel; set once, read by any thread
  std::atomic<bool> fwd_attr[17] = {};  // [d == 128][step form][five-slot ring][tile pairs]; 16: self-test
  std::atomic<bool> bwd_attr[3] = {};   // [d == 128]; 2: self-test
  std::atomic<bool> win_fwd_attr[4] = {};  // window form: [d == 128][tile pairs]
  std::atomic<bool> win_bwd_attr[2] = {};  // window form: [d == 128]
  std::atomic<bool> decode_attr[2] = {};   // [d == 128]
  std::atomic<bool> paged_attr[12] = {};   // [PagedKind][units of 16 rows][d == 128]
  std::atomic<bool> prefix_attr[2] = {};   // [d == 128]
  std::atomic<bool> qk_bwd_attr[4] = {};   // [d == 128][interleaved]
};

// State of the current device (CPATTN_ERR_UNSUPPORTED_ARCH unless sm_103).
int device_info(DeviceInfo** out);

// Grid of a persistent kernel over `units` work units: one CTA per SM, at
// most the cap set by cpattn_set_max_ctas, at most one per unit.
int persistent_grid(const DeviceInfo* di, int64_t units);

// Launches a call's second kernel, which begins with chain_wait(): it may be
// placed while the first one, which says chain_next(), still runs, so that its
// launch costs next to no time of its own (one 131K-token sequence decoded in
// 38 runs and joined: 98 -> 95.5 us; the sums of the weights' gradients behind
// a backward of 12 us: 22.4 -> 19.5 for the whole of forward and backward). The
// window backward's kernels gain nothing by it: they leave their successors no
// room until they end.
template <class... P, class... A>
cudaError_t launch_chained(void (*kernel)(P...), int64_t ctas, int threads, cudaStream_t st, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas));
  cfg.blockDim = dim3(unsigned(threads));
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}
inline int launched(cudaError_t e) {
  if (e == cudaSuccess) return CPATTN_OK;
  cudaGetLastError();
  return CPATTN_ERR_LAUNCH_FAILED;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline bool valid_scale(float scale) { return scale > 0.f && scale <= 3.0e38f; }
inline double default_scale(int d) { return 1.0 / std::sqrt(double(d)); }

}  // namespace cpattn
