// Host side of single-token attention that its entry points share: strides, the
// launch.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "api_common.h"
#include "decode_kernel.cuh"

namespace cpattn {

inline bool strides_ok(int64_t batch, int64_t token, int64_t head) {
  return batch >= 0 && token >= 0 && head >= 0 && batch % 8 == 0 && token % 8 == 0 && head % 8 == 0;
}

// A kernel of one CTA per run: clusters of up to 8 runs; `chained`: as
// launch_chained's second kernels.
template <class... P, class... A>
cudaError_t launch_runs(void (*kernel)(P...), int64_t ctas, int threads, int nsplit, int smem_bytes, bool chained,
                        cudaStream_t st, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas));
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = size_t(smem_bytes);
  cfg.stream = st;
  cudaLaunchAttribute attrs[2];
  cfg.attrs = attrs;
  if (nsplit > 1 && nsplit <= kDecMaxCluster) {
    cudaLaunchAttribute& cluster = attrs[cfg.numAttrs++];
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim.x = unsigned(nsplit);
    cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
  }
  if (chained) {
    cudaLaunchAttribute& behind = attrs[cfg.numAttrs++];
    behind.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    behind.val.programmaticStreamSerializationAllowed = 1;
  }
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

// Dynamic shared memory of a kernel, set once per device.
template <class K>
bool allow_smem(std::atomic<bool>& done, K kernel, int bytes) {
  if (done.load(std::memory_order_acquire)) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
  done.store(true, std::memory_order_release);
  return true;
}

}  // namespace cpattn
