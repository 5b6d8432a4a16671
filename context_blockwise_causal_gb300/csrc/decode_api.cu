// C-ABI entry points of single-token attention over a cache (include/cpattn.h).
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/cpattn.h"
#include "api_common.h"
#include "decode_kernel.cuh"

using namespace cpattn;

namespace {

int check_shape(int b, int hq, int hkv, int d, int cap, int window, int sinks) {
  if (b < 1 || hq < 1 || hkv < 1 || cap < 1 || window < 0 || sinks < 0) return CPATTN_ERR_INVALID_ARG;
  if ((d != 64 && d != 128) || hq % hkv != 0) return CPATTN_ERR_INVALID_ARG;
  if (cap > (1 << 30) || int64_t(b) * hq * kDecMaxSplit >= (int64_t(1) << 31)) return CPATTN_ERR_INVALID_ARG;
  return CPATTN_OK;
}

// Keys a sequence can see at most.
int64_t max_keys(int cap, int window, int sinks) {
  if (window == 0) return cap;
  const int64_t seen = int64_t(window) + sinks;
  return seen < cap ? seen : cap;
}

// Runs per (sequence, KV head group): two CTAs fit an SM.
//  * As many as fill the places without a second wave, of 64 keys or more (one
//    round of a CTA's warps), up to a cluster: 8 of one 1028-key sequence with
//    8 KV heads take 6.7 us, 4 take 7.7; with 8 such sequences 4 take 9.6 us
//    and 8, a second wave, 15.5.
//  * Runs of 2048 keys or more may fill the places twice, which levels out
//    different lengths: 16 sequences of 32K to 64K keys take 447 us in 4 runs,
//    507 in 2 and 465 in 8.
//  * Where a cluster's 8 leave half of the places empty, such long runs go up
//    to all places through device memory (one 131K-key sequence, 8 KV heads:
//    92 us in 38 runs with their join, 188 in 8). Clusters of 16 find too few
//    places together (122 us there).
int choose_split(int num_sms, int64_t units, int64_t keys) {
  const int64_t places = 2 * int64_t(num_sms);
  int64_t s = 1;
  while (2 * s <= kDecMaxCluster) {
    const int64_t ctas = 2 * s * units, run = keys / (2 * s);
    if (!(ctas <= places ? run >= 64 : ctas <= 2 * places && run >= 2048)) break;
    s *= 2;
  }
  if (s == kDecMaxCluster && 2 * s * units <= places) {
    int64_t more = places / units;
    if (more > keys / 2048) more = keys / 2048;
    if (more > s) s = more < kDecMaxSplit ? more : kDecMaxSplit;
  }
  return int(s);
}

// Workspace bytes (0: none).
size_t workspace_for(int b, int hq, int d, int nsplit) {
  if (nsplit <= kDecMaxCluster) return 0;
  const size_t rows = size_t(b) * hq * nsplit;
  return align256(rows * d * 4) + align256(rows * 4);
}

bool strides_ok(int64_t batch, int64_t token, int64_t head) {
  return batch >= 0 && token >= 0 && head >= 0 && batch % 8 == 0 && token % 8 == 0 && head % 8 == 0;
}

template <int D>
int launch(const DecodeArgs& a, DeviceInfo* di, cudaStream_t st) {
  std::atomic<bool>& done = di->decode_attr[D == 128 ? 1 : 0];
  if (!done.load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(cpattn_decode_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             DecodeCfg<D>::kSmemBytes) != cudaSuccess)
      return CPATTN_ERR_CUDA;
    done.store(true, std::memory_order_release);
  }
  const int64_t ctas = int64_t(a.b) * a.hkv * a.row_groups * a.nsplit;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas));
  cfg.blockDim = dim3(kDecWarps * 32);
  cfg.dynamicSmemBytes = DecodeCfg<D>::kSmemBytes;
  cfg.stream = st;
  cudaLaunchAttribute cluster;
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = unsigned(a.nsplit);
  cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
  if (a.nsplit > 1 && a.nsplit <= kDecMaxCluster) {
    cfg.attrs = &cluster;
    cfg.numAttrs = 1;
  }
  cudaError_t e = cudaLaunchKernelEx(&cfg, cpattn_decode_kernel<D>, a);
  if (e == cudaSuccess && a.nsplit > kDecMaxCluster)
    e = launch_chained(cpattn_decode_join_kernel<D>, (int64_t(a.b) * a.hq + 3) / 4, 128, st, a);
  return launched(e);
}

}  // namespace

extern "C" size_t cpattn_decode_workspace_bytes(int b, int hq, int hkv, int d, int cap, int window, int sinks) {
  if (check_shape(b, hq, hkv, d, cap, window, sinks)) return 0;
  DeviceInfo* di = nullptr;
  if (device_info(&di)) return 0;
  const int64_t units = int64_t(b) * hkv * ((hq / hkv + 15) / 16);
  return workspace_for(b, hq, d, choose_split(di->num_sms, units, max_keys(cap, window, sinks)));
}

extern "C" int cpattn_decode(const void* q, const void* k_cache, const void* v_cache, const int* lengths, void* o,
                             float* lse, void* workspace, size_t workspace_bytes, int b, int hq, int hkv, int d,
                             int cap, int64_t q_batch, int64_t k_batch, int64_t k_token, int64_t k_head,
                             int64_t v_batch, int64_t v_token, int64_t v_head, int window, int sinks, float scale,
                             void* stream) {
  if (!q || !k_cache || !v_cache || !lengths || !o || !lse) return CPATTN_ERR_NULL_PTR;
  int rc = check_shape(b, hq, hkv, d, cap, window, sinks);
  if (rc) return rc;
  if (!(scale == 0.f || valid_scale(scale))) return CPATTN_ERR_INVALID_ARG;
  if (!strides_ok(k_batch, k_token, k_head) || !strides_ok(v_batch, v_token, v_head) || q_batch < 0 || q_batch % 8 != 0)
    return CPATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o) || !aligned4(lse) ||
      !aligned4(lengths) || !aligned16(workspace))
    return CPATTN_ERR_MISALIGNED;
  DeviceInfo* di = nullptr;
  if ((rc = device_info(&di))) return rc;
  DecodeArgs a;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k_cache);
  a.v = static_cast<const __nv_bfloat16*>(v_cache);
  a.lengths = lengths;
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  a.q_batch = q_batch;
  a.k_batch = k_batch;
  a.k_token = k_token;
  a.k_head = k_head;
  a.v_batch = v_batch;
  a.v_token = v_token;
  a.v_head = v_head;
  a.b = b;
  a.hq = hq;
  a.hkv = hkv;
  a.G = hq / hkv;
  a.cap = cap;
  a.window = window;
  a.sinks = window > 0 ? sinks : 0;
  a.row_groups = (a.G + 15) / 16;
  const int64_t units = int64_t(b) * hkv * a.row_groups;
  a.nsplit = choose_split(di->num_sms, units, max_keys(cap, window, sinks));
  const size_t need = workspace_for(b, hq, d, a.nsplit);
  if (need > 0 && !workspace) return CPATTN_ERR_NULL_PTR;
  if (workspace_bytes < need) return CPATTN_ERR_WORKSPACE_TOO_SMALL;
  a.part_o = static_cast<float*>(workspace);
  a.part_lse = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + align256(size_t(b) * hq * a.nsplit * d * 4));
  a.scale_log2 = float(1.4426950408889634 * (scale == 0.f ? default_scale(d) : double(scale)));
  a.status = di->status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return d == 128 ? launch<128>(a, di, st) : launch<64>(a, di, st);
}
