// C-ABI entry points of the paged cache (include/cpattn.h): new tokens into
// it, single-token attention over it, and the same for sequences that begin
// alike.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <numeric>

#include "../../include/cpattn.h"
#include "api_common.h"
#include "append_kernel.cuh"
#include "decode_host.h"
#include "paged_kernel.cuh"
#include "prefix_kernel.cuh"
#include "qk_host.h"
#include "tmap.h"

using namespace cpattn;

namespace {

// Strides of a pool [pages, page_size, hkv, d]: 16-byte pieces, no two
// elements in one place, and extents that 64-bit offsets and tensor copies hold.
bool pool_strides_ok(const cpattn_pages* p, int hkv, int d, int64_t page, int64_t token, int64_t head) {
  struct Dim {
    int64_t stride, size;
  } dims[3] = {{page, p->pages}, {token, p->page_size}, {head, hkv}};
  std::sort(dims, dims + 3, [](const Dim& x, const Dim& y) { return x.stride < y.stride; });
  int64_t span = d;
  for (const Dim& x : dims) {
    if (x.size == 1) continue;
    if (x.stride % 8 != 0 || x.stride < span || x.stride >= int64_t(1) << 38) return false;
    if (x.size - 1 > ((int64_t(1) << 46) - span) / x.stride) return false;
    span += x.stride * (x.size - 1);
  }
  return true;
}

int64_t capacity(const cpattn_pages* p) { return int64_t(p->table_cols) * p->page_size; }

int check_pages(const cpattn_pages* p, int hkv, int d) {
  if (!p || !p->k || !p->v || !p->tables) return CPATTN_ERR_NULL_PTR;
  if (hkv < 1 || (d != 64 && d != 128)) return CPATTN_ERR_INVALID_ARG;
  if (p->pages < 1 || p->page_size < 16 || p->page_size % 16 != 0 || p->table_cols < 1 || p->tables_row < 0)
    return CPATTN_ERR_INVALID_ARG;
  if (p->page_size > (1 << 30) || capacity(p) > (1 << 30)) return CPATTN_ERR_INVALID_ARG;
  if (!pool_strides_ok(p, hkv, d, p->k_page, p->k_token, p->k_head) ||
      !pool_strides_ok(p, hkv, d, p->v_page, p->v_token, p->v_head))
    return CPATTN_ERR_INVALID_ARG;
  if (!aligned16(p->k) || !aligned16(p->v) || !aligned4(p->tables)) return CPATTN_ERR_MISALIGNED;
  return CPATTN_OK;
}

PagedPlace place_of(const cpattn_pages* p) {
  PagedPlace r;
  r.tables = p->tables;
  r.tables_row = p->tables_row;
  r.k_page = p->k_page;
  r.v_page = p->v_page;
  r.pages = p->pages;
  r.page_size = p->page_size;
  return r;
}

// Shapes of a decode over pages; b * hq * kDecMaxSplit rows fit 32 bits.
int check_decode(const cpattn_pages* p, int b, int hq, int hkv, int d, int window, int sinks) {
  if (b < 1 || hq < 1 || hkv < 1 || window < 0 || sinks < 0 || hq % hkv != 0) return CPATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return CPATTN_ERR_INVALID_ARG;
  if (int64_t(b) * hq * kDecMaxSplit >= (int64_t(1) << 31)) return CPATTN_ERR_INVALID_ARG;
  return p ? check_pages(p, hkv, d) : CPATTN_OK;
}

// What the calls' arguments have in common; o and lse as cpattn_decode.
void fill_decode(PagedArgs* pa, const void* q, const cpattn_pages* p, const int* lengths, void* o, float* lse, int b,
                 int hq, int hkv, int d, int64_t q_batch, float scale, DeviceInfo* di) {
  *pa = PagedArgs{};
  DecodeArgs* a = &pa->d;
  a->q = static_cast<const __nv_bfloat16*>(q);
  a->lengths = lengths;
  a->o = static_cast<__nv_bfloat16*>(o);
  a->lse = lse;
  a->q_batch = q_batch;
  a->b = b;
  a->hq = hq;
  a->hkv = hkv;
  a->G = hq / hkv;
  a->cap = int(capacity(p));
  a->row_groups = (a->G + unit_rows(a->G) - 1) / unit_rows(a->G);
  a->scale_log2 = float(1.4426950408889634 * (scale == 0.f ? default_scale(d) : double(scale)));
  a->status = di->status;
  pa->pg = place_of(p);
}

int check_pointers(const void* q, const int* lengths, const void* o, const float* lse, const void* workspace,
                   int64_t q_batch, float scale) {
  if (!q || !lengths || !o || !lse) return CPATTN_ERR_NULL_PTR;
  if (!(scale == 0.f || valid_scale(scale)) || q_batch < 0 || q_batch % 8 != 0) return CPATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(o) || !aligned4(lse) || !aligned4(lengths) || !aligned16(workspace))
    return CPATTN_ERR_MISALIGNED;
  return CPATTN_OK;
}

int check_groups(int b, int groups, int max_group) {
  return groups < 1 || groups > b || max_group < 1 || max_group > b ? CPATTN_ERR_INVALID_ARG : CPATTN_OK;
}

// Descriptors of the pools for copies of `box` tokens and 64 `cols` features.
bool encode_pools(CUtensorMap* tk, CUtensorMap* tv, const cpattn_pages* p, int hkv, int d, int box, int cols) {
  return encode_bf16_pages(tk, p->k, p->pages, p->page_size, hkv, d, p->k_page, p->k_token, p->k_head, box, cols) &&
         encode_bf16_pages(tv, p->v, p->pages, p->page_size, hkv, d, p->v_page, p->v_token, p->v_head, box, cols);
}

template <int D, PagedKind kKind, int kT>
int launch_paged_as(PagedArgs& pa, const cpattn_pages* p, DeviceInfo* di, cudaStream_t st) {
  using C = PagedCfg<D>;
  constexpr bool kParts = kKind != PagedKind::kWhole;
  const DecodeArgs& a = pa.d;
  const int64_t ctas = pa.common_ctas + int64_t(a.b) * a.hkv * a.row_groups * a.nsplit;
  const auto kernel = cpattn_decode_paged_kernel<D, kKind, kT>;
  CUtensorMap tk, tv;
  pa.box = std::gcd(p->page_size, 2 * kDecBlock);
  if (!encode_pools(&tk, &tv, p, a.hkv, D, pa.box, D / 64) ||
      !allow_smem(di->paged_attr[int(kKind) * 4 + (kT - 1) * 2 + (D == 128 ? 1 : 0)], kernel, C::kSmemBytes))
    return CPATTN_ERR_CUDA;
  cudaError_t e = launch_runs(kernel, ctas, kPagedThreads, kParts ? 1 : a.nsplit, C::kSmemBytes, true, st, tk, tv, pa);
  const int64_t out_rows = int64_t(a.b) * a.hq;
  if (e == cudaSuccess && (kParts || a.nsplit > kDecMaxCluster))
    e = pa.join_warps == 1 ? launch_chained(cpattn_shared_join_kernel<D, 1>, (out_rows + 3) / 4, 128, st, pa)
                           : launch_chained(cpattn_shared_join_kernel<D, 4>, out_rows, 128, st, pa);
  return launched(e);
}
template <int D, PagedKind kKind>
int launch_paged(int rows, PagedArgs& pa, const cpattn_pages* p, DeviceInfo* di, cudaStream_t st) {
  return rows == 8 ? launch_paged_as<D, kKind, 1>(pa, p, di, st) : launch_paged_as<D, kKind, 2>(pa, p, di, st);
}

template <int D>
int launch_shared(bool few, int own_rows, PagedArgs& pa, const PrefixArgs& a, const cpattn_pages* p, DeviceInfo* di,
                  cudaStream_t st) {
  if (few) return launch_paged<D, PagedKind::kBoth>(own_rows, pa, p, di, st);
  CUtensorMap tk, tv;
  if (!encode_pools(&tk, &tv, p, a.sh.hkv, D, a.box, a.box == kTile ? D / 64 : 1) ||
      !allow_smem(di->prefix_attr[D == 128 ? 1 : 0], cpattn_prefix_kernel<D>, PrefixCfg<D>::kSmemBytes))
    return CPATTN_ERR_CUDA;
  const int rc = launched(
      launch_runs(cpattn_prefix_kernel<D>, a.sh.ctas, kFwdThreads, 1, PrefixCfg<D>::kSmemBytes, true, st, tk, tv, a));
  return rc ? rc : launch_paged<D, PagedKind::kOwn>(own_rows, pa, p, di, st);
}

template <int D, bool kInter>
int launch_append(AppendArgs& a, DeviceInfo* di, cudaStream_t st) {
  constexpr int kRows = 32 / (D / 16), kWarps = kQkThreads / 32;
  const int64_t heads = int64_t(a.qk.t[0].h) + 2 * int64_t(a.qk.t[1].h);
  const int64_t groups = (heads + kRows - 1) / kRows;
  const int64_t tokens = int64_t(a.qk.b) * a.qk.n;
  // A token's heads stay with one warp (one set of cosines, one look-up) unless
  // that leaves fewer than eight warps per SM; then they spread over more.
  const int64_t want = (int64_t(di->num_sms) * 8 + tokens - 1) / tokens;
  const int64_t split = want < groups ? want : groups;
  a.qk.heads_per = int((groups + split - 1) / split * kRows);
  a.qk.split = int((heads + a.qk.heads_per - 1) / a.qk.heads_per);
  const int64_t ctas = (tokens * a.qk.split + kWarps - 1) / kWarps, most = int64_t(di->num_sms) * 2;  // resident at once
  return launched(launch_chained(cpattn_append_kernel<D, kInter>, ctas < most ? ctas : most, kQkThreads, st, a));
}

int decode_paged(const void* q, const cpattn_pages* pages, const int* lengths, void* o, float* lse, void* workspace,
                 size_t workspace_bytes, int b, int hq, int hkv, int d, int64_t q_batch, int window, int sinks,
                 float scale, void* stream, uint32_t waits) {
  int rc = check_pointers(q, lengths, o, lse, workspace, q_batch, scale);
  if (rc) return rc;
  if (!pages) return CPATTN_ERR_NULL_PTR;
  if ((rc = check_decode(pages, b, hq, hkv, d, window, sinks))) return rc;
  DeviceInfo* di = nullptr;
  if ((rc = device_info(&di))) return rc;
  PagedArgs pa;
  fill_decode(&pa, q, pages, lengths, o, lse, b, hq, hkv, d, q_batch, scale, di);
  DecodeArgs& a = pa.d;
  a.window = window;
  a.sinks = window > 0 ? sinks : 0;
  a.nsplit = paged_split(di->num_sms, d, a.G, int64_t(b) * hkv * a.row_groups, max_keys(a.cap, window, sinks));
  pa.join_warps = 4;
  pa.copy_waits = waits;
  const size_t need = workspace_for(b, hq, d, a.nsplit);
  if (need > 0 && !workspace) return CPATTN_ERR_NULL_PTR;
  if (workspace_bytes < need) return CPATTN_ERR_WORKSPACE_TOO_SMALL;
  a.part_o = static_cast<float*>(workspace);
  a.part_lse = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + align256(size_t(b) * hq * a.nsplit * d * 4));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int rows = unit_rows(a.G);
  return d == 128 ? launch_paged<128, PagedKind::kWhole>(rows, pa, pages, di, st)
                  : launch_paged<64, PagedKind::kWhole>(rows, pa, pages, di, st);
}

int decode_shared(const void* q, const cpattn_pages* pages, const int* lengths, const int* shared,
                  const int* group_offsets, int groups, int max_group, void* o, float* lse, void* workspace,
                  size_t workspace_bytes, int b, int hq, int hkv, int d, int64_t q_batch, float scale, void* stream,
                  uint32_t waits) {
  int rc = check_pointers(q, lengths, o, lse, workspace, q_batch, scale);
  if (rc) return rc;
  if (!pages || !shared || !workspace) return CPATTN_ERR_NULL_PTR;
  if ((rc = check_decode(pages, b, hq, hkv, d, 0, 0)) || (rc = check_groups(b, groups, max_group))) return rc;
  if (!group_offsets && groups != 1) return CPATTN_ERR_INVALID_ARG;
  if (!aligned4(shared) || !aligned4(group_offsets)) return CPATTN_ERR_MISALIGNED;
  DeviceInfo* di = nullptr;
  if ((rc = device_info(&di))) return rc;
  const SharedForms forms = shared_forms(di->num_sms, b, hq, hkv, d, groups, max_group);
  if (forms.bytes == 0) return CPATTN_ERR_INVALID_ARG;
  if (workspace_bytes < forms.bytes) return CPATTN_ERR_WORKSPACE_TOO_SMALL;
  const SharedForm form = shared_form(forms, hq, hkv, groups, max_group, capacity(pages));
  if (form == SharedForm::kAlone)  // (so many sequences need no workspace)
    return decode_paged(q, pages, lengths, o, lse, workspace, workspace_bytes, b, hq, hkv, d, q_batch, 0, 0, scale, stream,
                        waits);
  const bool few = form == SharedForm::kFew;
  const SharedShape& shape = few ? forms.few : forms.prefix;
  PagedArgs pa;
  fill_decode(&pa, q, pages, lengths, o, lse, b, hq, hkv, d, q_batch, scale, di);
  DecodeArgs& a = pa.d;
  a.nsplit = shape.own_runs;
  a.row_groups = (a.G + shape.own_rows - 1) / shape.own_rows;
  pa.join_warps = shape.join_warps;
  pa.copy_waits = waits;
  pa.common_ctas = few ? int(shape.ctas) : 0;
  uint8_t* ws = reinterpret_cast<uint8_t*>(align256(reinterpret_cast<uintptr_t>(workspace)));
  const auto take = [&ws](size_t bytes) {
    uint8_t* at = ws;
    ws += bytes;
    return at;
  };
  SharedPlan& sh = pa.sh;
  sh.lengths = lengths;
  sh.shared = shared;
  sh.offsets = group_offsets;
  sh.groups = groups;
  sh.max_group = max_group;
  sh.b = b;
  sh.hkv = hkv;
  sh.G = a.G;
  sh.cap = a.cap;
  sh.token_bytes = float(4 * d);
  sh.ctas = int(shape.ctas);
  sh.unit_rows = shape.unit_rows;
  sh.fixed_runs = shape.fixed_runs;
  sh.fixed_units = shape.fixed_units;
  sh.part_rows = shape.part_rows;
  sh.runs = reinterpret_cast<GroupRuns*>(take(shape.runs_bytes));
  sh.part_lse = reinterpret_cast<float*>(take(shape.lse_bytes));
  sh.part_o = reinterpret_cast<float*>(take(shape.o_bytes));
  a.part_lse = reinterpret_cast<float*>(take(shape.own_lse_bytes));
  a.part_o = reinterpret_cast<float*>(take(shape.own_o_bytes));
  PrefixArgs p;
  p.sh = sh;
  p.pg = pa.pg;
  p.q = a.q;
  p.q_batch = q_batch;
  p.hq = hq;
  p.sms = di->num_sms;
  p.box = std::gcd(pages->page_size, kTile);
  p.scale_log2 = a.scale_log2;
  p.status = di->status;
  p.producer_waits = waits;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return d == 128 ? launch_shared<128>(few, shape.own_rows, pa, p, pages, di, st)
                  : launch_shared<64>(few, shape.own_rows, pa, p, pages, di, st);
}

}  // namespace

extern "C" int cpattn_append_paged(const cpattn_rows* k, const cpattn_rows* v, const cpattn_pages* pages,
                                   const int* lengths, const int* cu_tokens, int seqs, const cpattn_rows* q,
                                   const cpattn_rows* q_out, int b, int n, int hq, int hkv, int d,
                                   const cpattn_rotary* rotary, void* stream) {
  if (!k || !v || !lengths || (!q) != (!q_out)) return CPATTN_ERR_NULL_PTR;
  AppendArgs a = {};
  int rc;
  if ((rc = check_pages(pages, hkv, d))) return rc;
  if (b < 1 || n < 1 || seqs < 1 || hq < 0 || (hq == 0) != (!q)) return CPATTN_ERR_INVALID_ARG;
  if (cu_tokens ? b != 1 : seqs != b) return CPATTN_ERR_INVALID_ARG;
  if (seqs > 1 && pages->tables_row < pages->table_cols) return CPATTN_ERR_INVALID_ARG;
  if (rotary) {
    // positions: the given ones, or each token's place in its sequence
    if (rotary->rank >= 0 || rotary->cu_seqlens) return CPATTN_ERR_INVALID_ARG;
    cpattn_rotary plan = *rotary;
    plan.s = n;
    if ((rc = fill_rotary(&plan, b, n, d, 0, &a.qk))) return rc;
  } else {
    a.qk.b = b;
    a.qk.n = n;
    a.qk.magnitude = 1.f;
  }
  if ((rc = check_rows(k, b, n, hkv, d, false)) || (rc = check_rows(v, b, n, hkv, d, false))) return rc;
  if (q && ((rc = check_rows(q, b, n, hq, d, false)) || (rc = check_rows(q_out, b, n, hq, d, true)))) return rc;
  if ((int64_t(hq) + 2 * int64_t(hkv)) * d >= kQkMaxFeatures) return CPATTN_ERR_INVALID_ARG;
  if (!aligned4(lengths) || !aligned4(cu_tokens)) return CPATTN_ERR_MISALIGNED;
  DeviceInfo* di = nullptr;
  if ((rc = device_info(&di))) return rc;
  if (q) set_tensor(&a.qk.t[0], q, nullptr, q_out, nullptr, hq);
  set_tensor(&a.qk.t[1], k, nullptr, k, nullptr, hkv);
  a.qk.status = di->status;
  a.v = static_cast<const __nv_bfloat16*>(v->data);
  a.v_batch = v->batch_stride;
  a.v_row = v->token_stride;
  a.k_pool = static_cast<__nv_bfloat16*>(pages->k);
  a.v_pool = static_cast<__nv_bfloat16*>(pages->v);
  a.pg = place_of(pages);
  a.k_token = pages->k_token;
  a.k_head = pages->k_head;
  a.v_token = pages->v_token;
  a.v_head = pages->v_head;
  a.lengths = lengths;
  a.cu = cu_tokens;
  a.seqs = seqs;
  a.cap = int(capacity(pages));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (rotary && rotary->layout == CPATTN_ROPE_INTERLEAVED)
    return d == 128 ? launch_append<128, true>(a, di, st) : launch_append<64, true>(a, di, st);
  return d == 128 ? launch_append<128, false>(a, di, st) : launch_append<64, false>(a, di, st);
}

extern "C" size_t cpattn_decode_paged_workspace_bytes(int b, int hq, int hkv, int d, int cap, int window, int sinks) {
  if (check_decode(nullptr, b, hq, hkv, d, window, sinks) || cap < 1 || cap > (1 << 30)) return 0;
  DeviceInfo* di = nullptr;
  if (device_info(&di)) return 0;
  const int G = hq / hkv;
  const int64_t units = int64_t(b) * hkv * ((G + unit_rows(G) - 1) / unit_rows(G));
  return workspace_for(b, hq, d, paged_split(di->num_sms, d, G, units, max_keys(cap, window, sinks)));
}

extern "C" int cpattn_decode_paged(const void* q, const cpattn_pages* pages, const int* lengths, void* o, float* lse,
                                   void* workspace, size_t workspace_bytes, int b, int hq, int hkv, int d,
                                   int64_t q_batch, int window, int sinks, float scale, void* stream) {
  return decode_paged(q, pages, lengths, o, lse, workspace, workspace_bytes, b, hq, hkv, d, q_batch, window, sinks, scale,
                      stream, kAllWaits);
}

extern "C" size_t cpattn_decode_shared_workspace_bytes(int b, int hq, int hkv, int d, int groups, int max_group) {
  if (check_decode(nullptr, b, hq, hkv, d, 0, 0) || check_groups(b, groups, max_group)) return 0;
  DeviceInfo* di = nullptr;
  if (device_info(&di)) return 0;
  return shared_forms(di->num_sms, b, hq, hkv, d, groups, max_group).bytes;  // whichever form the call takes
}

extern "C" int cpattn_decode_shared(const void* q, const cpattn_pages* pages, const int* lengths, const int* shared,
                                    const int* group_offsets, int groups, int max_group, void* o, float* lse,
                                    void* workspace, size_t workspace_bytes, int b, int hq, int hkv, int d,
                                    int64_t q_batch, float scale, void* stream) {
  return decode_shared(q, pages, lengths, shared, group_offsets, groups, max_group, o, lse, workspace, workspace_bytes, b, hq,
                       hkv, d, q_batch, scale, stream, kAllWaits);
}

// Self-test of the abort path: as the two calls, but the copying warps give up
// at their next wait for free room after so many.
extern "C" int cpattn_selftest_abort_paged(const void* q, const cpattn_pages* pages, const int* lengths,
                                           const int* shared, void* o, float* lse, void* workspace,
                                           size_t workspace_bytes, int b, int hq, int hkv, int d, int64_t q_batch,
                                           unsigned int waits, void* stream) {
  if (!shared)
    return decode_paged(q, pages, lengths, o, lse, workspace, workspace_bytes, b, hq, hkv, d, q_batch, 0, 0, 0.f, stream,
                        waits);
  return decode_shared(q, pages, lengths, shared, nullptr, 1, b, o, lse, workspace, workspace_bytes, b, hq, hkv, d, q_batch,
                       0.f, stream, waits);
}
