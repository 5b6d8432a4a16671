// What the kernels of a paged cache share: where a sequence's keys lie, and
// what groups of sequences have in common.
//
// A page holds page_size tokens (a multiple of 16) of every KV head; row i of
// the tables names the pages of sequence i in order, so its token t is slot
// t % page_size of page tables[i][t / page_size]. An entry that names no page
// of the pool is never followed: its tokens count as zeros, or are not written,
// and bit 17 of the status word is set.
#pragma once
#include <cstdint>

#include "paged_shape.h"
#include "ptx.cuh"

namespace cpattn {

constexpr unsigned int kStatusPage = 1u << 17;
constexpr uint32_t kAllWaits = 0xffffffffu;  // none of a copying warp's waits is made to run out (abort self-test)

struct PagedPlace {
  const int* tables;  // [b][cols], rows tables_row apart
  int64_t tables_row;
  int64_t k_page, v_page;  // elements
  int pages, page_size;
};

__device__ __forceinline__ bool page_ok(int page, const PagedPlace& pg, unsigned int* status) {
  const bool ok = unsigned(page) < unsigned(pg.pages);
  if (!ok) atomicOr(status, kStatusPage);
  return ok;
}

// ---------------------------------------------------------------- groups
// Sequences offsets[g] .. offsets[g + 1] - 1 are group g, which has its first
// shared[g] tokens in common. A member that holds fewer tokens, or comes after
// max_group others, shares nothing. The rows of a group for one KV head are
// its members' query heads, G of each; unit_rows of them are a unit, whose
// common keys are cut into runs, one CTA each.
struct SharedPlan {
  const int* lengths;
  const int* shared;
  const int* offsets;  // nullptr: the whole batch is one group
  int groups, max_group;
  int b, hkv, G, cap;
  float token_bytes;  // of a token's key and value in one KV head
  int ctas;       // runs at most
  int unit_rows;
  int part_rows;  // rows kept of each CTA, min(unit_rows, a group's)
  // Without the prefix kernel (fixed_runs > 0) every unit has so many runs and
  // every group the units of the largest one; with it both follow the counts.
  int fixed_runs, fixed_units;
  GroupRuns* runs;
  float* part_o;    // [ctas][part_rows][D], normalised
  float* part_lse;  // [ctas][part_rows], base 2
};

// First sequence and members of a group that share.
__device__ __forceinline__ void shared_group(const SharedPlan& s, int g, int& first, int& size) {
  if (!s.offsets) {
    first = 0;
    size = s.b;
  } else {
    first = s.offsets[g];
    int end = s.offsets[g + 1];
    first = first < 0 ? 0 : (first < s.b ? first : s.b);
    end = end < first ? first : (end < s.b ? end : s.b);
    size = end - first;
  }
  if (size > s.max_group) size = s.max_group;
}
__device__ __forceinline__ int shared_count(const SharedPlan& s, int g) {
  const int c = s.shared[g];
  return c < 0 ? 0 : (c < s.cap ? c : s.cap);
}
__device__ __forceinline__ int shared_units(const SharedPlan& s, int size) {
  return (size * s.G + s.unit_rows - 1) / s.unit_rows;
}

// A sequence's place in its group, and the keys that it leaves to the group (0: none).
struct SharedSeq {
  int group, member, units, keys;
  GroupRuns at;
};
__device__ __forceinline__ SharedSeq shared_seq(const SharedPlan& s, int bi, int n) {
  SharedSeq r;
  r.group = 0;
  if (s.offsets) {  // the last group that begins at or before it
    int lo = 0, hi = s.groups;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s.offsets[mid] <= bi) lo = mid; else hi = mid;
    }
    r.group = lo;
  }
  int first, size;
  shared_group(s, r.group, first, size);
  r.member = bi - first;
  r.units = s.fixed_runs > 0 ? s.fixed_units : shared_units(s, size);
  const int c = shared_count(s, r.group);
  r.keys = r.member >= 0 && r.member < size && n >= c ? c : 0;
  r.at = {r.group * s.hkv * s.fixed_units * s.fixed_runs, s.fixed_runs};
  return r;
}
// (after the prefix kernel)
__device__ __forceinline__ void shared_runs(const SharedPlan& s, SharedSeq& r) {
  if (s.fixed_runs > 0) return;
  const int2 v = __ldcg(reinterpret_cast<const int2*>(s.runs + r.group));
  r.at = {v.x, v.y};
}

// Where the first run's result of a row stands (those of the other runs part_rows
// apart). `head`: query head within the KV head's.
__device__ __forceinline__ int64_t shared_at(const SharedPlan& s, const SharedSeq& r, int kvh, int head) {
  const int row = r.member * s.G + head;
  const int64_t cta = r.at.first + int64_t(kvh * r.units + row / s.unit_rows) * r.at.runs;
  return cta * s.part_rows + row % s.unit_rows;
}

}  // namespace cpattn
