// Into how many runs the calls over a cache in pages cut their keys, which
// kernel takes the common ones of groups, and the workspace that this takes. No
// CUDA: host tests compile it by itself.
#pragma once
#include <algorithm>
#include <cstdint>

#include "decode_split.h"

namespace cpattn {

constexpr int kSharedRows = 256;  // the prefix kernel's units
constexpr int kSharedMaxCtas = 1 << 26;
constexpr int kJoinBatch = 8;  // results that a warp of the join kernel has on their way at once

// Of a group: the first of its runs' CTAs, and the runs of each of its units.
struct GroupRuns {
  int first, runs;
};

// Rows of a unit: 8 where they suffice (half of the work), or 16.
inline int unit_rows(int64_t rows) { return rows <= 8 ? 8 : 16; }

// CTAs of the paged kernel that an SM holds: its launch bounds ask the compiler for registers for so many, and
// no more fit (units of 16 heads of 64: five warps of 136 registers, of which three fit each quarter of an SM.
// Counted as three CTAs an SM, 24 sequences of 1000 to 2000 keys, 2 KV heads, were cut into runs that took
// two turns, 16.2 us; in one turn 10.5).
constexpr int paged_per_sm(int d, int unit_rows) { return d == 64 && unit_rows == 8 ? 4 : 2; }

// Runs over pages: the same rule, with the places of paged_per_sm, and more runs
// than a cluster's 8 already from 2048 keys on, of 256 keys or 16 of them: the
// kernel that joins them has four warps to a row and costs less than it saves.
// One sequence, d 128, us in 8 / 16 / 32 / 64 runs (captured graphs, caches cold): 4096
// keys, 8 KV heads 9.6 / 8.65 / 9.15 / 13.2, 1 KV head 9.4 / 7.4 / 6.8 / 7.3; 8192 keys
// 13.7 / 11.1 / 11.3 / 15.8 and 13.2 / 9.3 / 7.8 / 7.95; 32768 keys 36.3 / 25.9 / 25.4 /
// 29.4 (in the 38 that the rule takes 26.5) and 35.7 / 20.5 / 13.4 / 11.0.
// `keys` is what the tables have room for, since the lengths are on the device:
// wide tables are cut as if they were full. 16 sequences of 500 to 1000 keys, 64/8 heads,
// take 14.65 us in two runs each with tables for 1000, 19.4 in four, which take two turns,
// with tables for 131072; one of 1000 keys, 32/8 heads, 7.2 and 7.8.
inline int paged_split(int num_sms, int d, int G, int64_t units, int64_t keys) {
  const int64_t places = int64_t(paged_per_sm(d, unit_rows(G))) * num_sms;
  return choose_split(places, units, keys, keys < 2048 ? 0 : std::max<int64_t>(16, keys / 256));
}

// Common keys by the prefix kernel, whose matrix tiles have 128 rows, or, for
// groups of few rows, by the kernel that reads the own keys, a unit of its
// rows at a time: 16 rows behind 8192 keys of 8 heads (d 128, up to 256 own keys
// each) take 12.8 us there and 18.3 by the prefix kernel, 8 groups of 16 behind
// 2048 24.0 and 35.0. More rows are more units that read the same keys, which pays
// where there are few of those: 32 rows behind 1024 keys 8.7 and 12.8, behind 8192 17.4
// and 19.0, behind 32768 45.5 and 34.7; 64 rows behind 1024 keys 10.1 and 14.0, behind
// 20000 of one head 13.2 and 15.5, behind 8192 of 8 heads 35.6 and 20.2. The border is
// where the rounds take longer than the prefix kernel's plan, 128-row tiles and
// stores: 64 keys of a unit are 0.5 us of one of 304 places, 300000 keys of all units 7.7
// us of the call. How many keys there are is known here only as the tables' room for
// them: behind wide tables 32 rows take the prefix kernel whatever they share.
constexpr int kFewRows = 64, kFewMembers = 32;
inline bool may_be_few(int64_t rows, int max_group) { return rows <= kFewRows && max_group <= kFewMembers; }
inline bool is_few(int64_t rows, int hkv, int groups, int max_group, int64_t cap) {
  return may_be_few(rows, max_group) && (rows <= 16 || (rows + 7) / 8 * hkv * groups * cap <= 300000);
}

// Runs of the common and of the own keys and where their results go.
struct SharedShape {
  int unit_rows, part_rows, fixed_runs, fixed_units, own_rows, own_runs, join_warps;
  int64_t ctas;  // of the common keys
  size_t runs_bytes, lse_bytes, o_bytes, own_lse_bytes, own_o_bytes;
  // (results are stored in whole sectors, so the parts begin at the first multiple of 256)
  size_t bytes() const { return 256 + runs_bytes + lse_bytes + o_bytes + own_lse_bytes + own_o_bytes; }
};

inline bool shared_shape(SharedShape* s, bool few, int num_sms, int b, int hq, int hkv, int d, int groups, int max_group) {
  const int64_t G = hq / hkv, rows = int64_t(max_group) * G;
  if (rows >= int64_t(1) << 30) return false;
  // Few rows of one group: units of 8 though they read the common keys twice, since
  // theirs are the shorter rounds and the own keys need no more (16 rows behind 8192
  // keys: 12.8 us, in one unit 15.8). Of several groups: units of 16, which leave more runs to each
  // (8 groups of 16 rows behind 2048 keys: 23.9 us, with 8 rows 25.9).
  s->own_rows = unit_rows(few && groups > 1 ? rows : G);
  const int64_t own_units = int64_t(b) * hkv * ((G + s->own_rows - 1) / s->own_rows);
  // Own keys are mostly few, and how many is not known here: runs only where
  // sequences are few (64 sequences behind 32768 tokens, up to 1024 of their own: 66
  // us in one run each, 71 in two; 256 behind 16384, up to 2048: 243 and 254). Where
  // they are many this is slow: 5 sequences, 8 KV heads, of 2048 own keys at most 21 us, of
  // 32768 265; over whole sequences 11 and 67.
  s->own_runs = 1;
  while (s->own_runs < kDecMaxCluster && 2 * s->own_runs * own_units <= 64) s->own_runs *= 2;
  s->unit_rows = few ? s->own_rows : kSharedRows;
  const int64_t row_units = (rows + s->unit_rows - 1) / s->unit_rows, units = row_units * hkv * groups;
  if (units >= int64_t(1) << 30) return false;
  s->fixed_units = int(row_units);
  s->fixed_runs = 0;
  if (few) {
    // as many runs as fill the places that the own keys' CTAs leave
    const int64_t places = int64_t(paged_per_sm(d, s->own_rows)) * num_sms, own = own_units * s->own_runs;
    const int64_t runs = (places - std::min(own, places / 2)) / units;
    s->fixed_runs = int(runs < 1 ? 1 : runs > kDecMaxSplit ? kDecMaxSplit : runs);
    s->ctas = units * s->fixed_runs;
    s->join_warps = s->fixed_runs + s->own_runs > kJoinBatch ? 4 : 1;
  } else {
    // One run per SM, or as many as it takes for the units to be at most half of
    // them (so that runs of about the same length exist, whatever the groups'
    // lengths turn out to be).
    s->ctas = num_sms * ((2 * units + num_sms - 1) / num_sms);
    s->join_warps = s->ctas / units + s->own_runs > kJoinBatch ? 4 : 1;
  }
  if (s->ctas >= kSharedMaxCtas || s->ctas + own_units * s->own_runs >= int64_t(1) << 31) return false;
  s->part_rows = int(std::min<int64_t>(s->unit_rows, (rows + 15) / 16 * 16));
  const size_t parts = size_t(s->ctas) * s->part_rows, own_parts = size_t(b) * hq * s->own_runs;
  s->runs_bytes = align256(size_t(groups) * sizeof(GroupRuns));
  s->lse_bytes = align256(parts * 4);
  s->o_bytes = align256(parts * d * 4);
  s->own_lse_bytes = align256(own_parts * 4);
  s->own_o_bytes = align256(own_parts * d * 4);
  return true;
}

// The forms that a call may take, those whose results can be numbered, and the
// workspace that holds either (0: the call is refused). One form may be there
// without the other: 2^26 bounds the common keys' CTAs, which the prefix kernel
// rounds up to whole SMs.
struct SharedForms {
  bool prefix_ok, few_ok;
  SharedShape prefix, few;
  size_t bytes;
};
inline SharedForms shared_forms(int num_sms, int b, int hq, int hkv, int d, int groups, int max_group) {
  SharedForms f{};
  f.prefix_ok = shared_shape(&f.prefix, false, num_sms, b, hq, hkv, d, groups, max_group);
  f.few_ok = may_be_few(int64_t(max_group) * (hq / hkv), max_group) &&
             shared_shape(&f.few, true, num_sms, b, hq, hkv, d, groups, max_group);
  if (f.prefix_ok) f.bytes = f.prefix.bytes();
  if (f.few_ok) f.bytes = std::max(f.bytes, f.few.bytes());
  return f;
}

// The form that a call takes. Every CTA of the prefix kernel looks through all
// groups (prefix_plan), some 36 us of them for 1000, and there are as many CTAs as
// groups: so groups of few rows take the other form from 129 on (5 sequences of
// 4 heads behind 256 keys, d 64, us by the prefix kernel and the other one: 64 groups
// 14.6 and 12.5, 256 61 and 33, 1000 488 and 125, 4000 7600 and 515; 16 of them behind 2048,
// 8 KV heads, d 128: 128 groups 619 and 691, 256 1465 and 1382, 1000 11100 and 5470), and
// sequences of more than 1024 larger groups are computed by themselves.
constexpr int kManyGroups = 128, kPlanGroups = 1024;
enum class SharedForm { kPrefix, kFew, kAlone };
inline SharedForm shared_form(const SharedForms& f, int hq, int hkv, int groups, int max_group, int64_t cap) {
  if (f.few_ok && (!f.prefix_ok || groups > kManyGroups || is_few(int64_t(max_group) * (hq / hkv), hkv, groups, max_group, cap)))
    return SharedForm::kFew;
  return groups > kPlanGroups ? SharedForm::kAlone : SharedForm::kPrefix;
}

}  // namespace cpattn
