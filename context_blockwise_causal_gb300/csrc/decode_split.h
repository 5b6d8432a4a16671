// How many runs a sequence's keys are cut into for single-token attention, and
// the workspace that this takes. No CUDA: host tests compile it by itself.
#pragma once
#include <cstdint>

#include "align.h"

namespace cpattn {

constexpr int kDecMaxCluster = 8;  // the portable cluster size
constexpr int kDecMaxSplit = 64;

// Keys a sequence can see at most.
inline int64_t max_keys(int cap, int window, int sinks) {
  if (window == 0) return cap;
  const int64_t seen = int64_t(window) + sinks;
  return seen < cap ? seen : cap;
}

// Runs per (sequence, KV head group), for places CTAs at once: two fit an SM.
//  * As many as fill the places without a second wave, of 64 keys or more (one
//    round of a CTA's warps), up to a cluster: 8 of one 1028-key sequence with
//    8 KV heads take 6.5 us, 4 take 7.1; with 8 such sequences 4 take 10.7 us
//    and 8, a second wave, 16.9.
//  * Runs of 2048 keys or more may fill the places twice, which levels out
//    different lengths: 16 sequences of 32K to 64K keys take 442 us in 4 runs,
//    478 in 2 and 453 in 8.
//  * Where a cluster's 8 leave half of the places empty, such long runs go up
//    to all places through device memory (one 131K-key sequence, 8 KV heads:
//    91 us in 38 runs with their join, 132 in 8). Clusters of 16 find too few
//    places together.
inline int choose_split(int64_t places, int64_t units, int64_t keys, int64_t long_runs) {
  int64_t s = 1;
  while (2 * s <= kDecMaxCluster) {
    const int64_t ctas = 2 * s * units, run = keys / (2 * s);
    if (!(ctas <= places ? run >= 64 : ctas <= 2 * places && run >= 2048)) break;
    s *= 2;
  }
  if (s == kDecMaxCluster && 2 * s * units <= places) {
    int64_t more = places / units;
    if (more > long_runs) more = long_runs;
    if (more > s) s = more < kDecMaxSplit ? more : kDecMaxSplit;
  }
  return int(s);
}
inline int choose_split(int num_sms, int64_t units, int64_t keys) {
  return choose_split(2 * int64_t(num_sms), units, keys, keys / 2048);
}

// Workspace bytes (0: none).
inline size_t workspace_for(int b, int hq, int d, int nsplit) {
  if (nsplit <= kDecMaxCluster) return 0;
  const size_t rows = size_t(b) * hq * nsplit;
  return align256(rows * d * 4) + align256(rows * 4);
}

}  // namespace cpattn
