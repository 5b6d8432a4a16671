// The shapes of calls over a cache in pages (csrc/paged_shape.h). Prints, for
// each line "sms b hq hkv d groups max_group cap" of the input,
//   <workspace asked for> <form: 0 prefix, 1 few, -1 refused> <CTAs> <rows kept of each> <runs of own keys>
#include <cstdio>

#include "../context_blockwise_causal_gb300/csrc/paged_shape.h"

using namespace cpattn;

int main() {
  int sms, b, hq, hkv, d, groups, most;
  long long cap;
  while (std::scanf("%d %d %d %d %d %d %d %lld", &sms, &b, &hq, &hkv, &d, &groups, &most, &cap) == 8) {
    const SharedForms f = shared_forms(sms, b, hq, hkv, d, groups, most);
    if (f.bytes == 0) {
      std::printf("0 -1 0 0 0\n");
      continue;
    }
    const bool few = takes_few(f, hq, hkv, groups, most, cap);
    const SharedShape& s = few ? f.few : f.prefix;
    std::printf("%zu %d %lld %d %d\n", f.bytes, few ? 1 : 0, static_cast<long long>(s.ctas), s.part_rows, s.own_runs);
  }
}
