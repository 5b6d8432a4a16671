// The shapes of calls over a cache in pages (csrc/paged_shape.h). Prints, for
// each line "sms b hq hkv d groups max_group cap" of the input,
//   <workspace asked for> <form: 0 prefix, 1 few, 2 sequences by themselves, -1 refused> <CTAs> <rows kept of each> <runs of own keys>
// and, with any argument, for each line "sms d G units keys" the runs of a call over whole sequences
#include <cstdio>

#include "../context_blockwise_causal_gb300/csrc/paged_shape.h"

using namespace cpattn;

int main(int argc, char**) {
  if (argc > 1) {
    int sms, d, G;
    long long units, keys;
    while (std::scanf("%d %d %d %lld %lld", &sms, &d, &G, &units, &keys) == 5)
      std::printf("%d\n", paged_split(sms, d, G, units, keys));
    return 0;
  }
  int sms, b, hq, hkv, d, groups, most;
  long long cap;
  while (std::scanf("%d %d %d %d %d %d %d %lld", &sms, &b, &hq, &hkv, &d, &groups, &most, &cap) == 8) {
    const SharedForms f = shared_forms(sms, b, hq, hkv, d, groups, most);
    if (f.bytes == 0) {
      std::printf("0 -1 0 0 0\n");
      continue;
    }
    const SharedForm form = shared_form(f, hq, hkv, groups, most, cap);
    const SharedShape& s = form == SharedForm::kFew ? f.few : f.prefix;
    if (form == SharedForm::kAlone) {
      const int G = hq / hkv;
      const int runs = paged_split(sms, d, G, int64_t(b) * hkv * ((G + unit_rows(G) - 1) / unit_rows(G)), cap);
      std::printf("%zu 2 0 0 %d\n", f.bytes, runs > kDecMaxCluster ? runs : 0);  // (runs whose results need a workspace)
      continue;
    }
    std::printf("%zu %d %lld %d %d\n", f.bytes, form == SharedForm::kFew ? 1 : 0, static_cast<long long>(s.ctas), s.part_rows,
                s.own_runs);
  }
}
