// The workspace of plans with shared prefixes, with the room to widen and without: a plan a line from
// stdin, the two totals and the tiles to widen to stdout.  Built by tests/test_prefix_workspace.py.
#include <cstdio>

#include "shim.h"
#include "mla_common_host.h"
#include "mla_prefix_host.h"

int main() {
  long long B, H, max_q, packed, total_q, max_len, kv, groups, workers;
  while (std::scanf("%lld %lld %lld %lld %lld %lld %lld %lld %lld", &B, &H, &max_q, &packed, &total_q, &max_len, &kv, &groups,
                    &workers) == 9) {
    mla::Layout full{}, least{};
    mla::PrefixLayout pre{}, pre_least{};
    const size_t header = sizeof(int) * mla::kHdrWords;
    const bool a = mla::make_prefix_layout(B, H, max_q, packed != 0, total_q, max_len, (int)kv, groups, (int)workers, header, &full,
                                           &pre);
    const bool b = mla::make_prefix_layout(B, H, max_q, packed != 0, total_q, max_len, (int)kv, groups, (int)workers, header, &least,
                                           &pre_least, false);
    if (a != b || !a) return 3;
    // the list's regions are in the same places, so that tools find them whichever a run used
    if (full.items != least.items || full.worker_ranges != least.worker_ranges || pre_least.wide_tiles != 0) return 5;
    std::printf("%zu %zu %d\n", full.total, least.total, pre.wide_tiles);
  }
  return 0;
}
