// Prints the plan of attention over pages for the sizes given on stdin, one line each:
//   B R Hq Hkv D P max_ctx f8  ->  few direct prefix_parts prefix_chunk workspace own_parts wrong items
// wrong counts lengths (all to 5000, then every 61st) whose ranges are not
// whole tiles, leave keys out or are more than own_parts; items is the number of
// stacked rows that the items of a sequence hold.  Built from the library's own header
// (no GPU, no HIP calls).
#include <cstdio>

#include "sv_plan.h"

int main() {
  long long B, R, Hq, Hkv, D, P, ctx, f8;
  while (std::scanf("%lld %lld %lld %lld %lld %lld %lld %lld", &B, &R, &Hq, &Hkv, &D, &P, &ctx, &f8) == 8) {
    const sv::PagedPlan L = sv::plan_paged(B, R, Hq, Hkv, static_cast<int>(D), P, ctx, f8 != 0);
    long long wrong = 0;
    const auto look = [&](long long keys) {
      const long long own = sv::attend_own_range(L.split, static_cast<int>(keys));
      const long long parts = own > 0 ? (keys + own - 1) / own : -1;
      if (own < 128 || own % 128 != 0 || parts < 1 || parts > L.own_parts) ++wrong;
    };
    for (long long keys = 1; keys < ctx + R; keys += keys < 5000 ? 1 : 61) look(keys);
    look(ctx + R);
    std::printf("%d %d %d %d %lld %d %lld %d\n", L.few, L.direct, L.prefix_parts, L.prefix_chunk, static_cast<long long>(L.total), L.own_parts,
                wrong, L.own_tiles * (L.few ? L.few : 32 * L.own_waves));
  }
  return 0;
}
