// Prints the attention's plan for the sizes given on stdin, one line each:
//   B R Hq Hkv D P max_ctx  ->  prefix_parts prefix_chunk workspace own_parts wrong own[6]
// wrong counts lengths (all to 5000, then every 61st) whose ranges are not
// whole tiles, leave keys out or are more than own_parts; own[i] is the range
// of a sequence with 1, 128, 701, 4001, 20000 and 100000 keys of its own, 0
// past the capacity.  Built from the library's own header (no GPU, no HIP calls).
#include <cstdio>

#include "sv_plan.h"

int main() {
  long long B, R, Hq, Hkv, D, P, ctx;
  while (std::scanf("%lld %lld %lld %lld %lld %lld %lld", &B, &R, &Hq, &Hkv, &D, &P, &ctx) == 7) {
    const sv::AttendPlan L = sv::plan_attention(B, R, Hq, Hkv, static_cast<int>(D), P, ctx);
    long long wrong = 0;
    const auto look = [&](long long keys) {
      const long long own = sv::attend_own_range(L.split, static_cast<int>(keys));
      const long long parts = own > 0 ? (keys + own - 1) / own : -1;
      if (own < 128 || own % 128 != 0 || parts < 1 || parts > L.own_parts) ++wrong;
    };
    for (long long keys = 1; keys < ctx + R; keys += keys < 5000 ? 1 : 61) look(keys);
    look(ctx + R);
    std::printf("%d %d %lld %d %lld", L.prefix_parts, L.prefix_chunk, static_cast<long long>(L.total), L.own_parts, wrong);
    for (const long long keys : {1, 128, 701, 4001, 20000, 100000})
      std::printf(" %d", keys <= ctx + R ? sv::attend_own_range(L.split, static_cast<int>(keys)) : 0);
    std::printf("\n");
  }
  return 0;
}
