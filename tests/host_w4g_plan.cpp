// Host program for tests/w4g_plan.py: what the integer 4-bit projections' plan
// (csrc/w4g.h, linked from the library) chooses for each line "rows n k group
// experts grouped indexed sms" of the standard input.
#include <cstdio>

#include "w4g.h"

int main() {
  long long rows;
  int n, k, group, experts, grouped, indexed, sms;
  static const int32_t some = 0;
  while (std::scanf("%lld %d %d %d %d %d %d %d", &rows, &n, &k, &group, &experts, &grouped, &indexed, &sms) == 8) {
    bsr::W4gArgs g = {};
    g.offsets = grouped ? &some : nullptr;  // only looked at for null
    g.rows = indexed ? &some : nullptr;
    g.a_rows = g.rows_max = rows;
    g.experts = experts;
    g.n = n;
    g.k = k;
    g.group = group;
    const bsr::W4gPlan p = bsr::w4g_plan(g, sms);
    std::printf("%d %d %d %d %d %d %d %d %d\n", p.few ? 1 : 0, p.gemv.rt, p.gemv.nt, p.gemv.ks, p.gemv.slots,
                p.gemv.grid, p.gemm.bm, p.gemm.split, p.gemm.grid);
  }
  return 0;
}
