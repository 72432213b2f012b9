// Checks of the distillation kernel's layout of rows over CTAs and shared
// memory (lin_distill.h), run on the CPU by tests/test_distill_layout.py:
// prints "ok" or the first violated property.
#include <cstdio>

#include "lin_distill.h"

static int fail(const char* what, int warps, long long units, int K, const lin::DistillLayout& d) {
  std::printf("FAIL %s (%d warps, %lld units, K %d: cluster %d segs %d tile %d slots %d smem %zu)\n",
              what, warps, units, K, d.cluster, d.segs, d.tile, d.slots, d.smem);
  return 1;
}

int main() {
  for (int warps : {1, 2, 4, 8})
    for (int K = 0; K <= 1024; K += K < 900 ? 25 : 1) {
      // all widths up to two parts of the widest cluster, then coarser up to 2^31 entries
      for (long long units = 1; units <= (1LL << 29); units += units < 1200 ? 1 : units / 97) {
        if (warps < 8 && units > lin::distill_units(warps)) break;   // (the next width's)
        const lin::DistillLayout d = lin::distill_layout(warps, units, K);
        if (d.cluster < 1 || d.cluster > lin::kMaxCluster || (d.cluster & (d.cluster - 1)))
          return fail("cluster", warps, units, K, d);
        if (d.tile < 1 || d.tile > lin::distill_units(warps)) return fail("tile", warps, units, K, d);
        if ((long long)d.cluster * d.segs * d.tile < units) return fail("row not covered", warps, units, K, d);
        if (d.slots < 1 || d.slots > lin::kSlots) return fail("slots", warps, units, K, d);
        if (d.segs <= 2 && d.slots < d.segs) return fail("short row streamed twice", warps, units, K, d);
        // (a CTA may have 232448 bytes)
        if (d.smem + lin::kDistillStatic > 232448) return fail("shared memory", warps, units, K, d);
        if (d.smem != (size_t)d.slots * d.tile * 16 + (size_t)((K + 3) / 4 * 4) * 36)
          return fail("bytes", warps, units, K, d);
      }
    }
  std::puts("ok");
  return 0;
}
