// CPU check of the launch rules of the expert-layer calls
// (cluster_distributed_shared_gb300/csrc/launch_rules.h).  Prints "ok" and
// exits 0 when every check holds.
#include <stdio.h>

#include <initializer_list>

#include "launch_rules.h"

using namespace dsmh;

static int failures = 0;

#define CHECK(cond)                                              \
  do {                                                           \
    if (!(cond)) {                                               \
      printf("FAIL %s:%d: %s\n", __FILE__, __LINE__, #cond);     \
      ++failures;                                                \
    }                                                            \
  } while (0)

// Resident clusters of s CTAs that fill an SM each, as measured on 152 SMs.
static int resident(int s) { return s == 8 ? 15 : (s == 4 ? 36 : (s == 2 ? 76 : 152)); }

int main() {
  // Every tile's cluster is resident, and each CTA, of four at least, has four
  // stages of a narrow tile or eight of a wide one: with fewer the join costs
  // more than the split saves.
  CHECK(split_stages(16) == 4 && split_stages(64) == 8);
  for (int stages = 4; stages <= 8; stages += 4)
    for (int most = 1; most <= 8; most *= 2)
      for (int64_t depth = 1; depth <= 128; ++depth)
        for (int64_t tiles = 1; tiles <= 400; ++tiles) {
          const int split = split_for(tiles, depth, stages, most, resident);
          CHECK(split >= 1 && split <= most && (split & (split - 1)) == 0);
          if (split > 1) {
            CHECK(tiles <= resident(split));
            CHECK(depth >= stages * split && depth >= 4 * stages);
          }
          // No smaller than it could be.
          if (split < most && depth >= 4 * stages && depth >= 2 * stages * split) CHECK(tiles > resident(2 * split));
        }
  CHECK(split_for(15, 32, 4, 8, resident) == 8);
  CHECK(split_for(16, 32, 4, 8, resident) == 4);  // 16 x 8 CTAs would fit 152 SMs, but not as clusters
  CHECK(split_for(19, 32, 4, 8, resident) == 4);
  CHECK(split_for(8, 16, 4, 8, resident) == 4);
  CHECK(split_for(8, 15, 4, 8, resident) == 1);
  CHECK(split_for(18, 31, 8, 4, resident) == 1);
  CHECK(split_for(18, 32, 8, 4, resident) == 4);
  CHECK(split_for(37, 64, 8, 4, resident) == 2);
  CHECK(split_for(38, 64, 8, 4, resident) == 2);
  CHECK(split_for(77, 64, 8, 4, resident) == 1);
  // A device without clusters, or of which none could be asked.
  CHECK(split_for(1, 1024, 4, 8, [](int) { return 0; }) == 1);
  // Grouping: the counters fit, every warp of a cluster has work, and many keys
  // use every SM, whatever the groups.
  for (int groups = 1; groups <= 32768; groups += groups < 64 ? 1 : 61)
    for (int64_t n : {int64_t{0}, int64_t{1}, int64_t{31}, int64_t{33}, int64_t{4097}, int64_t{12288}, int64_t{12289},
                      int64_t{262144}, int64_t{262145}, int64_t{1} << 20, int64_t{1} << 24, int64_t{2147483647}}) {
      const GroupShape s = group_shape(n, groups, 152);
      const int rows = s.warps + (s.shared_totals ? 0 : 2);
      CHECK(s.warps >= 1 && s.warps <= 32 && (s.warps == 1 || !s.shared_totals));
      CHECK(s.smem_bytes <= kGroupSmemLimit && s.smem_bytes >= (rows * groups + 32) * 4);
      CHECK(s.one_cluster ? (s.ctas >= 1 && s.ctas <= 16 && (s.ctas & (s.ctas - 1)) == 0) : s.ctas >= 152);
      if (s.ctas > 1 && s.one_cluster) CHECK(n >= int64_t{s.ctas} * s.warps * 128);
      if (n > 262144) CHECK(s.ctas >= 152);
      CHECK(s.shared_totals == (groups > 17056));
    }
  CHECK(group_shape(12288, 17057, 152).ctas == 1);
  CHECK(group_shape(12289, 17057, 152).ctas == 304);
  CHECK(group_shape(1 << 20, 32768, 152).ctas == 152);
  CHECK(group_shape(131072, 256, 152).ctas == 16);
  if (failures == 0) printf("ok\n");
  return failures != 0;
}
