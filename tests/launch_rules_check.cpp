// CPU check of the launch rules of the expert-layer calls
// (cluster_distributed_shared_gb300/csrc/launch_rules.h).  Prints "ok" and
// exits 0 when every check holds.
#include <stdio.h>

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
  if (failures == 0) printf("ok\n");
  return failures != 0;
}
