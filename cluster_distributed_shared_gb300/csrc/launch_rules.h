// Rules by which the expert-layer calls choose how to launch.  Free of CUDA
// calls, so that the CPU tests can drive them.
#pragma once

#include <stdint.h>

namespace dsmh {

// CTAs of a cluster to split a product tile's depth over, where whole tiles
// leave SMs idle: as many, up to `most`, as leave each `stages` stages of depth
// or more, and none where four would have fewer than that: the join costs what
// some stages do, more for wide tiles.  And no more than let every tile's cluster
// be resident at once.  `resident(s)` is how many clusters of s CTAs are: fewer
// than their share of the SMs, since a cluster stays within a part of the chip
// (152 SMs: 76 of 2, 36 of 4, 15 of 8); a tile beyond waits for a whole tile's time.
// us, 8 tiles of 128 channels, whole / 2 / 4 / 8 CTAs a tile (64 depth a stage;
// tiles 16 rows wide for one row, 64 for 63 and for the weight gradient):
//   depth  512   one row  4.7 / 5.2 / 5.2 / 5.8    63 rows  5.1 / 6.7 / 7.6
//   depth 1024            6.2 / 6.0 / 5.7 / 6.2             6.7 / 7.5 / 8.1
//   depth 2048            9.6 / 8.0 / 6.9 / 7.2            10.2 / 10.5 / 9.6
//   depth 4096           15.0 / 10.7 / 8.3 / 7.9           16.0 / 14.6 / 11.9
//   256 x 256 weight gradient of 1024 rows 7.3 / 7.7 / 8.1, of 2048 10.4 / 9.3 / 8.8
// At the bound, one row, depth 2048, 4 / 8 CTAs: 15 tiles 7.2 / 7.9, 16 tiles
// 7.3 / 12.3, 19 tiles 7.5 / 12.5; 63 rows, depth 4096, 2 / 4 CTAs: 36 tiles
// 16.0 / 14.8, 37 tiles 16.0 / 22.0.
constexpr int split_stages(int cols) { return cols <= 16 ? 4 : 8; }

template <typename Resident>
int split_for(int64_t tiles, int64_t depth_blocks, int stages, int most, Resident resident) {
  int split = 1;
  while (split < most && depth_blocks >= stages * (split == 1 ? 4 : 2 * split) &&
         tiles <= resident(2 * split))
    split *= 2;
  return split;
}

// How a call groups n keys: one cluster of CTAs, or three launches over all SMs.
constexpr int kGroupSmemLimit = 200 * 1024;
constexpr int64_t kClusterKeys = int64_t{1} << 18, kOneWarpKeys = 12288;
struct GroupShape {
  int warps;           // of a CTA, each with a row of counters
  bool shared_totals;  // one warp, whose row is the CTA's totals and bases as well
  bool one_cluster;
  int ctas;
  int smem_bytes;
};
// Warps: as many counter rows as shared memory holds beside the totals and the
// bases, but no more than the keys fill with 32 each.  Where not even one row
// fits beside them (17,057 groups or more) one warp keeps all in one row.
// CTAs: one cluster, doubled while every warp still has 128 keys or more; with
// more keys than a cluster's 16 SMs (or the one warp) are good for, two an SM (one
// where the rows take its shared memory).  256 groups, one cluster / all SMs, us:
// 2^18 keys 17.1 / 17.7, 2^20 55 / 23, 2^24 770 / 175, 2^26 7009 / 1349 (bound by
// scattered 4-byte writes of the order).  17,057 groups, one warp / all SMs: 2^12
// keys 194 / 317, 2^14 367 / 317, 2^18 3815 / 328, 2^20 14857 / 365, and 2^24 keys
// 1278 (bound by each CTA's scan over the groups); 32,768 groups 313 / 476,
// 487 / 477, 3937 / 498, 14974 / 570, and 2432.
inline GroupShape group_shape(int64_t n, int groups, int sm_count) {
  GroupShape s = {};
  const int64_t fit = (kGroupSmemLimit / 4 - 32) / groups - 2;
  s.shared_totals = fit < 1;
  int64_t warps = (n + 31) / 32;
  if (warps > fit) warps = fit;
  s.warps = static_cast<int>(warps < 1 ? 1 : (warps > 32 ? 32 : warps));
  s.smem_bytes = ((s.warps + (s.shared_totals ? 0 : 2)) * groups + 32) * 4;
  s.one_cluster = n <= (s.shared_totals ? kOneWarpKeys : kClusterKeys);
  s.ctas = 1;
  if (!s.one_cluster)
    s.ctas = sm_count * (s.smem_bytes <= 100 * 1024 ? 2 : 1);
  else
    while (s.ctas < 16 && !s.shared_totals && n >= int64_t{2} * s.ctas * s.warps * 128) s.ctas *= 2;
  return s;
}

}  // namespace dsmh
