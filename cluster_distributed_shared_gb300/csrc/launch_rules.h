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

}  // namespace dsmh
