// Rules by which the expert-layer calls choose how to launch.  Free of CUDA
// calls, so that the CPU tests can drive them.
#pragma once

#include <stdint.h>

namespace dsmh {

// CTAs of a cluster to split a product tile's depth over, where whole tiles
// leave SMs idle: as many, up to `most`, as leave each CTA two stages of depth
// or more, and no more than let every tile's cluster be resident at once.
// `resident(s)` is how many clusters of s CTAs are.  That is fewer than their
// share of the SMs, since a cluster stays within a part of the chip (152 SMs: 76
// of 2, 36 of 4, 15 of 8), and a tile beyond it waits for a whole tile's time.
// Split over / whole, us: one row of 8 tiles of 128 channels, depth 1024, 4 CTAs
// 5.6 / 6.3, depth 4096, 8 CTAs 7.9 / 15.0; 63 rows of 18 such tiles, depth 4096,
// 4 CTAs 12.8 / 16.3.
// At the bound, one row, depth 2048, 4 / 8 CTAs: 15 tiles 7.2 / 7.9, 16 tiles
// 7.3 / 12.3, 19 tiles 7.5 / 12.5; 63 rows, depth 4096, 2 / 4 CTAs: 36 tiles
// 16.0 / 14.8, 37 tiles 16.0 / 22.0.
template <typename Resident>
int split_for(int64_t tiles, int64_t depth_blocks, int most, Resident resident) {
  int split = 1;
  while (split < most && depth_blocks >= split * 4 && tiles <= resident(split * 2)) split *= 2;
  return split;
}

}  // namespace dsmh
