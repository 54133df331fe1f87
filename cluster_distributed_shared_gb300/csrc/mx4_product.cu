// Products of microscaled 4-bit rows and matrices grouped by key, on the
// block-scaled tcgen05 matrix instructions.
//
// D[rows, channels] = x W[g]^T: 128 rows high, kCols channels wide, so that a
// lane of the accumulators is a row of the output.  One persistent CTA per SM.
// Warp 0 copies the matrices' values by TMA (256 elements of depth a stage: 128
// bytes a row, swizzled), warp 1 issues the matrix instructions, the next eight
// write finished sums out, four copy the rows that the order names, 16 bytes a
// copy, and the last two bring both sides' scales.  (Four more copying warps left the
// writing ones 96 registers instead of 128: 177 us, not 161, with the quantisation
// before it, in the case below.)  Scales are kept row by row, as
// quantisation writes them; shared memory has them in the order that tensor memory
// wants: chunks of 128 rows by 4 scales, row r at 16 (r % 32) + 4 (r / 32).
//
// 4-bit operands are multiplied so fast that a tile is bound by what it takes in:
// 128 x 256 tiles take in three quarters of the bytes of 128 x 128 ones.  Their
// sums fill half of tensor memory, beside the scales, so there is no second
// accumulator; the first stage of a tile is multiplied by halves instead, each
// of which begins when the last tile's half is in its warps' registers.
//
// Measured, 16384 tokens x 8 of 64 experts of 1024 x 2048, groups of unequal size, rows
// named by the order: 142 us, 3.9 PFLOP/s, where the bytes alone would take 53
// (matrices and rows once, bf16 results once) and the arithmetic 71.  The tiles take
// in 1.7 GB from L2, 12 TB/s; without rows, scales and results the matrices' 1.1 GB
// and the arithmetic still took 120.
// 32 tokens x 8 of 128 experts: 26 us for 127 MB, 4.9 TB/s.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "divisor.h"
#include "dtypes.cuh"
#include "experts.h"
#include "product.cuh"

namespace dsmh {
namespace {

constexpr int kHigh = 128;        // rows of a tile
constexpr int kStageBytes = 128;  // of a row in a stage: 256 elements
constexpr int kCopyThreads = 128;
constexpr int kOutWarps = 8;      // four for either half of a tile's columns
constexpr int kFirstCopy = 2 + kOutWarps;  // behind TMA, matrix instructions and output
constexpr int kFirstScale = kFirstCopy + kCopyThreads / 32;
constexpr int kScaleThreads = 64;
constexpr int kThreads = kFirstScale * 32 + kScaleThreads;
constexpr int kStageOut = 2048;         // output staging of a warp
constexpr int kBarrierBytes = 320;
constexpr int kChunk = 512;             // scales of 128 rows by 128 elements

template <int kCols>
struct Ring {
  static constexpr int kA = kHigh * kStageBytes, kB = kCols * kStageBytes;
  static constexpr int kChunksB = (kCols + 127) / 128;  // of 128 elements' scales
  static constexpr int kStage = kA + kB + 2 * (1 + kChunksB) * kChunk;
  static constexpr int kMostStages = kCols == 256 ? 4 : (kCols == 128 ? 6 : 8);
  // Tensor memory: the sums of one tile in two halves, or of two tiles, then each
  // stage's scales of the rows, and of the channels.
  static constexpr int kBuffers = kCols == 256 ? 1 : 2, kHalves = kCols == 256 ? 2 : 1;
  static constexpr int kMine = kCols / 2;  // columns of an output warp
  static constexpr int kRowScales = kBuffers * kCols, kChannelScales = kRowScales + 8 * kMostStages;
  static constexpr uint32_t kColumns = 512;
  static_assert(kChannelScales + 8 * kChunksB * kMostStages <= 512, "tensor memory");
  static int smem_bytes(int groups, int stages) {
    return 1024 + stages * kStage + kOutWarps * kStageOut + kBarrierBytes + 2 * 4 * (groups + 2);
  }
  // As many stages as fit.
  static int stages(int groups) {
    int n = kMostStages;
    while (smem_bytes(groups, n) > kMostShared) --n;
    return n;
  }
};

struct Maps {
  CUtensorMap weights;
  CUtensorMap out;  // where rows are whole 16-byte vectors
};

struct Args {
  const int32_t* offsets;
  const int32_t* order;
  int64_t n;
  int x_rows, groups, outer, quads, stages;
  Divisor fan;
  const uint8_t* x_values;
  const uint8_t* x_scales;
  const uint8_t* w_scales;
  void* out;
  int out_dtype, wide_out, wide_scales;
  uint32_t* status;
  long long wait_cycles;
  int withhold;  // test hook: each CTA's last stage of values is not copied
};

struct Tile {
  int group;  // `groups`: the rows behind the last group
  int row0, end, chan0;
  int blocks;  // stages of depth
};

template <int kCols>
struct Schedule {
  const int32_t* begin;  // [groups + 2] first row of each group, in shared memory
  const int32_t* first;  // [groups + 2] first tile
  int groups, chan_tiles, blocks, group;
  __device__ __forceinline__ Schedule(const int32_t* b, const int32_t* f, const Args& a)
      : begin(b), first(f), groups(a.groups), chan_tiles((a.outer + kCols - 1) / kCols), blocks((a.quads + 1) / 2),
        group(0) {}
  __device__ __forceinline__ int tiles_of(int rows) const { return (rows + kHigh - 1) / kHigh * chan_tiles; }
  // Tile t; t only grows from call to call.  Many groups may be empty.
  __device__ __forceinline__ Tile at(int t) {
    if (t >= first[group + 1]) {
      int low = group + 1, high = groups;
      while (low < high) {
        const int mid = (low + high) >> 1;
        if (t >= first[mid + 1]) low = mid + 1;
        else high = mid;
      }
      group = low;
    }
    const int i = t - first[group], high = (begin[group + 1] - begin[group] + kHigh - 1) / kHigh;
    Tile r;
    r.group = group;
    r.row0 = begin[group] + i % high * kHigh;
    r.end = begin[group + 1];
    r.chan0 = i / high * kCols;
    r.blocks = group < groups ? blocks : 0;
    return r;
  }
};

// The first of all tiles that is a CTA's.
__device__ __forceinline__ int share(int all, int cta) {
  return static_cast<int>(static_cast<int64_t>(all) * cta / static_cast<int>(gridDim.x));
}

// Descriptor of a chunk of scales: not swizzled, groups of 8 rows of 16 bytes.
__device__ __forceinline__ uint64_t scale_descriptor(uint32_t addr) {
  return (uint64_t{1} << 46) | (uint64_t{128 >> 4} << 32) | ((addr & 0x3ffffu) >> 4);
}

// kLine bytes of each of a warp's 32 rows, in lane l row l, as channels [chan, limit)
// to the output through its staging memory: 16-byte pieces of a row, exchanged so
// that neighbouring rows meet other banks, as a map with a swizzle of 64 bytes has
// them.  Where all rows are there, and whole 64 bytes, one TMA store takes them, and
// costs the warp a quarter of the instructions.  (Rows written sector by sector
// from the lanes that hold them took twice as long as this path without TMA.)
// Other rows are written value by value: 131072 rows of 1028 bf16 channels in 275 us,
// of 1032 in 183.  (By words, which begin elsewhere in each row: 406, not the 333 of
// that step.)
template <typename O, int kLine>
__device__ __forceinline__ void store_lines(const Args& a, const CUtensorMap* out_map, int row0, int end, int chan,
                                            int limit, const uint32_t (&r)[kLine / 4], uint32_t staging) {
  const int lane = threadIdx.x & 31, rows = min(32, end - row0);
  constexpr int V = 16 / sizeof(O), kPieces = kLine / 16;
  const auto piece_at = [&](int row, int q) {
    return staging + row * kLine + ((q ^ (row * kPieces / 8 & (kPieces - 1))) << 4);
  };
  if (lane == 0) store_wait_read();
  __syncwarp();
#pragma unroll
  for (int q = 0; q < kPieces; ++q)
    st_shared_16(piece_at(lane, q), make_uint4(r[4 * q], r[4 * q + 1], r[4 * q + 2], r[4 * q + 3]));
  if (kLine == 64 && a.wide_out && rows == 32) {
    fence_async_shared();
    __syncwarp();
    if (lane == 0) tma_store_2d(out_map, staging, chan, row0);
    return;
  }
  __syncwarp();
  O* out = static_cast<O*>(a.out) + static_cast<int64_t>(row0) * a.outer + chan;
  if (a.wide_out) {
    const int q = lane % kPieces;
    uint4* to = reinterpret_cast<uint4*>(out + static_cast<int64_t>(lane / kPieces) * a.outer + q * V);
    const int64_t step = static_cast<int64_t>(32 / kPieces) * a.outer / V;
    if (chan + q * V < limit) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i, to += step) {
        const int row = i * (32 / kPieces) + lane / kPieces;
        if (row < rows) *to = ld_shared_16(piece_at(row, q));
      }
    }
  } else {
    constexpr int kEach = kLine / static_cast<int>(sizeof(O));  // values of a line
    const int j = lane % kEach;
    if (chan + j < limit) {
#pragma unroll 1
      for (int row = lane / kEach; row < rows; row += 32 / kEach)
        out[static_cast<int64_t>(row) * a.outer + j] = ld_shared_value<O>(piece_at(row, j / V) + j % V * sizeof(O));
    }
  }
  __syncwarp();
}

// Zeros in the rows behind the last group.
template <int kCols, typename O>
__device__ __forceinline__ void store_zeros(const Args& a, int row0, int end, int chan) {
  const int lane = threadIdx.x & 31, rows = min(32, end - row0), cols = min(kCols, a.outer - chan);
  O* out = static_cast<O*>(a.out) + static_cast<int64_t>(row0) * a.outer + chan;
  constexpr int V = 16 / sizeof(O);
  for (int row = 0; row < rows; ++row, out += a.outer) {
    if (a.wide_out) {
      for (int c = lane * V; c < cols; c += 32 * V) *reinterpret_cast<uint4*>(out + c) = make_uint4(0, 0, 0, 0);
    } else {
      for (int c = lane; c < cols; c += 32) out[c] = O(0);
    }
  }
}

// A pair of values (bits of floats) rounded to bf16 or f16, of which the bits `kept`
// remain, here and now, in one place for both: left to the compiler, roundings move behind the next loads, whose
// values then do not fit registers.
__device__ __forceinline__ uint32_t pair_now(uint32_t low, uint32_t high, bool bf16, uint32_t kept) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %3, 0;\n\t@p cvt.rn.bf16x2.f32 %0, %1, %2;\n\t"
      "@!p cvt.rn.f16x2.f32 %0, %1, %2;\n\tand.b32 %0, %0, %4;\n\t}"
      : "=r"(r)
      : "f"(__uint_as_float(high)), "f"(__uint_as_float(low)), "r"(static_cast<uint32_t>(bf16)), "r"(kept));
  return r;
}

// The order's entry of a place, kBehind behind the tile's end, and the row of x
// that it names, -1 for none.
constexpr int kBehind = -2;
__device__ __forceinline__ int place_at(const Args& a, int p, int end) {
  return p < end ? (a.order ? max(a.order[p], -1) : p) : kBehind;
}
__device__ __forceinline__ int row_named(const Args& a, int o) {
  if (o < 0) return o;
  const int row = a.order ? a.fan.quotient(o) : o;
  return row < a.x_rows ? row : -1;
}

// A warp's 32 rows by kMine columns from tensor memory to the output, up to 64 bytes
// of a row at a time; free() is called when they have left tensor memory.  16-bit
// values are first all brought to registers, as pairs, so that this is soon.  A row
// without a source was multiplied as zeros, which a matrix's NaN makes NaN.
template <int kMine, typename O, typename Free>
__device__ __forceinline__ void store_tile(const Args& a, const CUtensorMap* out_map, const Tile& t, int row0,
                                           int chan, uint32_t tmem, uint32_t staging, bool none, Free free) {
  constexpr int kLine = kMine * static_cast<int>(sizeof(O)) < 64 ? kMine * static_cast<int>(sizeof(O)) : 64;
  constexpr int kN = kLine / static_cast<int>(sizeof(O)), kWords = kLine / 4;
  const int limit = min(a.outer, chan + kMine);
  const bool bf16 = a.out_dtype == DSMEM_BF16;
  const uint32_t kept = none ? 0u : ~0u;
  if constexpr (sizeof(O) == 2) {
    uint32_t line[kMine / kN][kWords];
    if (row0 < t.end) {
#pragma unroll
      for (int c = 0; c < kMine; c += 16) {
        uint32_t r[16];
        tmem_load16(tmem + c, r);
        tmem_wait_load();
#pragma unroll
        for (int l = 0; l < 8; ++l)
          line[c / kN][c % kN / 2 + l] = pair_now(r[2 * l], r[2 * l + 1], bf16, kept);
      }
    }
    free();
#pragma unroll
    for (int c = 0; c < kMine; c += kN)
      if (row0 < t.end && chan + c < limit)
        store_lines<O, kLine>(a, out_map, row0, t.end, chan + c, limit, line[c / kN], staging);
  } else {
#pragma unroll 1
    for (int c = 0; c < kMine && row0 < t.end && chan + c < limit; c += kN) {
      uint32_t r[kN];
      tmem_load16(tmem + c, r);
      tmem_wait_load();
#pragma unroll
      for (int l = 0; l < kN; ++l) r[l] &= kept;
      store_lines<O, kLine>(a, out_map, row0, t.end, chan + c, limit, r, staging);
    }
    free();
  }
}

// The copying warps.  A thread copies one of the eight pieces of every 16th row.
// Rows at and behind the tile's end are left as they are: what they hold reaches
// no other row.  Each thread's copies of a stage arrive on `landed` by themselves.
template <int kCols>
__device__ __forceinline__ void copy_rows(const Args& a, Schedule<kCols>& schedule, int i, int total, uint32_t base,
                                          uint32_t landed, uint32_t empty, uint32_t gave_up) {
  using R = Ring<kCols>;
  constexpr int kRows = kHigh * 8 / kCopyThreads, kLines = kCopyThreads / 8;
  const int tid = threadIdx.x - kFirstCopy * 32;
  const int64_t pitch = int64_t{64} * a.quads;
  // A tile's entries of the order are asked for while the tile before is copied.
  int ahead[kRows];
  const auto ask = [&](const Tile& t) {
#pragma unroll
    for (int r = 0; r < kRows; ++r) ahead[r] = place_at(a, t.row0 + r * kLines + tid / 8, t.end);
  };
  int stage = 0;
  uint32_t phase = 0;
  bool ok = true;
  Tile next;
  if (i < total) {
    next = schedule.at(i);
    ask(next);
  }
  while (i < total && ok) {
    const Tile t = next;
    int row[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) row[r] = row_named(a, ahead[r]);
    if (++i < total) {
      next = schedule.at(i);
      ask(next);
    }
    for (int k = 0; k < t.blocks; ++k) {
      ok = wait_for(empty + 8 * stage, phase ^ 1, gave_up, a.wait_cycles, a.status);
      ok = __all_sync(kFull, ok);
      if (!ok) break;
      const uint32_t sa = base + stage * R::kStage;
      const int c = tid & 7, at = k * kStageBytes + c * 16;
      const bool there = at < pitch;
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const int line = r * kLines + tid / 8;
        const bool read = row[r] >= 0 && there;
        if (row[r] != kBehind)
          copy16(sa + line * 128 + ((c ^ (line & 7)) << 4), a.x_values + (read ? row[r] * pitch + at : 0),
                 read ? 16 : 0);
      }
      copy_arrive(landed + 8 * stage);
      if (++stage == a.stages) {
        stage = 0;
        phase ^= 1;
      }
    }
  }
  copy_wait_all();
}

// The scales' warps.  A thread brings those of every kScaleThreads-th row and
// channel, two stages' at a time, which are asked for four stages ahead.
template <int kCols>
__device__ __forceinline__ void bring_scales(const Args& a, Schedule<kCols>& schedule, int i, int total, uint32_t base,
                                             uint32_t landed, uint32_t empty, uint32_t gave_up) {
  using R = Ring<kCols>;
  constexpr int kRows = kHigh / kScaleThreads, kLines = kRows + (kCols + kScaleThreads - 1) / kScaleThreads;
  const int tid = threadIdx.x - kFirstScale * 32, blocks = schedule.blocks;
  const int64_t pitch = int64_t{4} * a.quads;
  // What comes next to ask for: a tile's lines (null for none) and the stage; the
  // order's entry of the tile behind.
  const uint8_t* line[kLines];
  int tile = i, stage_ahead = 0, entry[kRows], chan0 = 0, group = 0;
  const auto look = [&] {
    if (tile >= total) return;
    const Tile t = schedule.at(tile);
#pragma unroll
    for (int r = 0; r < kRows; ++r) entry[r] = place_at(a, t.row0 + r * kScaleThreads + tid, t.end);
    chan0 = t.chan0, group = t.group;
  };
  const auto enter = [&] {
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int row = row_named(a, entry[r]);
      line[r] = row >= 0 ? a.x_scales + row * pitch : nullptr;
    }
#pragma unroll
    for (int l = kRows; l < kLines; ++l) {
      const int c = (l - kRows) * kScaleThreads + tid;
      line[l] = chan0 + c < a.outer && c < kCols
                    ? a.w_scales + (static_cast<int64_t>(group) * a.outer + chan0 + c) * pitch
                    : nullptr;
    }
    ++tile;
    look();
  };
  // Four quads of each line; zeros behind a line's end, and for none.
  struct Pair {
    uint4 of[kLines];
  };
  int64_t left = static_cast<int64_t>(total - i) * ((blocks + 1) / 2);  // pairs to ask for
  const auto ask = [&](Pair& p) {
    if (--left < 0) return;
    if (stage_ahead >= blocks) {
      stage_ahead = 0;
      enter();
    }
    const int first = 2 * stage_ahead;
    stage_ahead += 2;
#pragma unroll
    for (int l = 0; l < kLines; ++l) {
      p.of[l] = make_uint4(0, 0, 0, 0);
      if (!line[l]) continue;
      const uint32_t* q = reinterpret_cast<const uint32_t*>(line[l]) + first;
      if (a.wide_scales) {
        p.of[l] = __ldg(reinterpret_cast<const uint4*>(q));
      } else {
        p.of[l].x = __ldg(q);
        if (first + 1 < a.quads) p.of[l].y = __ldg(q + 1);
        if (first + 2 < a.quads) p.of[l].z = __ldg(q + 2);
        if (first + 3 < a.quads) p.of[l].w = __ldg(q + 3);
      }
    }
  };
  uint32_t stage = 0, phase = 0;
  int k = 0;
  bool ok = true;
  const auto put = [&](const Pair& p) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if (half == 1 && k == 0) break;  // a tile's last stage had no second
      ok = ok && wait_for(empty + 8 * stage, phase ^ 1, gave_up, a.wait_cycles, a.status);
      ok = __all_sync(kFull, ok);
      if (!ok) return;
      const uint32_t to = base + stage * R::kStage + R::kA + R::kB;
#pragma unroll
      for (int l = 0; l < kLines; ++l) {
        const bool row = l < kRows;
        const int c = (row ? l : l - kRows) * kScaleThreads + tid;
        if (!row && kCols % kScaleThreads != 0 && c >= kCols) break;
        const uint32_t at = to + (c & 31) * 16 + (c >> 5 & 3) * 4 + (row ? 0 : 2 * kChunk + (c >> 7) * kChunk);
        st_shared_u32(at, half ? p.of[l].z : p.of[l].x);
        st_shared_u32(at + (row ? 1 : R::kChunksB) * kChunk, half ? p.of[l].w : p.of[l].y);
      }
      __syncwarp();
      if (tid % 32 == 0) mbar_arrive_local(landed + 8 * stage);
      if (++stage == static_cast<uint32_t>(a.stages)) {
        stage = 0;
        phase ^= 1;
      }
      if (++k == blocks) k = 0;
    }
  };
  int64_t pairs = left;
  Pair first, second;
  if (pairs > 0) {
    look();
    enter();
  }
  ask(first);
  ask(second);
  while (pairs > 0 && ok) {
    put(first);
    if (--pairs == 0 || !ok) break;
    ask(first);
    put(second);
    --pairs;
    ask(second);
  }
}

template <int kCols>
__global__ void __launch_bounds__(kThreads, 1)
    mx4_product_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Args a) {
  using R = Ring<kCols>;
  constexpr int kStage = R::kStage;
  const int kStages = a.stages;
  extern __shared__ uint8_t raw[];
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  uint8_t* base_ptr = raw + (base - smem_u32(raw));
  const uint32_t out_staging = base + kStages * kStage;
  const uint32_t bars = out_staging + kOutWarps * kStageOut;
  const uint32_t full = bars, empty = full + 8 * R::kMostStages, landed = empty + 8 * R::kMostStages;
  const uint32_t acc_full = landed + 8 * R::kMostStages, acc_empty = acc_full + 16, drained = acc_empty + 16;
  const uint32_t tmem_at = drained + 8, gave_up = tmem_at + 4;
  static_assert(8 * (3 * R::kMostStages + 5) + 8 <= kBarrierBytes, "barriers");
  int32_t* begin = reinterpret_cast<int32_t*>(base_ptr + (bars - base) + kBarrierBytes);
  int32_t* first = begin + a.groups + 2;

  const int warp = __shfl_sync(kFull, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  Schedule<kCols> schedule(begin, first, a);
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(landed + 8 * s, kCopyThreads + kScaleThreads / 32);
      mbar_init(empty + 8 * s, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full + 8 * i, 1);
      mbar_init(acc_empty + 8 * i, kOutWarps / R::kHalves);
    }
    mbar_init(drained, 1);
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(gave_up), "r"(0u) : "memory");
    fence_mbar_init();
    prefetch_map(&maps.weights);
    if (a.wide_out) prefetch_map(&maps.out);
  }
  lay_groups<kThreads>(a.offsets, a.n, a.groups, a.groups + 1, begin, first,
                       [&](int rows) { return schedule.tiles_of(rows); },
                       [&] { if (warp == 1) tmem_alloc<false>(tmem_at, R::kColumns); });
  tcgen_fence_before();
  __syncthreads();
  tcgen_fence_after();
  uint32_t tmem;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(tmem_at));
  // A CTA's tiles are neighbours, row tiles of the same channels first: CTAs that
  // took every gridDim-th tile met in the same matrices, and waited together for
  // memory where one began.
  const int all = first[a.groups + 1], of_groups = first[a.groups];  // all, and those of real groups
  const int mine = share(all, blockIdx.x), total = share(all, blockIdx.x + 1);
  const int of_mine = min(of_groups, total);

  if (warp == 0) {
    uint32_t stage = 0, phase = 0, issued = 0;
    bool ok = true;
    for (int i = mine; i < of_mine && ok; ++i) {
      const Tile t = schedule.at(i);
      for (int k = 0; k < t.blocks; ++k) {
        ok = __all_sync(kFull, wait_for(empty + 8 * stage, phase ^ 1, gave_up, a.wait_cycles, a.status));
        if (!ok || (a.withhold && i + 1 == of_mine && k + 1 == t.blocks)) break;
        if (elect_one()) {
          mbar_expect_tx(full + 8 * stage, R::kB);
          tma_load_3d<false>(base + stage * kStage + R::kA, &maps.weights, k * kStageBytes, t.chan0, t.group,
                             full + 8 * stage);
        }
        __syncwarp();
        ++issued;
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    // After a wait that gave up: let this CTA's copies land before its shared
    // memory goes.  Copy j completes phase j / kStages of its stage.
    if (flag_set(gave_up)) {
      for (uint32_t j = issued > kStages ? issued - kStages : 0; j < issued; ++j) {
        const long long deadline = clock64() + kDefaultWaitCycles;
        while (!mbar_try_wait(full + 8 * (j % kStages), (j / kStages) & 1) && clock64() < deadline) {
        }
      }
    }
    __syncwarp();
  } else if (warp >= kFirstScale) {
    bring_scales<kCols>(a, schedule, mine, of_mine, base, landed, empty, gave_up);
  } else if (warp >= kFirstCopy) {
    copy_rows<kCols>(a, schedule, mine, of_mine, base, landed, empty, gave_up);
  } else if (warp == 1) {
    // A and B e2m1, K-major, scales e8m0.  Bits 4 and 29 choose the first or the
    // third of a row's four scales, of which an instruction takes two.
    constexpr int kHalf = kCols / R::kHalves;
    constexpr uint32_t kDesc = (1u << 7) | (1u << 10) | (1u << 23) | (uint32_t{kHigh >> 7} << 27);
    constexpr uint32_t kWhole = kDesc | (uint32_t{kCols >> 3} << 17), kPart = kDesc | (uint32_t{kHalf >> 3} << 17);
    constexpr uint32_t kSecond = (2u << 4) | (2u << 29);
    uint32_t stage = 0, phase = 0, done = 0;
    bool ok = true;
    const auto await = [&](uint32_t bar, uint32_t parity) {
      ok = __all_sync(kFull, wait_for(bar, parity, gave_up, a.wait_cycles, a.status));
      tcgen_fence_after();
      return ok;
    };
    for (int i = mine; i < of_mine && ok; ++i) {
      // Sums: a tile's own place of two, or the halves of the only one.
      const uint32_t place = R::kBuffers == 2 ? done & 1 : 0, d = tmem + place * kCols;
      const uint32_t turn = R::kBuffers == 2 ? done >> 1 & 1 : done & 1;
      if (!await(acc_empty + 8 * place, turn ^ 1)) break;
      for (int k = 0; k < schedule.blocks; ++k) {
        // Rows and scales come by plain copies, which this warp passes on to the
        // matrix instructions.  (A fence of the scales' warps waited for their loads
        // ahead too: 1400 cycles a stage.)
        if (!await(landed + 8 * stage, phase)) break;
        fence_async_shared();
        if (!await(full + 8 * stage, phase)) break;
        const uint32_t sa = base + stage * kStage;
        const uint64_t da = descriptor<false>(sa), db = descriptor<false>(sa + R::kA);
        const uint64_t ds = scale_descriptor(sa + R::kA + R::kB);
        // Each stage has columns of its own: the stage is handed back only when
        // the instructions that read them have completed.
        const uint32_t sfa = tmem + R::kRowScales + stage * 8;
        const uint32_t sfb = tmem + R::kChannelScales + stage * (8 * R::kChunksB);
        const auto multiply = [&](int half, uint32_t desc) {
#pragma unroll
          for (int s = 0; s < 4; ++s)
            mma_mx4(d + half * kHalf, da + 2 * s, db + 2 * s + half * (kHalf * kStageBytes >> 4),
                    s & 1 ? desc | kSecond : desc, sfa + 4 * (s >> 1), sfb + 4 * R::kChunksB * (s >> 1) + 4 * half,
                    k > 0 || s > 0);
        };
        if (elect_one()) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            copy_scales(sfa + 4 * q, ds + q * (kChunk >> 4));
#pragma unroll
            for (int c = 0; c < R::kChunksB; ++c)
              copy_scales(sfb + 4 * (R::kChunksB * q + c), ds + (2 + R::kChunksB * q + c) * (kChunk >> 4));
          }
          if (R::kHalves == 1 || k > 0) multiply(0, kWhole);
          else multiply(0, kPart);
        }
        __syncwarp();
        if (R::kHalves == 2 && k == 0) {
          if (!await(acc_empty + 8, turn ^ 1)) break;
          if (elect_one()) multiply(1, kPart);
          __syncwarp();
        }
        const bool last = k + 1 == schedule.blocks;
        if (elect_one()) {
          mma_commit<false>(empty + 8 * stage);
          if (last) mma_commit<false>(acc_full + 8 * place);
        }
        __syncwarp();
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
      ++done;
    }
    if (flag_set(gave_up)) {  // matrix instructions end before tensor memory is given back
      if (elect_one()) mma_commit<false>(drained);
      __syncwarp();
      const long long deadline = clock64() + kDefaultWaitCycles;
      while (!mbar_try_wait(drained, 0) && clock64() < deadline) {
      }
    }
    __syncwarp();
  } else {
    // Output: warp w may read lanes 32 (w % 4) .. of tensor memory.
    const int quadrant = warp & 3, half = (warp - 2) >> 2;
    const uint32_t staging = out_staging + (warp - 2) * kStageOut;
    uint32_t done = 0;
    for (int i = mine; i < total; ++i) {
      const Tile t = schedule.at(i);
      const int row0 = t.row0 + quadrant * 32, chan = t.chan0 + half * R::kMine;
      if (t.blocks == 0) {
        if (a.out_dtype == DSMEM_F32) store_zeros<R::kMine, float>(a, row0, t.end, chan);
        else store_zeros<R::kMine, uint16_t>(a, row0, t.end, chan);
        continue;
      }
      const uint32_t place = R::kBuffers == 2 ? done & 1 : 0;
      const uint32_t turn = R::kBuffers == 2 ? done >> 1 & 1 : done & 1;
      const bool none = row_named(a, place_at(a, row0 + lane, t.end)) == -1;
      // A long contraction may take longer than one bounded wait of a copy.
      const bool ok = wait_for(acc_full + 8 * place, turn, gave_up, a.wait_cycles + 4096ll * t.blocks, a.status);
      if (!__all_sync(kFull, ok)) break;
      tcgen_fence_after();
      const uint32_t d = tmem + place * kCols + half * R::kMine + (static_cast<uint32_t>(quadrant * 32) << 16);
      const auto free = [&] {
        tcgen_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_local(acc_empty + 8 * (R::kHalves == 2 ? half : place));
      };
      if (a.out_dtype == DSMEM_F32) store_tile<R::kMine, float>(a, &maps.out, t, row0, chan, d, staging, none, free);
      else store_tile<R::kMine, uint16_t>(a, &maps.out, t, row0, chan, d, staging, none, free);
      ++done;
    }
    if (lane == 0) store_wait();
    __syncwarp();
  }
  tcgen_fence_before();
  __syncthreads();
  tcgen_fence_after();
  if (warp == 1) tmem_dealloc<false>(tmem, R::kColumns);
}

// The matrices' values as bytes [groups, outer, pitch] in boxes of kCols rows by a
// stage's 128 bytes.
int make_map(CUtensorMap* map, const Mx4ProductArgs& p, int cols) {
  const EncodeFn encode = encoder();
  if (!encode) return fail_with(DSMEM_HIST_EUNSUPPORTED, "the driver has no tensor maps");
  const cuuint64_t pitch = cuuint64_t{64} * p.quads;
  const cuuint64_t dims[3] = {pitch, static_cast<cuuint64_t>(p.outer), static_cast<cuuint64_t>(p.groups)};
  const cuuint64_t strides[2] = {pitch, pitch * p.outer};
  const cuuint32_t box[3] = {kStageBytes, static_cast<cuuint32_t>(cols), 1}, unit[3] = {1, 1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(p.w_values), dims, strides,
                            box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail_with(DSMEM_HIST_ECUDA, "cuTensorMapEncodeTiled: error %d (4-bit matrices, %d x %d x %d)",
                     static_cast<int>(r), p.groups, p.outer, p.quads * 128);
  return DSMEM_HIST_OK;
}

// The output in boxes of 32 rows by 64 bytes.
int make_out_map(CUtensorMap* map, const Mx4ProductArgs& p) {
  const int size = dtype_size(p.out_dtype);
  const CUtensorMapDataType type = p.out_dtype == DSMEM_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : p.out_dtype == DSMEM_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                              : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(p.outer), static_cast<cuuint64_t>(p.n)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(p.outer) * size};
  const cuuint32_t box[2] = {64u / size, 32}, unit[2] = {1, 1};
  const CUresult r = encoder()(map, type, 2, p.out, dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
                               CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail_with(DSMEM_HIST_ECUDA, "cuTensorMapEncodeTiled: error %d (4-bit product's output, %lld x %d)",
                     static_cast<int>(r), static_cast<long long>(p.n), p.outer);
  return DSMEM_HIST_OK;
}

// Upper bound of a product's tiles: the group sizes are not known here.
int64_t tile_bound(const Mx4ProductArgs& p, int cols) {
  return (p.n / kHigh + std::min<int64_t>(p.groups + 1, p.n)) * ((p.outer + cols - 1) / cols);
}

template <int kCols>
int launch(const Mx4ProductArgs& p, const CallContext& ctx, cudaStream_t stream) {
  static SmemLimit limit;
  Args a{};
  a.offsets = p.offsets, a.order = p.order, a.n = p.n;
  a.x_rows = static_cast<int>(p.x_rows), a.groups = p.groups, a.outer = p.outer, a.quads = p.quads;
  a.fan = Divisor(static_cast<uint32_t>(p.fan));
  a.x_values = p.x_values, a.x_scales = p.x_scales, a.w_scales = p.w_scales;
  a.out = p.out, a.out_dtype = p.out_dtype;
  a.wide_out = reinterpret_cast<uintptr_t>(p.out) % 16 == 0 &&
               static_cast<int64_t>(p.outer) * dtype_size(p.out_dtype) % 16 == 0;
  // 16 bytes of scales at a time, where rows begin so (by words 16384 tokens take 190
  // us, not 161).
  a.wide_scales = p.quads % 4 == 0 && reinterpret_cast<uintptr_t>(p.x_scales) % 16 == 0 &&
                  reinterpret_cast<uintptr_t>(p.w_scales) % 16 == 0;
  a.status = ctx.status;
  a.wait_cycles = call_wait_cycles();
  a.withhold = call_withholds();
  Maps maps;
  int rc = make_map(&maps.weights, p, kCols);
  if (!rc && a.wide_out) rc = make_out_map(&maps.out, p);
  if (rc) return rc;
  const int64_t tiles = tile_bound(p, kCols);
  if (tiles > INT32_MAX - 1024)  // tile counters step past the last tile
    return fail_with(DSMEM_HIST_EINVAL, "4-bit grouped product: more than 2^31 output tiles");
  a.stages = Ring<kCols>::stages(p.groups);
  const int smem = Ring<kCols>::smem_bytes(p.groups, a.stages);
  const auto kernel = mx4_product_kernel<kCols>;
  cudaError_t e = limit.need(reinterpret_cast<const void*>(kernel), ctx.device, smem);
  if (e != cudaSuccess) return fail_with_cuda(e, "cudaFuncSetAttribute");
  kernel<<<static_cast<unsigned>(std::min<int64_t>(tiles, ctx.sm_count)), kThreads, smem, stream>>>(maps, a);
  e = cudaGetLastError();
  return e == cudaSuccess ? DSMEM_HIST_OK : fail_with_cuda(e, "4-bit grouped product launch");
}

}  // namespace

// The narrowest tiles of which no SM gets a second one, for a tile's time is that of
// its share of the matrices: one row of 64 experts of 1536 x 2048 takes 7.4 us with 32
// channels, 8.0 with 128 and 9.4 with 256; eight rows (384 tiles of 32, 96 of 128)
// 13.3, 9.1 and 10.1.  Otherwise the widest, which take in the least: 16 rows (192
// tiles of 128) 15.9, 12.1 and 10.8; 16384 rows 53.1 with 128 and 45.9 with 256.
int run_mx4_product(const Mx4ProductArgs& p, const CallContext& ctx, cudaStream_t stream) {
  if (tile_bound(p, 32) <= ctx.sm_count) return launch<32>(p, ctx, stream);
  if (tile_bound(p, 128) <= ctx.sm_count) return launch<128>(p, ctx, stream);
  return launch<256>(p, ctx, stream);
}

cudaError_t read_and_clear_mx4_status(uint32_t* out) { return take_product_status(out); }

}  // namespace dsmh
