// Products grouped by key on the tcgen05 tensor cores.
//
// All three products are D = A B with the weights' side as A, 128 channels
// high, and the rows' side as B, kCols columns wide, so that the width of a
// tile follows how many rows a group has while the weights keep full tiles:
//   forward       D[outer, rows]  = W[g] x^T        depth inner; both operands K-major
//   input grad    D[inner, rows]  = W[g]^T x^T      depth outer; A is MN-major
//   weight grad   D[outer, inner] = dy^T x          depth: the group's rows; both MN-major
// One persistent CTA per SM; warp 0 copies operand tiles of 64 depth
// (128 bytes, swizzled) into a ring of stages by TMA, warp 1 issues the matrix
// instructions into one of two accumulators in tensor memory, and warps 2..5
// write the other one out.  Rows named by an order are fetched by the warps
// behind them with 16-byte asynchronous copies straight into the swizzled
// layout, so no reordered copy of x exists anywhere.  (Four-row TMA gathers
// took about 70 cycles each, 4.5 times the time of the matrix instructions
// they feed.)  The same warps fill the ragged end of a group's contraction
// with zeros.
//
// Large products are bound by the tensor cores, and over long runs by the
// card's power: 131072 rows in 64 equal groups, 2048 x 1024, bf16, take 318 us
// (forward, gathered rows), 309 (input gradient) and 329 (weight gradient,
// gathered rows) or 1.67 to 1.78 PFLOP/s, where one library product of that
// size takes 288.  Few rows are bound by reading the weights: 32 tokens over
// 128 experts (469 MB) 73 to 76 us, 92 to 97% of the copy rate.
//
// The group sizes are on the device only: every CTA lays the groups' tiles
// end to end from the offsets and takes every gridDim-th.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "bounded_wait.h"
#include "dtypes.cuh"
#include "experts.h"
#include "launch_rules.h"
#include "ptx.cuh"
#include "tcgen.cuh"

namespace dsmh {
namespace {

using namespace ptx;

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kChannels = 128;  // channels of a tile in one CTA
constexpr int kDepth = 64;      // depth of a stage: 128 bytes of 16-bit elements
constexpr int kGatherThreads = 256;
constexpr int kShifts = 2;                        // groups of gathering warps that take stages in turn
constexpr int kShift = kGatherThreads / kShifts;  // threads of one
constexpr int kRelayWarp = 6 + kGatherThreads / 32;
// TMA, matrix instructions, 4 warps of output, gathering, relay.
constexpr int kThreads = (kRelayWarp + 1) * 32;
constexpr int kStageOut = 4096;  // output staging of a warp: 32 x 32 values of 4 bytes, or 32 x 64 of 2
constexpr int kABytes = kChannels * kDepth * 2;

constexpr int kBarrierBytes = 320;
constexpr int kMostSorted = 512;  // groups

// How CTAs work on a tile.
//   kSolo   each on its own.
//   kPair   two of a cluster on one 256 channels high: each holds 128 channels
//           of A and half of the columns of B, and one matrix instruction
//           reads both.  That halves the bytes of B a CTA takes in.
//   kSplit  a cluster of up to kMaxSplit on one tile, each on a part of its
//           depth; the first CTA adds the others' sums, which they write into
//           its shared memory, in the order of their ranks.
enum Team { kSolo, kPair, kSplit };

template <int kCols, int kTeam>
struct Ring {
  static constexpr int kMine = kTeam == kPair ? kCols / 2 : kCols;  // columns this CTA brings in
  static constexpr int kStage = kABytes + kMine * kDepth * 2;
  static constexpr int kHeight = kTeam == kPair ? 2 * kChannels : kChannels;  // channels of a tile
  static constexpr int kMaxSplit = kTeam != kSplit ? 1 : (kCols == 16 ? 8 : 4);
  static constexpr int kJoin = kChannels * kCols * 4;  // one CTA's sums
  // As many stages as fit beside the sums and the tables (227 KB in all).
  static constexpr int kStages = kTeam == kSplit ? (kCols == 16 ? 8 : 4)
                                                 : (kMine == 128 ? 6 : (kMine == 64 ? 8 : 10));
  static int smem_bytes(int groups, int split) {
    return 1024 + kStages * kStage + (split - 1) * kJoin + 4 * kStageOut + kBarrierBytes +
           2 * 4 * (groups + 2);
  }
};

struct Maps {
  CUtensorMap a;  // weights (3-D), or dy
  CUtensorMap b;  // x
};

// Division of 31-bit values by a fixed divisor: with l = ceil(log2 d) and
// m = floor(2^32 (2^l - d) / d) + 1, the quotient is (mulhi(m, v) + v) >> l.
struct Divisor {
  uint32_t m, l;
  Divisor(uint32_t d = 1) : m(0), l(0) {
    while ((uint64_t{1} << l) < d) ++l;
    m = static_cast<uint32_t>((uint64_t{1} << 32) * ((uint64_t{1} << l) - d) / d + 1);
  }
  __device__ __forceinline__ int quotient(int v) const {
    return static_cast<int>((__umulhi(m, static_cast<uint32_t>(v)) + static_cast<uint32_t>(v)) >> l);
  }
};

struct TileArgs {
  const int32_t* offsets;
  const int32_t* order;
  int64_t n;
  int x_rows, groups;
  Divisor fan, by_chan_tiles, by_group_tiles;  // tiles over the channels; weight gradient: of a group
  int channels;  // extent of the tiles' height: outer, inner, outer
  int depth;     // extent of the contraction (forward and input gradient)
  int width;     // weight gradient: extent of the tiles' width, inner
  int dtype, out_dtype;
  const uint16_t* x;   // for the gathered copies: rows 16-byte aligned
  int64_t x_stride;
  const uint16_t* dy;  // weight gradient
  int64_t dy_stride;
  void* out;
  int wide_out;        // rows of the output are 16-byte aligned
  uint32_t* status;
  long long wait_cycles;
  int withhold;        // test hook: each unit's last stage is not copied
};

__device__ uint32_t g_product_status;  // kStatusProduct once a bounded wait gave up

__device__ __forceinline__ uint32_t flag_set(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

// Waits for phase `parity` of an mbarrier, at most `limit` cycles or until
// another wait of this CTA has given up.
__device__ __noinline__ bool wait_slow(uint32_t mbar, uint32_t parity, uint32_t gave_up, long long limit,
                                       uint32_t* status) {
  const Waited how = bounded_wait([&] { return mbar_try_wait(mbar, parity); },
                                  [&] { return flag_set(gave_up) != 0u; }, [] { return clock64(); }, limit);
  if (how != Waited::kGaveUp) return how == Waited::kArrived;
  asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(gave_up), "r"(1u) : "memory");
  atomicOr(&g_product_status, kStatusProduct);
  if (status) *reinterpret_cast<volatile uint32_t*>(status) = kStatusProduct;
  return false;
}
__device__ __forceinline__ bool wait_for(uint32_t mbar, uint32_t parity, uint32_t gave_up,
                                         long long limit, uint32_t* status) {
  return mbar_try_wait(mbar, parity) || wait_slow(mbar, parity, gave_up, limit, status);
}

// Shared-memory matrix descriptors, 128-byte swizzle.  K-major: rows of 128
// bytes, groups of 8 rows 1024 bytes apart.  MN-major: boxes of 64 elements by
// 64 depth, 8192 bytes each, in them groups of 8 depth 1024 bytes apart.
constexpr uint64_t kDescBase = (uint64_t{1} << 46) | (uint64_t{2} << 61) | (uint64_t{1024 >> 4} << 32);
template <bool kMnMajor>
__device__ __forceinline__ uint64_t descriptor(uint32_t addr) {
  return kDescBase | (uint64_t{kMnMajor ? 8192 >> 4 : 1} << 16) | ((addr & 0x3ffffu) >> 4);
}

__device__ __forceinline__ uint4 ld_shared_16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
template <typename P>
__device__ __forceinline__ void st_shared_16(uint32_t addr, const P& p) {
  static_assert(sizeof(P) == 16, "one vector");
  const uint4 v = *reinterpret_cast<const uint4*>(&p);
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
template <typename O>
__device__ __forceinline__ void st_shared_value(uint32_t addr, O v) {
  if constexpr (sizeof(O) == 2) {
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"(*reinterpret_cast<const uint16_t*>(&v)) : "memory");
  } else {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(static_cast<float>(v)) : "memory");
  }
}

template <typename O>
__device__ __forceinline__ O ld_shared_value(uint32_t addr) {
  O v;
  if constexpr (sizeof(O) == 2) {
    uint16_t bits;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(bits) : "r"(addr) : "memory");
    *reinterpret_cast<uint16_t*>(&v) = bits;
  } else {
    float bits;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(bits) : "r"(addr) : "memory");
    v = static_cast<O>(bits);
  }
  return v;
}

struct Tile {
  int group;       // `groups`: the rows behind the last group
  int begin, end;  // the group's rows
  int col0;        // first row (weight gradient: first inner column) of the tile
  int chan0;       // first channel
  int block0;      // this CTA's first stage of depth
  int blocks;      // and how many it has
};

template <int kKind, int kCols, int kTeam>
struct Schedule {
  const int32_t* begin;  // [groups + 2] first row of each group, in shared memory
  const int32_t* first;  // [groups + 2] first tile of each group; weight gradient: the groups
                         // by falling size
  Divisor by_chan_tiles, by_group_tiles;  // a tile's place needs no division: 32 rows of 64 experts,
                                          // weight gradient, 99 -> 94 us
  int groups, chan_tiles, width_tiles, depth_blocks;
  int group;
  uint32_t rank, split;
  static constexpr int kHeight = Ring<kCols, kTeam>::kHeight;

  __device__ __forceinline__ Schedule(const int32_t* b, const int32_t* f, const TileArgs& a, uint32_t rank,
                                      uint32_t split)
      : begin(b), first(f), by_chan_tiles(a.by_chan_tiles), by_group_tiles(a.by_group_tiles),
        groups(a.groups), chan_tiles((a.channels + kHeight - 1) / kHeight),
        width_tiles(kKind == kWeightGrad ? (a.width + kCols - 1) / kCols : 0),
        depth_blocks((a.depth + kDepth - 1) / kDepth), group(0), rank(rank), split(split) {}
  __device__ __forceinline__ int tiles_of(int rows) const {
    return (kKind == kWeightGrad ? width_tiles : (rows + kCols - 1) / kCols) * chan_tiles;
  }
  // Groups that own tiles; the weight gradient has none for the rows behind.
  __device__ __forceinline__ int owners() const { return kKind == kWeightGrad ? groups : groups + 1; }
  __device__ __forceinline__ int total() const {
    return kKind == kWeightGrad ? groups * tiles_of(0) : first[owners()];
  }
  // The j-th tile of a unit.  Tiles of the weight gradient differ in depth:
  // with the deepest first, and every other turn the other way, units differ
  // by a fraction of a tile.
  __device__ __forceinline__ static int turn(int j, int unit, int units) {
    return j * units + (kKind == kWeightGrad && (j & 1) ? units - 1 - unit : unit);
  }
  // Tile t; t only grows from call to call.
  __device__ __forceinline__ Tile at(int t) {
    int i;
    if (kKind == kWeightGrad) {
      const int place = by_group_tiles.quotient(t);
      group = first[place];
      i = t - place * tiles_of(0);
    } else {
      // The next group with tiles is often one of the next, but many may be empty.
      for (int near = 0; near < 3 && t >= first[group + 1]; ++near) ++group;
      if (t >= first[group + 1]) {
        int low = group + 1, high = owners() - 1;
        while (low < high) {
          const int mid = (low + high) >> 1;
          if (t >= first[mid + 1]) low = mid + 1;
          else high = mid;
        }
        group = low;
      }
      i = t - first[group];
    }
    Tile r;
    r.group = group;
    r.begin = begin[group];
    r.end = begin[group + 1];
    const int across = by_chan_tiles.quotient(i);
    r.chan0 = (i - across * chan_tiles) * kHeight;
    if (kKind == kWeightGrad) {
      r.col0 = across * kCols;
      r.blocks = (r.end - r.begin + kDepth - 1) / kDepth;
    } else {
      r.col0 = r.begin + across * kCols;
      r.blocks = group < groups ? depth_blocks : 0;
    }
    r.block0 = 0;
    if (kTeam == kSplit) {
      const int all = r.blocks;
      r.block0 = part(all, rank);
      r.blocks = part(all, rank + 1) - r.block0;
    }
    return r;
  }
  // Stages of tile t, all that the matrix instructions and the relay need to
  // know: a tile's whole description would hold them up between two tiles.
  __device__ __forceinline__ int blocks_at(int t, int of_groups) {
    if (kKind == kWeightGrad) return at(t).blocks;
    const int all = t < of_groups ? depth_blocks : 0;
    return kTeam == kSplit ? part(all, rank + 1) - part(all, rank) : all;
  }
  // First stage of a rank's part of `blocks`; the first rank's part is empty
  // only if all are.
  __device__ __forceinline__ int part(int blocks, uint32_t of) const {
    return static_cast<int>((blocks * of + split - 1) >> (31 - __clz(split)));  // split: a power of 2
  }
};

// kN accumulator columns of a warp's 32 lanes (channels) to global memory.
// Rows of the output are columns of the tile (forward, input gradient) or
// channels (weight gradient); either way the warp's block becomes 16-byte
// pieces of output rows through its staging memory.  Without 16-byte rows
// values go one by one, neighbouring lanes to neighbouring places.
template <int kKind, int kN, typename O>
__device__ __forceinline__ void store_block(const TileArgs& a, const Tile& t, int col, int channel0,
                                            const uint32_t (&r)[kN], uint32_t staging) {
  const int lane = threadIdx.x & 31;
  constexpr int V = 16 / sizeof(O);
  if (kKind == kWeightGrad) {
    constexpr int kPieces = kN / V;  // 16-byte pieces of a staged row
    // Exchanged within a row so that rows 128 bytes on meet other banks.
    const auto piece_at = [&](int row, int q) {
      return staging + row * (kN * sizeof(O)) + ((q ^ (row * kPieces / 8 & (kPieces - 1))) << 4);
    };
    O* out = static_cast<O*>(a.out) + static_cast<int64_t>(t.group) * a.channels * a.width;
#pragma unroll
    for (int q = 0; q < kPieces; ++q) {
      Pack<O, V> p;
#pragma unroll
      for (int v = 0; v < V; ++v) p.v[v] = from_float<O>(__uint_as_float(r[q * V + v]));
      st_shared_16(piece_at(lane, q), p);
    }
    __syncwarp();
    if (a.wide_out) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int row = (i * 32 + lane) / kPieces, q = lane & (kPieces - 1);
        const uint4 p = ld_shared_16(piece_at(row, q));
        if (channel0 + row < a.channels && col + q * V < a.width)
          *reinterpret_cast<uint4*>(out + static_cast<int64_t>(channel0 + row) * a.width + col + q * V) = p;
      }
    } else {
      out += static_cast<int64_t>(channel0) * a.width + col;
      const int rows = min(32, a.channels - channel0);
      for (int row = 0; row < rows; ++row, out += a.width)
#pragma unroll
        for (int j = lane; j < kN; j += 32)
          if (col + j < a.width) out[j] = ld_shared_value<O>(piece_at(row, j / V) + j % V * sizeof(O));
    }
    __syncwarp();
  } else {
    O* out = static_cast<O*>(a.out) + static_cast<int64_t>(col) * a.channels + channel0;
    if (a.wide_out) {
      constexpr int kPieces = 32 / V;  // of a staged row: 32 channels
#pragma unroll
      for (int j = 0; j < kN; ++j)
        st_shared_value(staging + (j * 32 + lane) * sizeof(O), from_float<O>(__uint_as_float(r[j])));
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kN * kPieces / 32; ++i) {
        const int row = (i * 32 + lane) / kPieces, q = lane & (kPieces - 1);
        const uint4 p = ld_shared_16(staging + (row * kPieces + q) * 16);
        if (col + row < t.end && channel0 + q * V < a.channels)
          *reinterpret_cast<uint4*>(out + static_cast<int64_t>(row) * a.channels + q * V) = p;
      }
      __syncwarp();
    } else if (channel0 + lane < a.channels) {
      out += lane;
      const int rows = t.end - col;
#pragma unroll
      for (int j = 0; j < kN; ++j, out += a.channels)
        if (j < rows) *out = from_float<O>(__uint_as_float(r[j]));
    }
  }
}

// Zeros in a warp's 32 channels of a tile without any depth: the rows behind
// the last group, the matrices of empty groups.
template <int kKind, int kCols>
__device__ __forceinline__ void store_zeros(const TileArgs& a, const Tile& t, int channel0) {
  // In bytes: `lines` lines of `length`, `pitch` apart.
  const int size = a.out_dtype == DSMEM_F32 ? 4 : 2, lane = threadIdx.x & 31;
  const int channels = min(32, a.channels - channel0);
  if (channels <= 0) return;
  const int cols = min(kCols, (kKind == kWeightGrad ? a.width : t.end) - t.col0);
  const int lines = kKind == kWeightGrad ? channels : cols;
  const int length = (kKind == kWeightGrad ? cols : channels) * size;
  const int64_t pitch = static_cast<int64_t>(kKind == kWeightGrad ? a.width : a.channels) * size;
  const int64_t first = kKind == kWeightGrad
                            ? (static_cast<int64_t>(t.group) * a.channels + channel0) * a.width + t.col0
                            : static_cast<int64_t>(t.col0) * a.channels + channel0;
  uint8_t* out = static_cast<uint8_t*>(a.out) + first * size;
  const auto clear = [&](auto zero) {
    const int per_line = length / static_cast<int>(sizeof(zero));
    int shift = 0;  // 1 << shift lanes a line
    while (shift < 5 && (1 << shift) < per_line) ++shift;
    for (int i = lane & ((1 << shift) - 1); i < per_line; i += 1 << shift) {
      uint8_t* p = out + (lane >> shift) * pitch + i * static_cast<int>(sizeof(zero));
#pragma unroll 8
      for (int line = lane >> shift; line < lines; line += 32 >> shift, p += (32 >> shift) * pitch)
        *reinterpret_cast<decltype(zero)*>(p) = zero;
    }
  };
  if (a.wide_out) clear(make_uint4(0, 0, 0, 0));
  else if (size == 4) clear(uint32_t{0});
  else clear(uint16_t{0});
}

template <int kKind, int kN>
__device__ __forceinline__ void store_any(const TileArgs& a, const Tile& t, int col, int channel0,
                                          const uint32_t (&r)[kN], uint32_t staging) {
  if (kN <= 32 && a.out_dtype == DSMEM_F32) store_block<kKind, kN, float>(a, t, col, channel0, r, staging);
  else if (a.out_dtype == DSMEM_F16) store_block<kKind, kN, __half>(a, t, col, channel0, r, staging);
  else store_block<kKind, kN, __nv_bfloat16>(a, t, col, channel0, r, staging);
}

// The gathering warps: x's rows named by the order, and the rows of a ragged
// stage of the weight gradient (dy's too), 16 bytes a copy.  Each thread's
// copies of a stage arrive on `landed` by themselves, so that the warps go on
// to the next stage at once; the relay warp passes a landed stage on.  (Warps
// that waited for their own copies had three stages in flight at most, and
// the forward product took 370 instead of 360 us at that step.)
template <int kKind, int kCols, int kTeam>
__device__ __forceinline__ void gather_rows(const TileArgs& a, Schedule<kKind, kCols, kTeam>& schedule,
                                            int unit, int units, uint32_t half, int total, uint32_t base,
                                            uint32_t landed, uint32_t empty, uint32_t gave_up) {
  using R = Ring<kCols, kTeam>;
  constexpr int kStages = R::kStages, kStage = R::kStage, kMine = R::kMine;
  constexpr bool kBMn = kKind == kWeightGrad;
  const int shift = (threadIdx.x - 6 * 32) / kShift, tid = (threadIdx.x - 6 * 32) % kShift;
  const int lane = threadIdx.x & 31;
  uint32_t before = 0;  // stages of earlier tiles
  bool ok = true;

  // The order's entry for place p and the row of x it names.  Apart, so that
  // the load's latency is not waited for where it is issued.
  const auto place = [&](int p, int end) { return p < end ? (a.order ? a.order[p] : p) : -1; };
  const auto named_row = [&](int o) {
    const int row = o < 0 ? -1 : (a.order ? a.fan.quotient(o) : o);
    return row < a.x_rows ? row : -1;
  };
  // Forward and input gradient: 8 threads a row of 128 bytes; the rows are the
  // same in every stage of a tile.
  constexpr int kLines = kShift / 8, kRows = kBMn ? 1 : (kMine + kLines - 1) / kLines;
  // Weight gradient: kPieces threads a row of kMine elements.  A warp needs
  // kFound rows of a stage; its lanes look up those of kBatch stages at once,
  // a batch ahead.
  constexpr int kPieces = kMine / 8, kAtOnce = kShift / kPieces, kPerWarp = 32 / kPieces;
  constexpr int kFound = kDepth / (kShift / 32), kBatch = 32 / kFound;
  static_assert(kFound <= 32 && kPerWarp >= 1 && kAtOnce >= 1, "a warp looks up a stage's rows at once");
  // This shift's stages of a tile are first_of(before), and every kShifts-th.
  const auto first_of = [&](uint32_t stages) {
    return static_cast<int>((shift - stages % kShifts + kShifts) % kShifts);
  };
  const auto batch_place = [&](const Tile& t, int first_k, int m) {
    const int l = lane % kFound;
    const int r = l / kPerWarp * kAtOnce + (tid >> 5) * kPerWarp + l % kPerWarp;
    return place(t.begin + (t.block0 + first_k + (m + lane / kFound) * kShifts) * kDepth + r, t.end);
  };
  // A tile's entries of the order are asked for while the tile before is
  // copied: they take longer to arrive than a stage.
  int ahead[kRows];
  const auto ask = [&](const Tile& t, uint32_t stages) {
#pragma unroll
    for (int r = 0; r < kRows; ++r)
      ahead[r] = kBMn ? batch_place(t, first_of(stages), 0)
                      : place(t.col0 + static_cast<int>(half) * kMine + r * kLines + tid / 8, t.end);
  };

  Tile next;
  if (unit < total) {
    next = schedule.at(unit);
    ask(next, 0);
  }
  for (int j = 0, i = unit; i < total && ok;) {
    const Tile t = next;
    const int col0 = t.col0 + half * kMine, chan0 = t.chan0 + half * kChannels;
    const int first_k = first_of(before);
    int row[kRows];
    int here = 0, later = kBMn ? ahead[0] : 0;
    if (!kBMn) {
#pragma unroll
      for (int r = 0; r < kRows; ++r) row[r] = named_row(ahead[r]);
    }
    i = schedule.turn(++j, unit, units);
    if (i < total) {
      next = schedule.at(i);
      ask(next, before + t.blocks);
    }

    for (int m = 0, k = first_k; k < t.blocks; ++m, k += kShifts) {
      if (kBMn && m % kBatch == 0) {
        here = named_row(later);
        later = batch_place(t, first_k, m + kBatch);
      }
      const uint32_t stage = (before + k) % kStages, phase = (before + k) / kStages & 1;
      ok = wait_for(empty + 8 * stage, phase ^ 1, gave_up, a.wait_cycles, a.status);
      ok = __all_sync(kFull, ok);
      if (!ok) break;
      const uint32_t sa = base + stage * kStage, sb = sa + kABytes;
      if (!kBMn) {
        const int c = tid & 7, col = (t.block0 + k) * kDepth + c * 8;
        const int left = max(0, min(8, a.depth - col)) * 2;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          const int line = r * kLines + tid / 8;
          const bool read = row[r] >= 0 && left > 0;
          if (kMine % kLines == 0 || line < kMine)
            copy16(sb + line * 128 + ((c ^ (line & 7)) << 4),
                 a.x + (read ? row[r] * a.x_stride + col : 0), read ? left : 0);
        }
      } else {
        const int p0 = t.begin + (t.block0 + k) * kDepth;
        const bool ragged = p0 + kDepth > t.end;
        if (a.order || ragged) {
          const int c = tid % kPieces, col = col0 + c * 8;
          const int left = max(0, min(8, a.width - col)) * 2;
#pragma unroll
          for (int r = 0; r < kDepth / kAtOnce; ++r) {
            const int line = r * kAtOnce + tid / kPieces;
            const int from = __shfl_sync(kFull, here, m % kBatch * kFound + r * kPerWarp + lane / kPieces);
            const bool read = from >= 0 && left > 0;
            copy16(sb + (c >> 3) * 8192 + line * 128 + (((c & 7) ^ (line & 7)) << 4),
                   a.x + (read ? from * a.x_stride + col : 0), read ? left : 0);
          }
        }
        if (ragged) {
          const int c = tid & 15, col = chan0 + c * 8;
          const int left = max(0, min(8, a.channels - col)) * 2;
#pragma unroll
          for (int r = 0; r < kDepth * 16 / kShift; ++r) {
            const int line = r * (kShift / 16) + tid / 16;
            const bool read = p0 + line < t.end && left > 0;
            copy16(sa + (c >> 3) * 8192 + line * 128 + (((c & 7) ^ (line & 7)) << 4),
                   a.dy + (read ? (p0 + line) * a.dy_stride + col : 0), read ? left : 0);
          }
        }
      }
      copy_arrive(landed + 8 * stage);
    }
    before += t.blocks;
  }
  copy_wait_all();
}

template <int kKind, int kCols, int kTeam>
__global__ void __launch_bounds__(kThreads, 1)
    product_kernel(const __grid_constant__ Maps maps, const __grid_constant__ TileArgs a) {
  using R = Ring<kCols, kTeam>;
  constexpr bool kTwo = kTeam == kPair;
  constexpr int kStages = R::kStages, kStage = R::kStage, kMine = R::kMine;
  constexpr bool kAMn = kKind != kForward, kBMn = kKind == kWeightGrad;
  constexpr uint32_t kTmemColumns = 2 * kCols < 32 ? 32 : 2 * kCols;
  constexpr int kLoad = kCols < 32 ? 16 : 32;
  // Descriptor steps of 16 depth, in 16-byte units.
  constexpr uint64_t kAStep = (kAMn ? 2048 : 32) / 16, kBStep = (kBMn ? 2048 : 32) / 16;

  extern __shared__ uint8_t raw[];
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  uint8_t* base_ptr = raw + (base - smem_u32(raw));
  const uint32_t join = base + kStages * kStage;
  const uint32_t members = kTeam == kSplit ? cluster_nctarank() : (kTwo ? 2u : 1u);
  const uint32_t out_staging = join + (kTeam == kSplit ? members - 1 : 0) * R::kJoin;
  const uint32_t bars = out_staging + 4 * kStageOut;
  const uint32_t full = bars, empty = bars + 8 * kStages;
  const uint32_t landed = empty + 8 * kStages;
  const uint32_t acc_full = landed + 8 * kStages, acc_empty = acc_full + 16, drained = acc_empty + 16;
  const uint32_t tmem_at = drained + 8, gave_up = tmem_at + 4;
  static_assert(8 * (3 * kStages + 5) + 8 <= kBarrierBytes, "barriers");
  int32_t* begin = reinterpret_cast<int32_t*>(base_ptr + (bars - base) + kBarrierBytes);
  int32_t* first = begin + a.groups + 2;

  const int warp = __shfl_sync(kFull, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  // A unit works on a tile: a CTA, or a cluster whose first CTA leads.
  const uint32_t rank = kTeam != kSolo ? cluster_ctarank() : 0u;
  const uint32_t half = kTwo ? rank : 0u;
  const int unit = blockIdx.x / members, units = gridDim.x / members;
  Schedule<kKind, kCols, kTeam> schedule(begin, first, a, rank, members);
  // The gathering warps take part in every stage where x is gathered, or
  // where a contraction may end inside a stage.
  const bool gathering = kBMn || a.order;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      // The TMA thread and the relays; of a pair, the leader's barriers count
      // both CTAs.
      mbar_init(full + 8 * s, 1 + (gathering ? (kTwo ? 2 : 1) : 0));
      mbar_init(landed + 8 * s, kShift);
      mbar_init(empty + 8 * s, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full + 8 * i, 1);
      mbar_init(acc_empty + 8 * i, kTwo ? 8 : 4);
    }
    mbar_init(drained, 1);
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(gave_up), "r"(0u) : "memory");
    fence_mbar_init();
    prefetch_map(&maps.a);
    prefetch_map(&maps.b);
  }
  // begin[g + 1] := the group's end, clamped into [0, n]; then the ends are made
  // monotone and the tiles laid end to end.
  for (int g = threadIdx.x; g < a.groups; g += kThreads) {
    const int64_t e = a.offsets[g + 1];
    begin[g + 1] = static_cast<int32_t>(e < 0 ? 0 : (e > a.n ? a.n : e));
  }
  if (threadIdx.x == 0) {
    begin[0] = 0;
    if (kKind != kWeightGrad) first[0] = 0;
    begin[a.groups + 1] = static_cast<int32_t>(a.n);
  }
  if (warp == 1) tmem_alloc<kTwo>(tmem_at, kTmemColumns);
  __syncthreads();
  // Each warp takes 32 groups of every kWarps * 32: the running maximum
  // of their ends, then the running sum of their tiles.
  constexpr int kWarps = kThreads / 32;
  __shared__ int of_warp[2][32];
  int end_before = 0, tiles_before = 0;
  for (int g0 = 0; g0 < schedule.owners(); g0 += kWarps * 32) {
    const int g = g0 + warp * 32 + lane;
    const bool owner = g < schedule.owners();
    int end = owner ? begin[g + 1] : 0;
    const int most = __reduce_max_sync(kFull, end);
    if (lane == 0) of_warp[0][warp] = most;
    __syncthreads();
    const int other = lane < kWarps ? of_warp[0][lane] : 0;
    const int earlier = max(end_before, __reduce_max_sync(kFull, lane < warp ? other : 0));
    end_before = max(end_before, __reduce_max_sync(kFull, other));
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(kFull, end, d);
      if (lane >= d) end = max(end, up);
    }
    end = max(end, earlier);
    int start = __shfl_up_sync(kFull, end, 1);
    if (lane == 0) start = earlier;
    int tiles = owner ? schedule.tiles_of(end - start) : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(kFull, tiles, d);
      if (lane >= d) tiles += up;
    }
    if (lane == 31) of_warp[1][warp] = tiles;
    __syncthreads();
    const int sum = lane < kWarps ? of_warp[1][lane] : 0;
    tiles += tiles_before + __reduce_add_sync(kFull, lane < warp ? sum : 0);
    tiles_before += __reduce_add_sync(kFull, sum);
    if (owner) {
      begin[g + 1] = end;
      if (kKind != kWeightGrad) first[g + 1] = tiles;
    }
  }
  if (kKind == kWeightGrad) {
    // The groups by falling size (by number alone where counting the larger
    // ones of each would take longer than it saves).
    __syncthreads();
    for (int g = threadIdx.x; g < a.groups; g += kThreads) {
      int place = g;
      if (a.groups <= kMostSorted) {
        const int size = begin[g + 1] - begin[g];
        place = 0;
        for (int h = 0; h < a.groups; ++h) {
          const int other = begin[h + 1] - begin[h];
          place += other > size || (other == size && h < g);
        }
      }
      first[place] = g;
    }
  }
  tcgen_fence_before();
  if (kTeam != kSolo) cluster_barrier();
  else __syncthreads();
  tcgen_fence_after();
  uint32_t tmem;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(tmem_at));
  const int total = schedule.total();
  const int of_groups = kKind == kWeightGrad ? total : first[a.groups];  // tiles of real groups

  // Output: warp w may read lanes 32 (w % 4) .. of tensor memory.
  const int quadrant = warp & 3;

  if (warp == 0) {
    // TMA copies.
    uint32_t stage = 0, phase = 0, issued = 0;
    bool ok = true;
    for (int j = 0, i = unit; i < total && ok; i = schedule.turn(++j, unit, units)) {
      const Tile t = schedule.at(i);
      for (int k = 0; k < t.blocks; ++k) {
        ok = __all_sync(kFull, wait_for(empty + 8 * stage, phase ^ 1, gave_up, a.wait_cycles, a.status));
        if (!ok || (a.withhold && schedule.turn(j + 1, unit, units) >= total && k + 1 == t.blocks)) break;
        const uint32_t sa = base + stage * kStage, sb = sa + kABytes;
        const uint32_t bar = kTwo ? map_rank(full + 8 * stage, 0) : full + 8 * stage;
        const int k0 = (t.block0 + k) * kDepth;
        const int p0 = t.begin + k0;  // weight gradient: the stage's first row
        const int chan0 = t.chan0 + half * kChannels, col0 = t.col0 + half * kMine;
        const bool ragged = kBMn && p0 + kDepth > t.end;
        if (elect_one()) {
          if (half == 0)
            mbar_expect_tx(full + 8 * stage, (ragged ? 0 : (a.order ? kABytes : kStage)) * (kTwo ? 2 : 1));
          if (kKind == kForward) {
            tma_load_3d<kTwo>(sa, &maps.a, k0, chan0, t.group, bar);
          } else if (kKind == kInputGrad) {
            tma_load_3d<kTwo>(sa, &maps.a, chan0, k0, t.group, bar);
            tma_load_3d<kTwo>(sa + 8192, &maps.a, chan0 + 64, k0, t.group, bar);
          } else if (!ragged) {
            tma_load_2d<kTwo>(sa, &maps.a, chan0, p0, bar);
            tma_load_2d<kTwo>(sa + 8192, &maps.a, chan0 + 64, p0, bar);
          }
          if (!a.order && !ragged) {
            if (kBMn) {
#pragma unroll
              for (int box = 0; box < kMine / 64; ++box)
                tma_load_2d<kTwo>(sb + box * 8192, &maps.b, col0 + box * 64, p0, bar);
            } else {
              tma_load_2d<kTwo>(sb, &maps.b, k0, col0, bar);
            }
          }
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
    // memory goes.  Copy j (from 0) completes phase j / kStages of its stage
    // (where the gathering warps came along; else the wait runs out).  The
    // leader's barriers count the pair's copies, and the other CTA stays until
    // the leader is done.
    if (half == 0 && flag_set(gave_up)) {
      for (uint32_t j = issued > kStages ? issued - kStages : 0; j < issued; ++j) {
        const long long deadline = clock64() + kDefaultWaitCycles;
        while (!mbar_try_wait(full + 8 * (j % kStages), (j / kStages) & 1) && clock64() < deadline) {
        }
      }
    }
    __syncwarp();
  } else if (warp == kRelayWarp) {
    // Gathered stages, once landed, on to the matrix instructions.
    if (gathering && lane == 0) {
      uint32_t stage = 0, phase = 0;
      bool ok = true;
      for (int j = 0, i = unit; i < total && ok; i = schedule.turn(++j, unit, units)) {
        const int blocks = schedule.blocks_at(i, of_groups);
        for (int k = 0; k < blocks; ++k) {
          ok = wait_for(landed + 8 * stage, phase, gave_up, a.wait_cycles, a.status);
          if (!ok) break;
          fence_async_shared();
          if (kTwo) mbar_arrive_pair(map_rank(full + 8 * stage, 0));
          else mbar_arrive_local(full + 8 * stage);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
    }
    __syncwarp();
  } else if (warp >= 6) {
    if (gathering)
      gather_rows<kKind, kCols, kTeam>(a, schedule, unit, units, half, total, base, landed, empty, gave_up);
  } else if (warp == 1) {
    // Matrix instructions; a pair's by its leader.
    if (half == 0) {
      const uint32_t idesc = (1u << 4) | (a.dtype == DSMEM_BF16 ? (1u << 7) | (1u << 10) : 0u) |
                             (kAMn ? 1u << 15 : 0u) | (kBMn ? 1u << 16 : 0u) |
                             (uint32_t{kCols >> 3} << 17) | (uint32_t{R::kHeight >> 4} << 24);
      uint32_t stage = 0, phase = 0, done = 0;
      bool ok = true;
      for (int j = 0, i = unit; i < total && ok; i = schedule.turn(++j, unit, units)) {
        const int blocks = schedule.blocks_at(i, of_groups);
        if (blocks == 0) continue;
        const uint32_t buffer = done & 1, d = tmem + buffer * kCols;
        ok = __all_sync(kFull, wait_for(acc_empty + 8 * buffer, ((done >> 1) & 1) ^ 1, gave_up, a.wait_cycles,
                                        a.status));
        if (!ok) break;
        tcgen_fence_after();
        for (int k = 0; k < blocks; ++k) {
          ok = __all_sync(kFull, wait_for(full + 8 * stage, phase, gave_up, a.wait_cycles, a.status));
          if (!ok) break;
          tcgen_fence_after();
          const uint32_t sa = base + stage * kStage;
          const uint64_t da = descriptor<kAMn>(sa), db = descriptor<kBMn>(sa + kABytes);
          if (elect_one()) {
#pragma unroll
            for (int s = 0; s < kDepth / 16; ++s)
              mma_f16<kTwo>(d, da + s * kAStep, db + s * kBStep, idesc, k > 0 || s > 0);
            mma_commit<kTwo>(empty + 8 * stage);
            if (k + 1 == blocks) mma_commit<kTwo>(acc_full + 8 * buffer);
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
        if (elect_one()) mma_commit<kTwo>(drained);
        __syncwarp();
        const long long deadline = clock64() + kDefaultWaitCycles;
        while (!mbar_try_wait(drained, 0) && clock64() < deadline) {
        }
      }
    }
    __syncwarp();
  } else if (kTeam == kSplit) {
    // A unit has one tile at most.  All but the leader hand it their sums.
    if (unit < total) {
      const Tile t = schedule.at(unit);
      if (t.blocks > 0) {
        const bool ok = wait_for(acc_full, 0, gave_up, a.wait_cycles + 4096ll * t.blocks, a.status);
        if (__all_sync(kFull, ok) && rank != 0) {
          tcgen_fence_after();
          const uint32_t d = tmem + (static_cast<uint32_t>(quadrant * 32) << 16);
          const uint32_t to = map_rank(join + (rank - 1) * R::kJoin + (quadrant * 32 + lane) * 16, 0);
#pragma unroll 1
          for (int c = 0; c < kCols; c += 16) {
            uint32_t r[16];
            tmem_load16(d + c, r);
            tmem_wait_load();
#pragma unroll
            for (int j = 0; j < 16; j += 4)
              st_cluster_16(to + (c + j) / 4 * (kChannels * 16), r[j], r[j + 1], r[j + 2], r[j + 3]);
          }
        }
      }
    }
    __syncwarp();
  } else {
    uint32_t done = 0;
    for (int j = 0, i = unit; i < total; i = schedule.turn(++j, unit, units)) {
      const Tile t = schedule.at(i);
      const uint32_t buffer = done & 1;
      if (t.blocks > 0) {
        // A long contraction may take longer than one bounded wait of a copy.
        const long long limit = a.wait_cycles + 4096ll * t.blocks;
        const bool ok = wait_for(acc_full + 8 * buffer, (done >> 1) & 1, gave_up, limit, a.status);
        if (!__all_sync(kFull, ok)) break;
        tcgen_fence_after();
      }
      const uint32_t d = tmem + buffer * kCols + (static_cast<uint32_t>(quadrant * 32) << 16);
      const uint32_t staging = out_staging + quadrant * kStageOut;
      const int limit = kKind == kWeightGrad ? a.width : t.end;
      const int channel0 = t.chan0 + half * kChannels + quadrant * 32;
      if (t.blocks == 0) {
        store_zeros<kKind, kCols>(a, t, channel0);
        continue;
      }
      if (kKind == kWeightGrad && kCols >= 64 && a.out_dtype != DSMEM_F32) {
        // 128 bytes of an output row at a time.
#pragma unroll 1
        for (int c = 0; c < kCols && t.col0 + c < limit; c += 64) {
          uint32_t r[64];
          tmem_load32(d + c, reinterpret_cast<uint32_t(&)[32]>(r[0]));
          tmem_load32(d + c + 32, reinterpret_cast<uint32_t(&)[32]>(r[32]));
          tmem_wait_load();
          store_any<kKind, 64>(a, t, t.col0 + c, channel0, r, staging);
        }
      } else {
#pragma unroll 1
        for (int c = 0; c < kCols && t.col0 + c < limit; c += kLoad) {
          uint32_t r[kLoad];
          if constexpr (kLoad == 32) tmem_load32(d + c, r);
          else tmem_load16(d + c, r);
          tmem_wait_load();
          store_any<kKind, kLoad>(a, t, t.col0 + c, channel0, r, staging);
        }
      }
      tcgen_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (kTwo) mbar_arrive_pair(map_rank(acc_empty + 8 * buffer, 0));
        else mbar_arrive_local(acc_empty + 8 * buffer);
      }
      ++done;
    }
    __syncwarp();
  }
  // Nothing of a cluster leaves while another CTA may read or write its memory
  // or arrive on its barriers.
  tcgen_fence_before();
  if (kTeam != kSolo) cluster_barrier();
  else __syncthreads();
  tcgen_fence_after();
  if (kTeam == kSplit && rank == 0 && warp >= 2 && warp < 6 && unit < total) {
    // The leader's sums, then the other ranks', in their order.
    const Tile t = schedule.at(unit);
    const int all = t.group < a.groups ? (kKind == kWeightGrad ? (t.end - t.begin + kDepth - 1) / kDepth
                                                               : schedule.depth_blocks) : 0;
    const uint32_t d = tmem + (static_cast<uint32_t>(quadrant * 32) << 16);
    const uint32_t from = join + (quadrant * 32 + lane) * 16;
    const int limit = kKind == kWeightGrad ? a.width : t.end;
#pragma unroll 1
    for (int c = 0; c < kCols; c += 16) {
      if (t.col0 + c >= limit) break;
      uint32_t r[16];
      if (all > 0) {
        tmem_load16(d + c, r);
        tmem_wait_load();
        for (uint32_t o = 1; o < members; ++o) {
          if (schedule.part(all, o) == schedule.part(all, o + 1)) continue;
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            const uint4 v = ld_shared_16(from + (o - 1) * R::kJoin + (c + j) / 4 * (kChannels * 16));
            r[j] = __float_as_uint(__uint_as_float(r[j]) + __uint_as_float(v.x));
            r[j + 1] = __float_as_uint(__uint_as_float(r[j + 1]) + __uint_as_float(v.y));
            r[j + 2] = __float_as_uint(__uint_as_float(r[j + 2]) + __uint_as_float(v.z));
            r[j + 3] = __float_as_uint(__uint_as_float(r[j + 3]) + __uint_as_float(v.w));
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) r[j] = 0u;
      }
      store_any<kKind, 16>(a, t, t.col0 + c, t.chan0 + quadrant * 32, r, out_staging + quadrant * kStageOut);
    }
  }
  if (kTeam == kSplit) {
    tcgen_fence_before();
    __syncthreads();
    tcgen_fence_after();
  }
  if (warp == 1) tmem_dealloc<kTwo>(tmem, kTmemColumns);
}

// Lays rows whose bases or strides TMA cannot take out with rows of a
// multiple of 8 elements; both sources of a product in one launch.  A CTA takes
// a block of a group's rows, a warp 256 elements of a row at a time and a lane
// 8: 32-bit words, joined where the row begins between two of them, and single
// elements at a row's ends.  Matrices of groups without rows are left out.
// Bound by memory: 402 MB of matrices in 143 us, 5.6 TB/s.
struct Layout {
  const uint16_t* src;
  int64_t row_stride, group_stride;
  uint16_t* dst;
  const int32_t* offsets;  // of the groups, or null
  int rows, cols, dst_stride;
  int pieces, block, blocks;  // 256-element pieces of a row, rows of a block, blocks of a group
  int ctas;
  Divisor by_pieces;
};
struct Layouts {
  Layout of[2];
};
__device__ __forceinline__ uint4 aligned_piece(const uint16_t* row, int c, int cols, bool between) {
  if (!between && c + 8 <= cols) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(row + c);
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (between && c > 0 && c + 8 < cols) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(row + c - 1);
    const uint32_t w0 = w[0], w1 = w[1], w2 = w[2], w3 = w[3], w4 = w[4];
    return make_uint4(__funnelshift_r(w0, w1, 16), __funnelshift_r(w1, w2, 16), __funnelshift_r(w2, w3, 16),
                      __funnelshift_r(w3, w4, 16));
  }
  uint32_t e[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) e[k] = c + k < cols ? row[c + k] : 0u;
  return make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
}
__global__ void __launch_bounds__(256) layout_kernel(const __grid_constant__ Layouts layouts) {
  const int cta = blockIdx.x;
  const bool second = cta >= layouts.of[0].ctas;
  const Layout& l = layouts.of[second];
  const int j = second ? cta - layouts.of[0].ctas : cta;
  const int group = j / l.blocks, row0 = (j - group * l.blocks) * l.block;
  if (l.offsets && l.offsets[group + 1] <= (group > 0 ? l.offsets[group] : 0)) return;
  const uint16_t* src = l.src + group * l.group_stride;
  uint16_t* dst = l.dst + static_cast<int64_t>(group) * l.rows * l.dst_stride;
  const int total = min(l.block, l.rows - row0) * l.pieces;
#pragma unroll 4
  for (int q = threadIdx.x >> 5; q < total; q += 8) {
    const int line = l.by_pieces.quotient(q);
    const int c = (q - line * l.pieces) * 256 + (threadIdx.x & 31) * 8;
    if (c >= l.dst_stride) continue;
    const uint16_t* row = src + (row0 + line) * l.row_stride;
    *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(row0 + line) * l.dst_stride + c) =
        aligned_piece(row, c, l.cols, (reinterpret_cast<uintptr_t>(row) & 2u) != 0);
  }
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encoder() {
  static EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) !=
            cudaSuccess || found != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// A 16-bit tensor [groups, rows, cols] in boxes of box_rows x 64.
int make_map(CUtensorMap* map, int dtype, const void* data, int64_t cols, int64_t rows, int64_t groups,
             int64_t row_stride, int64_t group_stride, int box_rows, bool three) {
  const EncodeFn encode = encoder();
  if (!encode) return fail_with(DSMEM_HIST_EUNSUPPORTED, "the driver has no tensor maps");
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(groups)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(row_stride) * 2,
                                 static_cast<cuuint64_t>(group_stride) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1}, unit[3] = {1, 1, 1};
  const CUresult r = encode(
      map, dtype == DSMEM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
      three ? 3 : 2, const_cast<void*>(data), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail_with(DSMEM_HIST_ECUDA, "cuTensorMapEncodeTiled: error %d (%lld x %lld x %lld)",
                     static_cast<int>(r), static_cast<long long>(cols), static_cast<long long>(rows),
                     static_cast<long long>(groups));
  return DSMEM_HIST_OK;
}

bool tma_ready(const void* p, int64_t row_stride, int64_t group_stride, int64_t groups) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && row_stride % 8 == 0 &&
         (groups == 1 || group_stride % 8 == 0);
}

// One source of a product, [groups, rows, cols] of 16-bit elements.
struct Source {
  const void* data;
  int64_t row_stride, group_stride, rows, cols, groups;
  const int32_t* offsets;  // groups whose offsets show no rows are not read, or null
};

// Lays the sources TMA cannot read in place out in scratch, which the caller
// gives back.
int lay_out(const CallContext& ctx, Source* sources[2], void** scratch, cudaStream_t stream) {
  Layouts layouts = {};
  int64_t bytes = 0, ctas = 0;
  for (int i = 0; i < 2; ++i) {
    Source& s = *sources[i];
    if (tma_ready(s.data, s.row_stride, s.group_stride, s.groups)) {
      if (s.groups == 1) s.group_stride = s.row_stride;  // unused, but checked
      continue;
    }
    Layout& l = layouts.of[i];
    l.src = static_cast<const uint16_t*>(s.data);
    l.row_stride = s.row_stride, l.group_stride = s.group_stride;
    l.rows = static_cast<int>(s.rows), l.cols = static_cast<int>(s.cols);
    l.dst_stride = static_cast<int>((s.cols + 7) / 8 * 8);
    l.offsets = s.offsets;
    l.pieces = (l.dst_stride + 255) / 256;
    l.by_pieces = Divisor(static_cast<uint32_t>(l.pieces));
    // 8 to 64 pieces a CTA, small sources over all SMs several times.
    const int64_t each = s.groups * s.rows * l.pieces / (ctx.sm_count * 8);
    l.block = std::max(1, static_cast<int>(std::min<int64_t>(std::max<int64_t>(each, 8), 64)) / l.pieces);
    l.blocks = (l.rows + l.block - 1) / l.block;
    const int64_t mine = s.groups * l.blocks;
    if (mine + ctas > INT32_MAX) return fail_with(DSMEM_HIST_EINVAL, "grouped product: too many rows to lay out");
    l.ctas = static_cast<int>(mine);
    ctas += mine;
    bytes += s.groups * s.rows * l.dst_stride * 2;
  }
  if (ctas == 0) return DSMEM_HIST_OK;
  int rc = pool_alloc(ctx, scratch, static_cast<size_t>(bytes), stream);
  if (rc) return rc;
  uint16_t* at = static_cast<uint16_t*>(*scratch);
  for (int i = 0; i < 2; ++i) {
    Layout& l = layouts.of[i];
    if (l.ctas == 0) continue;
    l.dst = at;
    at += sources[i]->groups * sources[i]->rows * l.dst_stride;
    sources[i]->data = l.dst;
    sources[i]->row_stride = l.dst_stride;
    sources[i]->group_stride = static_cast<int64_t>(l.dst_stride) * l.rows;
  }
  layout_kernel<<<static_cast<unsigned>(ctas), 256, 0, stream>>>(layouts);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? DSMEM_HIST_OK : fail_with_cuda(e, "layout launch");
}

// Upper bound of a product's tiles: the group sizes are not known here.
int64_t tile_bound(const ProductArgs& p, int cols, int height) {
  const int64_t channels = p.kind == kInputGrad ? p.inner : p.outer;
  const int64_t across = p.kind == kWeightGrad ? static_cast<int64_t>(p.groups) * ((p.inner + cols - 1) / cols)
                                               : p.n / cols + std::min<int64_t>(p.groups + 1, p.n);
  return across * ((channels + height - 1) / height);
}

cudaLaunchAttribute cluster_of(int ctas) {
  cudaLaunchAttribute a = {};
  a.id = cudaLaunchAttributeClusterDimension;
  a.val.clusterDim.x = static_cast<unsigned>(ctas);
  a.val.clusterDim.y = a.val.clusterDim.z = 1;
  return a;
}

template <int kKind, int kCols, int kTeam>
cudaError_t allow_smem(int device, int bytes) {
  static SmemLimit limit;
  return limit.need(reinterpret_cast<const void*>(product_kernel<kKind, kCols, kTeam>), device, bytes);
}

template <int kKind, int kCols, int kTeam>
int launch(const ProductArgs& p, const CallContext& ctx, const Source& x, const Source& w, int split,
           cudaStream_t stream) {
  using R = Ring<kCols, kTeam>;
  TileArgs a{};
  a.offsets = p.offsets, a.order = p.order, a.n = p.n;
  a.x_rows = static_cast<int>(p.x_rows), a.groups = p.groups, a.fan = Divisor(static_cast<uint32_t>(p.fan));
  a.channels = kKind == kInputGrad ? p.inner : p.outer;
  a.depth = kKind == kInputGrad ? p.outer : p.inner;
  a.width = p.inner;
  const uint32_t chan_tiles = static_cast<uint32_t>((a.channels + R::kHeight - 1) / R::kHeight);
  a.by_chan_tiles = Divisor(chan_tiles);
  a.dtype = p.dtype, a.out_dtype = p.out_dtype, a.out = p.out;
  a.x = static_cast<const uint16_t*>(x.data), a.x_stride = x.row_stride;
  a.dy = static_cast<const uint16_t*>(w.data), a.dy_stride = w.row_stride;
  const int64_t out_cols = kKind == kWeightGrad ? a.width : a.channels;
  a.wide_out = reinterpret_cast<uintptr_t>(p.out) % 16 == 0 && out_cols * dtype_size(p.out_dtype) % 16 == 0;
  a.status = ctx.status;
  a.wait_cycles = call_wait_cycles();
  a.withhold = call_withholds();

  Maps m;
  const int x_cols = kKind == kInputGrad ? p.outer : p.inner;
  int rc;
  if (kKind == kWeightGrad) {
    if ((rc = make_map(&m.a, p.dtype, w.data, p.outer, p.n, 1, w.row_stride, 0, kDepth, false)) ||
        (rc = make_map(&m.b, p.dtype, x.data, x_cols, p.x_rows, 1, x.row_stride, 0, kDepth, false)))
      return rc;
  } else {
    if ((rc = make_map(&m.a, p.dtype, w.data, p.inner, p.outer, p.groups, w.row_stride, w.group_stride,
                       kKind == kForward ? kChannels : kDepth, true)) ||
        (rc = make_map(&m.b, p.dtype, x.data, x_cols, p.x_rows, 1, x.row_stride, 0, R::kMine, false)))
      return rc;
  }

  const int64_t tiles = tile_bound(p, kCols, R::kHeight);
  if (tiles > INT32_MAX - 1024)  // tile counters step past the last tile
    return fail_with(DSMEM_HIST_EINVAL, "grouped product: more than 2^31 output tiles");
  if (kKind == kWeightGrad) a.by_group_tiles = Divisor(static_cast<uint32_t>(tiles / p.groups));
  const int smem = R::smem_bytes(p.groups, kTeam == kSplit ? split : 1);
  const auto kernel = product_kernel<kKind, kCols, kTeam>;
  cudaError_t e = allow_smem<kKind, kCols, kTeam>(ctx.device, smem);
  if (e != cudaSuccess) return fail_with_cuda(e, "cudaFuncSetAttribute");
  const int per_unit = kTeam == kSplit ? split : (kTeam == kPair ? 2 : 1);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(tiles, ctx.sm_count / per_unit)) * per_unit);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr = cluster_of(per_unit);
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, m, a);
  return e == cudaSuccess ? DSMEM_HIST_OK : fail_with_cuda(e, "grouped product launch");
}

// Clusters of `split` CTAs of a split kernel that are resident together, asked
// of the runtime once.  (One CTA fills an SM, whatever the tables of the groups
// take of its shared memory.)
constexpr int kMostGroupsOf8 = 1024;  // beside longer tables the sums of 8 CTAs do not fit
template <int kKind, int kCols>
int resident_clusters(const CallContext& ctx, int split) {
  static std::atomic<int> known[kMaxDevices][4] = {};  // one more than the count; 0: not asked yet
  std::atomic<int>& mine = known[ctx.device][split == 8 ? 3 : split / 2];
  int have = mine.load(std::memory_order_relaxed);
  if (have > 0) return have - 1;
  const int smem = Ring<kCols, kSplit>::smem_bytes(
      split == 8 ? kMostGroupsOf8 : DSMEM_PRODUCT_MAX_GROUPS, split);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(split));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr = cluster_of(split);
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int count = 0;
  cudaError_t e = allow_smem<kKind, kCols, kSplit>(ctx.device, smem);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&count, product_kernel<kKind, kCols, kSplit>, &cfg);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return 0;  // whole tiles need no clusters
  }
  mine.store(count + 1, std::memory_order_relaxed);
  return count;
}

template <int kKind, int kCols>
int launch_narrow(const ProductArgs& p, const CallContext& ctx, const Source& x, const Source& w,
                  cudaStream_t stream) {
  const int64_t depth = kKind == kForward ? p.inner : (kKind == kInputGrad ? p.outer : p.n / p.groups);
  const int most = std::min(Ring<kCols, kSplit>::kMaxSplit, p.groups > kMostGroupsOf8 ? 4 : 8);
  const int split = split_for(tile_bound(p, kCols, kChannels), depth / kDepth, split_stages(kCols), most,
                              [&](int of) { return resident_clusters<kKind, kCols>(ctx, of); });
  if (split > 1) return launch<kKind, kCols, kSplit>(p, ctx, x, w, split, stream);
  return launch<kKind, kCols, kSolo>(p, ctx, x, w, 1, stream);
}

// Tiles about as wide as the average group, so that few columns are padding,
// and narrower where wide ones would not give every SM (pair of SMs) one.
// Forward, 64 groups of 2048 x 1024, us at this many rows a group:
//   16 / 64 wide    12: 47.3 / 47.7    24: 49.9 / 48.4
//   64 / 128 (pair) 64: 51.2 / 51.1    80: 57.2 / 52.3
//   128 / 256       128: 55.4 / 60.4   160: 69.9 / 62.4
//   4 groups of 512 rows by 1024 x 1024 (52 tiles 256 wide): 8.7 / 11.8;
//   by 2048 x 2048 (104): 18.4 / 17.6
//   4 groups of 512 rows by 1024 x 512 (42 pairs' tiles 128 wide), 64 / 128: 8.1 / 8.5,
//   by 1024 x 1024: 11.6 / 8.7
// 128 wide, pairs against single CTAs: 8.7 / 9.1 to 18.4 / 20.7; single ones
// are left for up to 128 channels.
template <int kKind>
int launch_rows(const ProductArgs& p, const CallContext& ctx, const Source& x, const Source& w,
                cudaStream_t stream) {
  const int64_t average = p.n / p.groups, pairs = ctx.sm_count / 2;
  const int channels = kKind == kInputGrad ? p.inner : p.outer;
  if (average <= 16) return launch_narrow<kKind, 16>(p, ctx, x, w, stream);
  if (average <= 64 || tile_bound(p, 128, 128) < pairs) return launch_narrow<kKind, 64>(p, ctx, x, w, stream);
  if (channels <= kChannels) return launch<kKind, 128, kSolo>(p, ctx, x, w, 1, stream);
  if (average > 128 && tile_bound(p, 256, 256) >= pairs) return launch<kKind, 256, kPair>(p, ctx, x, w, 1, stream);
  return launch<kKind, 128, kPair>(p, ctx, x, w, 1, stream);
}

// 256 x 256 tiles of pairs while there are half as many as pairs, 128 x 128
// ones while there are as many, else 128 x 64 with their depth split.  us,
// 256 / 128 / 64: 4 groups of 1024 rows, 1024 x 1024 (64 tiles of 256)
// 12.2 / 15.3 / 20.2; 7 of 333, 512 x 1024 (56) 8.7 / 9.7 / 10.8; 2 of 2048,
// 512 x 1024 (16; 64 tiles of 128) 15.3 / 13.8 / 11.8.
// A tile's whole depth is one unit's but for the split: 64 groups of 256 x 256
// over 131072 rows take 28.7 us where they are equal and 283 where one has half
// of the rows.
int launch_weight_grad(const ProductArgs& p, const CallContext& ctx, const Source& x, const Source& w,
                       cudaStream_t stream) {
  const int64_t pairs = ctx.sm_count / 2;
  if (p.outer > kChannels && 2 * tile_bound(p, 256, 256) >= pairs)
    return launch<kWeightGrad, 256, kPair>(p, ctx, x, w, 1, stream);
  if (tile_bound(p, 128, 128) >= pairs) return launch<kWeightGrad, 128, kSolo>(p, ctx, x, w, 1, stream);
  return launch_narrow<kWeightGrad, 64>(p, ctx, x, w, stream);
}

}  // namespace

int run_product(const ProductArgs& p, const CallContext& ctx, cudaStream_t stream) {
  Source x{p.x, p.x_stride, 0, p.x_rows, p.kind == kInputGrad ? p.outer : p.inner, 1, nullptr};
  Source w{p.w, p.w_stride, p.w_group_stride, p.outer, p.inner, p.groups, p.offsets};
  if (p.kind == kWeightGrad) w = Source{p.w, p.w_stride, 0, p.n, p.outer, 1, nullptr};
  Source* sources[2] = {&x, &w};
  void* scratch = nullptr;
  int rc = lay_out(ctx, sources, &scratch, stream);
  if (!rc) {
    if (p.kind == kForward) rc = launch_rows<kForward>(p, ctx, x, w, stream);
    else if (p.kind == kInputGrad) rc = launch_rows<kInputGrad>(p, ctx, x, w, stream);
    else rc = launch_weight_grad(p, ctx, x, w, stream);
  }
  if (scratch) {
    const int freed = pool_free(scratch, stream);
    if (!rc) rc = freed;
  }
  return rc;
}

cudaError_t read_and_clear_product_status(uint32_t* out) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_product_status, sizeof(uint32_t));
  if (e != cudaSuccess) return e;
  const uint32_t zero = 0;
  return *out ? cudaMemcpyToSymbol(g_product_status, &zero, sizeof(uint32_t)) : cudaSuccess;
}

}  // namespace dsmh
