// Products of microscaled 4-bit rows and matrices grouped by key, on the
// block-scaled tcgen05 matrix instructions.
//
// D[rows, channels] = x W[g]^T: 128 rows high, kCols channels wide, so that a
// lane of the accumulators is a row of the output.  One persistent CTA per SM.
// Warp 0 copies the matrices' values by TMA (256 elements of depth a stage: 128
// bytes a row, swizzled), warp 1 issues the matrix instructions, warps 2..5 write
// finished accumulators out, the next eight copy the rows that the order names,
// 16 bytes a copy, and the last four bring both sides' scales, four stages at a
// time.  Scales are kept row by row, as quantisation writes them; shared memory
// has them in the order that tensor memory wants: chunks of 128 rows by 4 scales,
// row r at 16 (r % 32) + 4 (r / 32).
//
// 4-bit operands are multiplied so fast that a tile is bound by what it takes in:
// 128 x 256 tiles take in three quarters of the bytes of 128 x 128 ones.  Their
// sums fill half of tensor memory, beside the scales, so there is no second
// accumulator; the first stage of a tile is multiplied by halves instead, each
// of which begins when the last tile's half has been written out.
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
constexpr int kShifts = 2;        // groups of copying warps that take stages in turn
constexpr int kShift = 128;       // threads of one
constexpr int kFirstCopy = 6;     // TMA, matrix instructions, 4 warps of output
constexpr int kRelayWarp = kFirstCopy + kShifts * kShift / 32;
constexpr int kFirstScale = kRelayWarp + 1;
constexpr int kScaleThreads = 128;
constexpr int kThreads = kFirstScale * 32 + kScaleThreads;
constexpr int kLine = 64;               // bytes of an output row that a warp writes at a time
constexpr int kStageOut = 32 * kLine;   // output staging of a warp
constexpr int kBarrierBytes = 320;
constexpr int kChunk = 512;             // scales of 128 rows by 128 elements
constexpr int kBlock = 4;               // stages whose scales are brought together

template <int kCols>
struct Ring {
  static constexpr int kA = kHigh * kStageBytes, kB = kCols * kStageBytes;
  static constexpr int kStage = kA + kB;
  static constexpr int kMostStages = kCols == 256 ? 4 : 8;
  static constexpr int kChunksB = (kCols + 127) / 128;             // of 128 elements' scales
  static constexpr int kScales = 2 * kBlock * (1 + kChunksB) * kChunk;  // of a block
  // Tensor memory: the sums of one tile in two halves, or of two tiles, then each
  // stage's scales.
  static constexpr int kBuffers = kCols == 256 ? 1 : 2, kHalves = kCols == 256 ? 2 : 1;
  static constexpr int kScaleColumns = 8 * (1 + kChunksB);
  static constexpr uint32_t kColumns = 512;
  static_assert(kBuffers * kCols + kMostStages * kScaleColumns <= 512, "tensor memory");
  static int smem_bytes(int groups, int stages) {
    return 1024 + stages * kStage + 2 * kScales + 4 * kStageOut + kBarrierBytes + 2 * 4 * (groups + 2);
  }
  // As many stages as fit.
  static int stages(int groups) {
    int n = kMostStages;
    while (smem_bytes(groups, n) > 227 * 1024) --n;
    return n;
  }
};

struct Args {
  const int32_t* offsets;
  const int32_t* order;
  int64_t n;
  int x_rows, groups, outer, quads, stages;
  Divisor fan, by_chan_tiles;
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
  Divisor by_chan_tiles;
  int groups, chan_tiles, blocks, group;
  __device__ __forceinline__ Schedule(const int32_t* b, const int32_t* f, const Args& a)
      : begin(b), first(f), by_chan_tiles(a.by_chan_tiles), groups(a.groups),
        chan_tiles((a.outer + kCols - 1) / kCols), blocks((a.quads + 1) / 2), group(0) {}
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
    const int i = t - first[group], across = by_chan_tiles.quotient(i);
    Tile r;
    r.group = group;
    r.row0 = begin[group] + across * kHigh;
    r.end = begin[group + 1];
    r.chan0 = (i - across * chan_tiles) * kCols;
    r.blocks = group < groups ? blocks : 0;
    return r;
  }
};

// Descriptor of a chunk of scales: not swizzled, groups of 8 rows of 16 bytes.
__device__ __forceinline__ uint64_t scale_descriptor(uint32_t addr) {
  return (uint64_t{1} << 46) | (uint64_t{128 >> 4} << 32) | ((addr & 0x3ffffu) >> 4);
}

// kN columns of a warp's 32 rows, through its staging memory: 16-byte pieces of
// a row, exchanged so that neighbouring rows meet other banks.
template <int kN, typename O>
__device__ __forceinline__ void store_columns(const Args& a, int row0, int end, int chan, const uint32_t (&r)[kN],
                                              uint32_t staging) {
  const int lane = threadIdx.x & 31;
  constexpr int V = 16 / sizeof(O), kPieces = kN / V;
  const auto piece_at = [&](int row, int q) {
    return staging + row * (kN * sizeof(O)) + ((q ^ (row * kPieces / 8 & (kPieces - 1))) << 4);
  };
#pragma unroll
  for (int q = 0; q < kPieces; ++q) {
    Pack<O, V> p;
#pragma unroll
    for (int v = 0; v < V; ++v) p.v[v] = from_float<O>(__uint_as_float(r[q * V + v]));
    st_shared_16(piece_at(lane, q), p);
  }
  __syncwarp();
  O* out = static_cast<O*>(a.out) + static_cast<int64_t>(row0) * a.outer + chan;
  const int rows = min(32, end - row0);
  if (a.wide_out) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int row = (i * 32 + lane) / kPieces, q = lane & (kPieces - 1);
      const uint4 p = ld_shared_16(piece_at(row, q));
      if (row < rows && chan + q * V < a.outer)
        *reinterpret_cast<uint4*>(out + static_cast<int64_t>(row) * a.outer + q * V) = p;
    }
  } else {
    for (int row = 0; row < rows; ++row, out += a.outer)
#pragma unroll
      for (int j = lane; j < kN; j += 32)
        if (chan + j < a.outer) out[j] = ld_shared_value<O>(piece_at(row, j / V) + j % V * sizeof(O));
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
      for (int c = lane; c < cols; c += 32) out[c] = from_float<O>(0.0f);
    }
  }
}

// A warp's 32 rows of a tile's columns [first, last) from tensor memory to the output.
template <typename O>
__device__ __forceinline__ void store_tile(const Args& a, const Tile& t, int row0, int first, int last, uint32_t tmem,
                                           uint32_t staging) {
  constexpr int kN = kLine / static_cast<int>(sizeof(O));
#pragma unroll 1
  for (int c = first; c < last && t.chan0 + c < a.outer; c += kN) {
    uint32_t r[kN];
    if constexpr (kN == 32) tmem_load32(tmem + c, r);
    else tmem_load16(tmem + c, r);
    tmem_wait_load();
    store_columns<kN, O>(a, row0, t.end, t.chan0 + c, r, staging);
  }
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

// The copying warps.  A thread copies one of the eight pieces of every 16th row.
// Rows at and behind the tile's end are left as they are: what they hold reaches
// no other row.  Each thread's copies of a stage arrive on `landed` by themselves;
// the relay warp passes a landed stage on.
template <int kCols>
__device__ __forceinline__ void copy_rows(const Args& a, Schedule<kCols>& schedule, int total, uint32_t base,
                                          uint32_t landed, uint32_t empty, uint32_t gave_up) {
  using R = Ring<kCols>;
  constexpr int kRows = kHigh * 8 / kShift, kLines = kShift / 8;
  const int shift = (threadIdx.x - kFirstCopy * 32) / kShift, tid = (threadIdx.x - kFirstCopy * 32) % kShift;
  const int64_t pitch = int64_t{64} * a.quads;
  // A tile's entries of the order are asked for while the tile before is copied.
  int ahead[kRows];
  const auto ask = [&](const Tile& t) {
#pragma unroll
    for (int r = 0; r < kRows; ++r) ahead[r] = place_at(a, t.row0 + r * kLines + tid / 8, t.end);
  };
  int stage = shift, skip = shift;  // skip: stages until this shift's next
  uint32_t phase = 0;
  bool ok = true;
  Tile next;
  int i = blockIdx.x;
  if (i < total) {
    next = schedule.at(i);
    ask(next);
  }
  while (i < total && ok) {
    const Tile t = next;
    int row[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) row[r] = row_named(a, ahead[r]);
    i += gridDim.x;
    if (i < total) {
      next = schedule.at(i);
      ask(next);
    }
    int k = skip;
    for (; k < t.blocks; k += kShifts) {
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
          copy16(sa + line * 128 + ((c ^ (line & 7)) << 4), a.x_values + (read ? row[r] * pitch + at : 0), read ? 16 : 0);
      }
      copy_arrive(landed + 8 * stage);
      stage += kShifts;
      if (stage >= a.stages) {
        stage -= a.stages;
        phase ^= 1;
      }
    }
    skip = k - t.blocks;
  }
  copy_wait_all();
}

// Eight times four scales (of a block's 1024 elements) of a row, from element
// 1024 * block on, to their chunks; zeros behind the row's end, and for no row.
__device__ __forceinline__ void put_scales(uint32_t chunks, int apart, int line, const uint8_t* row, int block,
                                           const Args& a) {
  uint32_t s[2 * kBlock];
  const int first = block * 2 * kBlock;
  if (row && a.wide_scales && first + 2 * kBlock <= a.quads) {
#pragma unroll
    for (int q = 0; q < 2 * kBlock; q += 4) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(row + (first + q) * 4));
      s[q] = v.x, s[q + 1] = v.y, s[q + 2] = v.z, s[q + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int q = 0; q < 2 * kBlock; ++q)
      s[q] = row && first + q < a.quads ? __ldg(reinterpret_cast<const uint32_t*>(row) + first + q) : 0u;
  }
  const uint32_t to = chunks + (line & 31) * 16 + (line >> 5 & 3) * 4 + (line >> 7) * kChunk;
#pragma unroll
  for (int q = 0; q < 2 * kBlock; ++q) st_shared_u32(to + q * apart, s[q]);
}

// The scales' warps: a thread brings one row's of x, and kCols / 128 channels' (or
// one's, of the first kCols).
template <int kCols>
__device__ __forceinline__ void bring_scales(const Args& a, Schedule<kCols>& schedule, int of_groups, uint32_t scales,
                                             uint32_t full, uint32_t empty, uint32_t gave_up) {
  using R = Ring<kCols>;
  const int tid = threadIdx.x - kFirstScale * 32;
  const int64_t pitch = int64_t{4} * a.quads;
  uint32_t buffer = 0, phase = 0;
  bool ok = true;
  for (int i = blockIdx.x; i < of_groups && ok; i += gridDim.x) {
    const Tile t = schedule.at(i);
    const int row = row_named(a, place_at(a, t.row0 + tid, t.end));
    const uint8_t* x = row >= 0 ? a.x_scales + row * pitch : nullptr;
    for (int b = 0; b * kBlock < t.blocks; ++b) {
      ok = wait_for(empty + 8 * buffer, phase ^ 1, gave_up, a.wait_cycles, a.status);
      ok = __all_sync(kFull, ok);
      if (!ok) break;
      const uint32_t to = scales + buffer * R::kScales;
      put_scales(to, kChunk, tid, x, b, a);
#pragma unroll
      for (int c = 0; c < kCols; c += kScaleThreads) {
        const int channel = t.chan0 + c + tid;
        if (c + tid < kCols)
          put_scales(to + 2 * kBlock * kChunk, R::kChunksB * kChunk, c + tid,
                     channel < a.outer ? a.w_scales + (static_cast<int64_t>(t.group) * a.outer + channel) * pitch : nullptr,
                     b, a);
      }
      fence_async_shared();
      mbar_arrive_local(full + 8 * buffer);
      if (++buffer == 2) {
        buffer = 0;
        phase ^= 1;
      }
    }
  }
}

template <int kCols>
__global__ void __launch_bounds__(kThreads, 1)
    mx4_product_kernel(const __grid_constant__ CUtensorMap weights, const __grid_constant__ Args a) {
  using R = Ring<kCols>;
  constexpr int kStage = R::kStage;
  const int kStages = a.stages;
  extern __shared__ uint8_t raw[];
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  uint8_t* base_ptr = raw + (base - smem_u32(raw));
  const uint32_t scales = base + kStages * kStage, out_staging = scales + 2 * R::kScales;
  const uint32_t bars = out_staging + 4 * kStageOut;
  const uint32_t full = bars, empty = full + 8 * R::kMostStages, landed = empty + 8 * R::kMostStages;
  const uint32_t acc_full = landed + 8 * R::kMostStages, acc_empty = acc_full + 16, scales_full = acc_empty + 16;
  const uint32_t scales_empty = scales_full + 16, drained = scales_empty + 16;
  const uint32_t tmem_at = drained + 8, gave_up = tmem_at + 4;
  static_assert(8 * (3 * R::kMostStages + 9) + 8 <= kBarrierBytes, "barriers");
  int32_t* begin = reinterpret_cast<int32_t*>(base_ptr + (bars - base) + kBarrierBytes);
  int32_t* first = begin + a.groups + 2;

  const int warp = __shfl_sync(kFull, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  Schedule<kCols> schedule(begin, first, a);
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full + 8 * s, 2);  // the TMA thread and the relay
      mbar_init(landed + 8 * s, kShift);
      mbar_init(empty + 8 * s, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full + 8 * i, 1);
      mbar_init(acc_empty + 8 * i, 4);
      mbar_init(scales_full + 8 * i, kScaleThreads);
      mbar_init(scales_empty + 8 * i, 1);
    }
    mbar_init(drained, 1);
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(gave_up), "r"(0u) : "memory");
    fence_mbar_init();
    prefetch_map(&weights);
  }
  lay_groups<kThreads>(a.offsets, a.n, a.groups, a.groups + 1, begin, first,
                       [&](int rows) { return schedule.tiles_of(rows); },
                       [&] { if (warp == 1) tmem_alloc<false>(tmem_at, R::kColumns); });
  tcgen_fence_before();
  __syncthreads();
  tcgen_fence_after();
  uint32_t tmem;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(tmem_at));
  const int total = first[a.groups + 1], step = gridDim.x;
  const int of_groups = first[a.groups];  // tiles of real groups

  if (warp == 0) {
    uint32_t stage = 0, phase = 0, issued = 0;
    bool ok = true;
    for (int i = blockIdx.x; i < total && ok; i += step) {
      const Tile t = schedule.at(i);
      for (int k = 0; k < t.blocks; ++k) {
        ok = __all_sync(kFull, wait_for(empty + 8 * stage, phase ^ 1, gave_up, a.wait_cycles, a.status));
        if (!ok || (a.withhold && i + step >= of_groups && k + 1 == t.blocks)) break;
        if (elect_one()) {
          mbar_expect_tx(full + 8 * stage, R::kB);
          tma_load_3d<false>(base + stage * kStage + R::kA, &weights, k * kStageBytes, t.chan0, t.group,
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
  } else if (warp == kRelayWarp) {
    // Copied stages, once landed, on to the matrix instructions.
    if (lane == 0) {
      uint32_t stage = 0, phase = 0;
      bool ok = true;
      for (int i = blockIdx.x; i < of_groups && ok; i += step) {
        for (int k = 0; k < schedule.blocks; ++k) {
          ok = wait_for(landed + 8 * stage, phase, gave_up, a.wait_cycles, a.status);
          if (!ok) break;
          fence_async_shared();
          mbar_arrive_local(full + 8 * stage);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
    }
    __syncwarp();
  } else if (warp >= kFirstScale) {
    bring_scales<kCols>(a, schedule, of_groups, scales, scales_full, scales_empty, gave_up);
  } else if (warp >= kFirstCopy) {
    copy_rows<kCols>(a, schedule, of_groups, base, landed, empty, gave_up);
  } else if (warp == 1) {
    // A and B e2m1, K-major, scales e8m0.  Bits 4 and 29 choose the first or the
    // third of a row's four scales, of which an instruction takes two.
    constexpr int kHalf = kCols / R::kHalves;
    constexpr uint32_t kDesc = (1u << 7) | (1u << 10) | (1u << 23) | (uint32_t{kHigh >> 7} << 27);
    constexpr uint32_t kWhole = kDesc | (uint32_t{kCols >> 3} << 17), kPart = kDesc | (uint32_t{kHalf >> 3} << 17);
    constexpr uint32_t kSecond = (2u << 4) | (2u << 29);
    uint32_t stage = 0, phase = 0, done = 0, buffer = 0, scale_phase = 0;
    bool ok = true;
    const auto await = [&](uint32_t bar, uint32_t parity) {
      ok = __all_sync(kFull, wait_for(bar, parity, gave_up, a.wait_cycles, a.status));
      tcgen_fence_after();
      return ok;
    };
    for (int i = blockIdx.x; i < of_groups && ok; i += step) {
      // Sums: a tile's own place of two, or the halves of the only one.
      const uint32_t place = R::kBuffers == 2 ? done & 1 : 0, d = tmem + place * kCols;
      const uint32_t turn = R::kBuffers == 2 ? done >> 1 & 1 : done & 1;
      if (!await(acc_empty + 8 * place, turn ^ 1)) break;
      for (int k = 0; k < schedule.blocks; ++k) {
        if (k % kBlock == 0 && !await(scales_full + 8 * buffer, scale_phase)) break;
        if (!await(full + 8 * stage, phase)) break;
        const uint32_t sa = base + stage * kStage;
        const uint64_t da = descriptor<false>(sa), db = descriptor<false>(sa + R::kA);
        const uint32_t chunks = scales + buffer * R::kScales + k % kBlock * 2 * kChunk;
        const uint64_t dsa = scale_descriptor(chunks);
        const uint64_t dsb = scale_descriptor(chunks + 2 * kBlock * kChunk + k % kBlock * 2 * (R::kChunksB - 1) * kChunk);
        // Each stage has columns of its own: the stage is handed back only when
        // the instructions that read them have completed.
        const uint32_t sfa = tmem + R::kBuffers * kCols + stage * R::kScaleColumns, sfb = sfa + 8;
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
            copy_scales(sfa + 4 * q, dsa + q * (kChunk >> 4));
#pragma unroll
            for (int c = 0; c < R::kChunksB; ++c)
              copy_scales(sfb + 4 * (R::kChunksB * q + c), dsb + (R::kChunksB * q + c) * (kChunk >> 4));
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
          if (last || k % kBlock == kBlock - 1) mma_commit<false>(scales_empty + 8 * buffer);
          if (last) mma_commit<false>(acc_full + 8 * place);
        }
        __syncwarp();
        if (last || k % kBlock == kBlock - 1) {
          buffer ^= 1;
          scale_phase ^= buffer == 0;
        }
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
    const int quadrant = warp & 3;
    const uint32_t staging = out_staging + quadrant * kStageOut;
    uint32_t done = 0;
    for (int i = blockIdx.x; i < total; i += step) {
      const Tile t = schedule.at(i);
      const int row0 = t.row0 + quadrant * 32;
      if (t.blocks == 0) {
        if (a.out_dtype == DSMEM_F32) store_zeros<kCols, float>(a, row0, t.end, t.chan0);
        else store_zeros<kCols, __half>(a, row0, t.end, t.chan0);
        continue;
      }
      const uint32_t place = R::kBuffers == 2 ? done & 1 : 0;
      const uint32_t turn = R::kBuffers == 2 ? done >> 1 & 1 : done & 1;
      // A long contraction may take longer than one bounded wait of a copy.
      const bool ok = wait_for(acc_full + 8 * place, turn, gave_up, a.wait_cycles + 4096ll * t.blocks, a.status);
      if (!__all_sync(kFull, ok)) break;
      tcgen_fence_after();
      const uint32_t d = tmem + place * kCols + (static_cast<uint32_t>(quadrant * 32) << 16);
#pragma unroll 1
      for (int half = 0; half < R::kHalves; ++half) {
        constexpr int kHalf = kCols / R::kHalves;
        const int from = half * kHalf, to = from + kHalf;
        if (row0 < t.end) {
          if (a.out_dtype == DSMEM_F32) store_tile<float>(a, t, row0, from, to, d, staging);
          else if (a.out_dtype == DSMEM_F16) store_tile<__half>(a, t, row0, from, to, d, staging);
          else store_tile<__nv_bfloat16>(a, t, row0, from, to, d, staging);
        }
        tcgen_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_local(acc_empty + 8 * (R::kHalves == 2 ? half : place));
      }
      ++done;
    }
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
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(p.w_values), dims, strides, box,
                            unit, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail_with(DSMEM_HIST_ECUDA, "cuTensorMapEncodeTiled: error %d (4-bit matrices, %d x %d x %d)",
                     static_cast<int>(r), p.groups, p.outer, p.quads * 128);
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
  a.by_chan_tiles = Divisor(static_cast<uint32_t>((p.outer + kCols - 1) / kCols));
  a.x_values = p.x_values, a.x_scales = p.x_scales, a.w_scales = p.w_scales;
  a.out = p.out, a.out_dtype = p.out_dtype;
  a.wide_out = reinterpret_cast<uintptr_t>(p.out) % 16 == 0 &&
               static_cast<int64_t>(p.outer) * dtype_size(p.out_dtype) % 16 == 0;
  a.wide_scales = p.quads % 4 == 0 && reinterpret_cast<uintptr_t>(p.x_scales) % 16 == 0 &&
                  reinterpret_cast<uintptr_t>(p.w_scales) % 16 == 0;
  a.status = ctx.status;
  a.wait_cycles = call_wait_cycles();
  a.withhold = call_withholds();
  CUtensorMap map;
  const int rc = make_map(&map, p, kCols);
  if (rc) return rc;
  const int64_t tiles = tile_bound(p, kCols);
  if (tiles > INT32_MAX - 1024)  // tile counters step past the last tile
    return fail_with(DSMEM_HIST_EINVAL, "4-bit grouped product: more than 2^31 output tiles");
  a.stages = Ring<kCols>::stages(p.groups);
  const int smem = Ring<kCols>::smem_bytes(p.groups, a.stages);
  const auto kernel = mx4_product_kernel<kCols>;
  cudaError_t e = limit.need(reinterpret_cast<const void*>(kernel), ctx.device, smem);
  if (e != cudaSuccess) return fail_with_cuda(e, "cudaFuncSetAttribute");
  kernel<<<static_cast<unsigned>(std::min<int64_t>(tiles, ctx.sm_count)), kThreads, smem, stream>>>(map, a);
  e = cudaGetLastError();
  return e == cudaSuccess ? DSMEM_HIST_OK : fail_with_cuda(e, "4-bit grouped product launch");
}

}  // namespace

// Narrow tiles where wide ones would not give every SM one.
int run_mx4_product(const Mx4ProductArgs& p, const CallContext& ctx, cudaStream_t stream) {
  if (tile_bound(p, 128) < ctx.sm_count) return launch<32>(p, ctx, stream);
  if (tile_bound(p, 256) < 2 * ctx.sm_count) return launch<128>(p, ctx, stream);
  return launch<256>(p, ctx, stream);
}

cudaError_t read_and_clear_mx4_status(uint32_t* out) { return take_product_status(out); }

}  // namespace dsmh
