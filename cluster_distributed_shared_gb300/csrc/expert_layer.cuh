// A whole expert layer for a few tokens, in two kernels (f16 matrices: three).
//
// With e = ids[t, j] and w = weights[t, j] of a token's routing,
//   up kernel    h[t, j] = w act(up[e] x[t]),  or  w act(gate[e] x[t]) * (up[e] x[t])
//   down kernel  y[t]    = sum over j of down[e] h[t, j]
// and between them, beside f16 matrices, a scale of each row of h.
// A few tokens do little arithmetic on many weights, so both kernels are bound
// by reading the chosen experts' matrices once, and everything follows from
// keeping loads of them in flight:
//   * Rows of the matrices go from global memory straight to the registers of
//     mma.sync fragments, kSteps steps ahead.  The depth may be summed in any
//     order, so lane (g, t) = (lane / 4, lane % 4) takes 16 consecutive bytes of
//     rows g and g + 8 and the same elements of the rows' side: no shared memory,
//     no exchange between lanes, one load for two (16-bit) or eight (4-bit)
//     instructions.  (A tcgen05 tile would be 128 rows high, of which one token's
//     share of an SM fills 27, and would pass every byte through shared memory.  A
//     batch of 32 fills it; tiles for those have not been tried.)
//   * Every SM reads the same number of rows, every warp the same number of
//     batches of kSteps steps.
//   * Each CTA of the up kernel routes all tokens for itself instead of waiting for
//     a launch that does, and the first passes the routing on.  The down kernel is
//     launched while the up kernel runs (programmatic dependent launch), so that
//     its CTAs wait where the up kernel's leave.
//   * Code that runs once costs about 10 cycles an instruction, for its fetch:
//     hence loops where unrolled code would do less work.
// Sums are 32-bit: in the fragments along a warp's part of the depth, then over
// the warps through shared memory in their order.  Nothing is added atomically.
//
// Measured with 128 experts of 2048 x 1024, 8 a token, gated, 32 tokens (210 us of
// reading): 16-bit 229 us, 6.1 TB/s; 4-bit 179 us, bound by instructions (17 for 8
// elements of decoding, 280 a step in all; 55% of issue slots and of the logic pipe).
// One token, 4 experts: 20.5 and 18.9 us, of which 7.5 and 2 are reading, the rest
// launches, routing and first touches of code.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "divisor.h"
#include "dtypes.cuh"
#include "experts.h"
#include "mx4.cuh"
#include "ptx.cuh"
#include "route.cuh"

namespace dsmh {
namespace {

constexpr int kMaxTokens = DSMEM_LAYER_MAX_TOKENS;
constexpr int kMaxRows = kMaxTokens * DSMEM_ROUTE_MAX_TOP_K;
// How the matrices are held, and with them the type of the fragments: 16-bit
// matrices have x's type; 4-bit ones become bf16, which holds every value they
// stand for exactly.
enum Held { kBf16, kF16, kMx4Bf16, kMx4F16 };
template <int kHeld>
constexpr bool kIsMx4 = kHeld == kMx4Bf16 || kHeld == kMx4F16;
// Warps of a CTA: as many as 128 registers a thread allow.  (With 8 a CTA, and both
// kernels' CTAs on an SM together, 4 tokens of 64 experts of 2048 x 768, 4 a token,
// took 40.0 us, not 34.9, and 1 token 19.1, not 18.8.)
constexpr int kWarps = 16;
// Steps of depth that a warp has in flight, a batch: as registers allow.  (16-bit: 2
// instead of 4 took 108 us, not 97, at 32 tokens of 64 experts of 2048 x 768.  4-bit,
// whose decoding hides a load's way: 2 instead of 1 took 184 us, not 179, in the case
// above; with four column tiles its down kernel spills 88 bytes, not 32, and the up
// kernel of f16 tokens 70, not none.)
template <int kHeld>
constexpr int kSteps = kIsMx4<kHeld> ? 1 : 4;
template <int kHeld>
constexpr int kDepth = kIsMx4<kHeld> ? 128 : 32;  // elements of a step

// Everything a CTA knows about the routing.  Rows are (token, expert) pairs,
// expert after expert, an expert's rows by token.
struct alignas(32) Routing {
  unsigned long long tokens_of[DSMEM_ROUTE_MAX_EXPERTS];  // a bit for each token
  uint16_t place_of[DSMEM_ROUTE_MAX_EXPERTS];             // among the active experts
  uint16_t active[DSMEM_ROUTE_MAX_EXPERTS];               // experts that any token chose, by number
  uint16_t start[DSMEM_ROUTE_MAX_EXPERTS];                // of active experts: first row
  uint16_t rows_of[DSMEM_ROUTE_MAX_EXPERTS];              // of active experts
  float weight[kMaxRows];                                 // of each row; behind scale_kernel, the row's scale
  uint8_t token[kMaxRows];
  uint32_t of_warp[16];
  int count;  // of active experts
};

// What a token's warp hands from its choices to its rows.
struct Choice {
  float weight;
  int id;
};

// The choices of two tokens, `between` apart (the second may lie behind the last),
// by one warp, the j-th in lane j, as in routing.
template <int R>
__device__ __forceinline__ void choose(const LayerArgs& a, int token, int between, Choice (&choice)[2]) {
  const int first = (threadIdx.x & 31) * R;
  uint32_t key[2][R];
  float v[2][R];
  const auto load = [&](auto* logits) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int r = 0; r < R; ++r)
        v[i][r] = first + r < a.experts && token + i * between < a.tokens
                      ? to_float(logits[(token + i * between) * a.logits_stride + first + r])
                      : -INFINITY;
  };
  if (a.logits_dtype == DSMEM_F32) load(static_cast<const float*>(a.logits));
  else if (a.logits_dtype == DSMEM_F16) load(static_cast<const __half*>(a.logits));
  else load(static_cast<const __nv_bfloat16*>(a.logits));
  Best best[2];
  float top[2], all[2] = {};
  int id[2] = {-1, -1};
  uint32_t chosen[2] = {};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int r = 0; r < R; ++r) key[i][r] = rank_key(v[i][r]);
    best[i] = two_best(key[i], 0u);
    top[i] = rank_value(__reduce_max_sync(kFullWarp, best[i].key));
    if (!a.renormalize) {
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (key[i][r]) all[i] += raised(rank_value(key[i][r]), top[i]);
    }
  }
  pick(key, best, a.top_k, id, chosen);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float mine = id[i] >= 0 ? raised(rank_value(chosen[i]), top[i]) : 0.0f;
    const float sum = warp_sum(a.renormalize ? mine : all[i]);
    choice[i] = Choice{id[i] >= 0 ? mine / sum : 0.0f, id[i]};
  }
}

// Fills `r` and returns the number of active experts; all threads of the CTA.
// choices: shared memory for tokens * top_k of them.
__device__ __forceinline__ int route_all(const LayerArgs& a, Routing& r, Choice* choices) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kEach = DSMEM_ROUTE_MAX_EXPERTS / (kWarps * 32);  // experts of a lane
  for (int e = threadIdx.x; e < a.experts; e += kWarps * 32) r.tokens_of[e] = 0ull;
  __syncthreads();
#pragma unroll 1
  for (int token = warp; token < a.tokens; token += 2 * kWarps) {
    Choice c[2];
    if (a.experts <= 64) choose<2>(a, token, kWarps, c);
    else if (a.experts <= 128) choose<4>(a, token, kWarps, c);
    else if (a.experts <= 256) choose<8>(a, token, kWarps, c);
    else choose<DSMEM_ROUTE_MAX_EXPERTS / 32>(a, token, kWarps, c);
    if (lane < a.top_k) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int of = token + i * kWarps;
        if (of >= a.tokens) break;
        choices[of * a.top_k + lane] = c[i];
        if (c[i].id >= 0) atomicOr(&r.tokens_of[c[i].id], 1ull << of);
      }
    }
  }
  __syncthreads();
  // Places among the active experts in the upper half of a word, rows in the lower.
  const int first = (warp * 32 + lane) * kEach;
  uint32_t mine = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int rows = first + i < a.experts ? __popcll(r.tokens_of[first + i]) : 0;
    mine += rows + ((rows > 0) << 16);
  }
  uint32_t before = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t up = __shfl_up_sync(kFullWarp, before, d);
    if (lane >= d) before += up;
  }
  if (lane == 31) r.of_warp[warp] = before;
  __syncthreads();
  const uint32_t other = lane < kWarps ? r.of_warp[lane] : 0u;
  before += __reduce_add_sync(kFullWarp, lane < warp ? other : 0u) - mine;
  const int count = static_cast<int>(__reduce_add_sync(kFullWarp, other) >> 16);
  if (threadIdx.x == 0) r.count = count;
  if (mine > 0) {
    int place = static_cast<int>(before >> 16), row = static_cast<int>(before & 0xffffu);
#pragma unroll 1
    for (int e = first; e < min(first + kEach, a.experts); ++e) {
      const int rows = __popcll(r.tokens_of[e]);
      if (rows == 0) continue;
      r.place_of[e] = static_cast<uint16_t>(place);
      r.active[place] = static_cast<uint16_t>(e);
      r.start[place] = static_cast<uint16_t>(row);
      r.rows_of[place] = static_cast<uint16_t>(rows);
      ++place;
      row += rows;
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int token = warp; token < a.tokens; token += kWarps) {
    const Choice c = lane < a.top_k ? choices[token * a.top_k + lane] : Choice{0.0f, -1};
    if (c.id < 0) continue;
    const int to = r.start[r.place_of[c.id]] + __popcll(r.tokens_of[c.id] & ((1ull << token) - 1ull));
    r.token[to] = static_cast<uint8_t>(token);
    r.weight[to] = c.weight;
  }
  __syncthreads();
  return count;
}

// The routing to the down kernel and there, by all threads.
__device__ __forceinline__ void pass_on(void* to, const Routing& r) {
  static_assert(sizeof(Routing) % 16 == 0, "whole vectors");
  for (int i = threadIdx.x; i < static_cast<int>(sizeof(Routing) / 16); i += blockDim.x)
    static_cast<uint4*>(to)[i] = reinterpret_cast<const uint4*>(&r)[i];
}
__device__ __forceinline__ void take_over(Routing& r, const void* from) {
  for (int i = threadIdx.x; i < static_cast<int>(sizeof(Routing) / 16); i += blockDim.x)
    reinterpret_cast<uint4*>(&r)[i] = __ldcg(static_cast<const uint4*>(from) + i);
  __syncthreads();
}

// ------------------------------------------------------------ fragments

template <int kHeld>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1) {
  if constexpr (kHeld == kF16) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  } else {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
}

// Weights pass by once.  Volatile, so that the loads stay where they are
// issued, kSteps ahead of their use.
__device__ __forceinline__ uint4 load_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Eight elements of the rows' side as fragments' words: pairs in the order of
// the matrices', and for values that one 16-bit number does not hold a second
// one, the rest.
struct Eight {
  uint32_t high[4], low[4];
};

// A lane's part of a step: 16 bytes of two rows; for 4-bit elements (32 of them,
// one block) their scales, else its part of the first column tile too.
struct Slot {
  uint4 row[2];
  uint32_t scale[2];
  Eight column;
};

// Where a lane's part of the next batch of steps lies: in two rows of a matrix,
// and in its row of the first column tile.
struct Ahead {
  const uint8_t* row[2];
  const uint8_t* scale[2];
  const uint16_t* column;
};

// Row `row` of expert `e`, at the batch that begins with step `step`.
template <int kHeld>
__device__ __forceinline__ void point_at(const LayerMatrix& m, int e, int row, int step, Ahead& to, int i) {
  const int t = threadIdx.x & 3;
  const int64_t size = kIsMx4<kHeld> ? 1 : 2;
  to.row[i] = static_cast<const uint8_t*>(m.values) + (e * m.group_stride + row * m.row_stride) * size + step * 64 +
              t * 16;
  if (kIsMx4<kHeld>)
    to.scale[i] = m.scales + (static_cast<int64_t>(e) * m.rows + row) * m.scale_stride + step * 4 + t;
}
// On to the next batch of the same rows.
template <int kHeld, typename From>
__device__ __forceinline__ void move_on(Ahead& at) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    at.row[i] += kSteps<kHeld> * 64;
    if (kIsMx4<kHeld>) at.scale[i] += kSteps<kHeld> * 4;
  }
  if (!kIsMx4<kHeld>) at.column += kSteps<kHeld> * From::kStep;
}

// The part of a matrix's rows that a batch takes.
struct Batch {
  int step;    // its first step
  bool whole;  // all of its steps lie inside the rows
};

// Step d of a batch.  kWide: rows of 16-bit matrices begin at 16-byte boundaries
// and are whole vectors.  (4-bit rows always do and are.)
template <int kHeld, bool kWide>
__device__ __forceinline__ void load_rows(Slot& s, const Ahead& at, int d, const Batch& b, int steps, int depth) {
  if (!b.whole && b.step + d >= steps) return;
  if constexpr (kIsMx4<kHeld>) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      s.row[i] = load_once(at.row[i] + d * 64);
      s.scale[i] = __ldg(at.scale[i] + d * 4);
    }
  } else if (kWide && b.whole) {
#pragma unroll
    for (int i = 0; i < 2; ++i) s.row[i] = load_once(at.row[i] + d * 64);
  } else {
    const int t = threadIdx.x & 3, c = (b.step + d) * 32 + t * 8;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      s.row[i] = make_uint4(0, 0, 0, 0);
      if constexpr (kWide) {
        if (c < depth) s.row[i] = load_once(at.row[i] + d * 64);
      } else {
        const uint16_t* row = reinterpret_cast<const uint16_t*>(at.row[i] + d * 64) - c;
        s.row[i] = aligned_piece(row, c, depth, (reinterpret_cast<uintptr_t>(row) & 2u) != 0);
      }
    }
  }
}
template <int kHeld, typename From>
__device__ __forceinline__ void load_column(Slot& s, const Ahead& at, int d, const Batch& b, int steps,
                                            const From& from) {
  if (kIsMx4<kHeld> || (!b.whole && b.step + d >= steps)) return;
  from.fetch(at.column + d * From::kStep, (b.step + d) * 32 + (threadIdx.x & 3) * 8, s.column);
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) {
  return i == 0 ? v.x : (i == 1 ? v.y : (i == 2 ? v.z : v.w));
}

// Where the rows' side comes from.  at() is where a lane's piece q of eight
// elements of a step lies in its row (4-bit: of four, else the only one), and
// fetch() takes one, c of its row.  x: a token's
// vector, 16-bit, any alignment, read again and again.
template <int kHeld, bool kWide>
struct FromX {
  static constexpr bool kTwo = kHeld == kMx4F16;  // f16 is the sum of two bf16
  static constexpr int kStep = kDepth<kHeld>;
  const uint16_t* x;
  int64_t stride;
  int depth;
  __device__ __forceinline__ const uint16_t* row(int r) const { return x + r * stride; }
  __device__ __forceinline__ static int at(int step, int q) {
    return step * kStep + (threadIdx.x & 3) * (kStep / 4) + q * 8;
  }
  __device__ __forceinline__ void fetch(const uint16_t* p, int c, Eight& e) const {
    uint4 v = make_uint4(0, 0, 0, 0);
    if constexpr (kWide) {
      if (c < depth) v = __ldg(reinterpret_cast<const uint4*>(p));
    } else {
      v = aligned_piece(p - c, c, depth, (reinterpret_cast<uintptr_t>(p) & 2u) != 0);
    }
    if constexpr (kIsMx4<kHeld>) {
      const uint32_t w[4] = {__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                             __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632)};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        e.high[i] = w[i];
        if constexpr (kHeld == kMx4F16) {
          const float2 f = pair_to_floats(w[i], __half());
          e.high[i] = floats_to_pair(f, __nv_bfloat16());
          const float2 h = pair_to_floats(e.high[i], __nv_bfloat16());
          // An infinity's rest is 0, not inf - inf.
          e.low[i] = floats_to_pair(make_float2(isinf(h.x) ? 0.0f : f.x - h.x, isinf(h.y) ? 0.0f : f.y - h.y),
                                    __nv_bfloat16());
        }
      }
    } else {
      e.high[0] = v.x, e.high[1] = v.y, e.high[2] = v.z, e.high[3] = v.w;
    }
  }
};
// h: the up kernel's rows, each element as two numbers, with zeros up to whole
// steps; each row is read once by a CTA for every 16 of its channels.  A piece is
// eight first numbers and eight second ones, a sector, in the fragments' order, and
// the pieces that the four lanes of a row take together lie side by side.
template <int kHeld>
struct FromH {
  static constexpr bool kTwo = true;
  static constexpr int kStep = 2 * kDepth<kHeld>;
  const uint16_t* h;
  int pitch;  // elements of a row
  __device__ __forceinline__ const uint16_t* row(int r) const { return h + static_cast<int64_t>(r) * 2 * pitch; }
  __device__ __forceinline__ static int at(int step, int q) {
    return step * kStep + (q * 4 + (threadIdx.x & 3)) * 16;
  }
  // Element c of a row.  Two bf16 numbers hold 16 bits of it, whatever its size.  Two
  // f16 numbers would hold less below 2^-9 and nothing below 2^-25 or above 65504,
  // which a small x or a small routing weight passes, so that beside f16 matrices a
  // piece is at first eight floats, and scale_kernel makes the numbers of them.
  __device__ __forceinline__ static void put(uint16_t* row, int c, float value) {
    if constexpr (kHeld == kF16) {
      reinterpret_cast<float*>(row)[c] = value;
    } else {
      // Where the first number lies; the second is 8 further on.
      uint16_t* to = row + (kIsMx4<kHeld> ? (c >> 7) * kStep + ((c >> 3 & 3) * 4 + (c >> 5 & 3)) * 16 +
                                                ((c & 3) << 1) + (c >> 2 & 1)
                                          : (c >> 3) * 16 + (c & 7));
      const __nv_bfloat16 b = __float2bfloat16_rn(value);
      to[0] = __bfloat16_as_ushort(b);
      to[8] = __bfloat16_as_ushort(__float2bfloat16_rn(__hisinf(b) ? 0.0f : value - __bfloat162float(b)));
    }
  }
  __device__ __forceinline__ void fetch(const uint16_t* p, int, Eight& e) const {
    asm("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(e.high[0]), "=r"(e.high[1]), "=r"(e.high[2]), "=r"(e.high[3]), "=r"(e.low[0]), "=r"(e.low[1]),
                   "=r"(e.low[2]), "=r"(e.low[3])
                 : "l"(p));
  }
};

template <int kHeld, bool kTwo>
__device__ __forceinline__ void mma_eight(float (&sum)[4], uint32_t a0, uint32_t b0, uint32_t a1, uint32_t b1,
                                          uint32_t a2, uint32_t b2, uint32_t a3, uint32_t b3, const Eight& e) {
  mma<kHeld>(sum, a0, b0, a1, b1, e.high[0], e.high[1]);
  mma<kHeld>(sum, a2, b2, a3, b3, e.high[2], e.high[3]);
  if (kTwo) {
    mma<kHeld>(sum, a0, b0, a1, b1, e.low[0], e.low[1]);
    mma<kHeld>(sum, a2, b2, a3, b3, e.low[2], e.low[3]);
  }
}

// A batch: the slots' two rows by up to kTiles tiles of eight columns; column[n]
// is the row of the other side that this lane brings into tile n.  reload(d)
// fills slot d again as soon as it has been used.  The last tiles come first, so
// that this is after tile 0 for any number of them.
template <int kHeld, int kTiles, typename From, typename Reload>
__device__ __forceinline__ void multiply(Slot (&slot)[kSteps<kHeld>], const Batch& b, int steps, int tiles,
                                         const int (&column)[kTiles], const From& from, float (&sum)[kTiles][4],
                                         Reload reload) {
  const int t = threadIdx.x & 3;
  if constexpr (kIsMx4<kHeld>) {
#pragma unroll
    for (int d = 0; d < kSteps<kHeld>; ++d) {
      if (!b.whole && b.step + d >= steps) {
        reload(d);
        continue;
      }
      const Slot& s = slot[d];
      const bool twice = __any_sync(kFullWarp, max(s.scale[0], s.scale[1]) > 128u);
      const auto fetch = [&](int n, Eight (&e)[4]) {
        const uint16_t* p = from.row(column[n]) + From::at(b.step + d, 0);
        const int c = (b.step + d) * 128 + t * 32;
#pragma unroll
        for (int q = 0; q < 4; ++q) from.fetch(p + (From::at(0, q) - From::at(0, 0)), c + q * 8, e[q]);
      };
      // The columns' way from the caches passes behind the decoding.
      Eight columns[4];
      fetch(0, columns);
      uint32_t v[4][4], w[4][4];
      const uint32_t f0 = factor_of(s.scale[0], twice), f1 = factor_of(s.scale[1], twice);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        decode8(word_of(s.row[0], q), f0, v[q]);
        decode8(word_of(s.row[1], q), f1, w[q]);
      }
      if (twice) {
        const uint32_t g0 = again_of(s.scale[0]), g1 = again_of(s.scale[1]);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          v[i / 4][i % 4] = times_bf16(v[i / 4][i % 4], g0);
          w[i / 4][i % 4] = times_bf16(w[i / 4][i % 4], g1);
        }
      }
      reload(d);
#pragma unroll
      for (int n = 0; n < kTiles; ++n) {
        if (n >= tiles) break;
        if (n > 0) fetch(n, columns);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          mma_eight<kHeld, From::kTwo>(sum[n], v[q][0], w[q][0], v[q][1], w[q][1], v[q][2], w[q][2], v[q][3], w[q][3],
                                       columns[q]);
      }
    }
  } else {
#pragma unroll
    for (int n = kTiles - 1; n >= 1; --n) {
      if (n >= tiles) continue;
#pragma unroll
      for (int d0 = 0; d0 < kSteps<kHeld>; d0 += 2) {  // the columns of two steps are loaded together
        Eight e[2];
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          const int step = b.step + d0 + d;
          const uint16_t* p = from.row(column[n]) + From::at(step, 0);
          if (b.whole || step < steps) from.fetch(p, step * 32 + t * 8, e[d]);
        }
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          const Slot& s = slot[d0 + d];
          if (b.whole || b.step + d0 + d < steps)
            mma_eight<kHeld, From::kTwo>(sum[n], s.row[0].x, s.row[1].x, s.row[0].y, s.row[1].y, s.row[0].z,
                                         s.row[1].z, s.row[0].w, s.row[1].w, e[d]);
        }
      }
    }
#pragma unroll
    for (int d = 0; d < kSteps<kHeld>; ++d) {
      const Slot& s = slot[d];
      if (b.whole || b.step + d < steps)
        mma_eight<kHeld, From::kTwo>(sum[0], s.row[0].x, s.row[1].x, s.row[0].y, s.row[1].y, s.row[0].z, s.row[1].z,
                                     s.row[0].w, s.row[1].w, s.column);
      reload(d);
    }
  }
}

// A warp's way through the batches [begin, end) of tiles of `batches` batches each.
// Experts of more than kTiles column tiles have their rows passed by again for each
// kTiles of them, a warp's share of a tile at a time.  Between its passes all warps read
// so much that the rows come from the cache only where the kernel's matrices fit it:
// 64 tokens of 8 experts, 4 a token, two passes, read 1.0 times up and gate and 1.0
// times down from memory with 1024 x 2048, and 1.7 and 2.0 times with 4096 x 2048.
//   point(tile, from, step, at)  where the lane's part of the batch at a tile's step
//                                lies, and its row of column tile `from`
//   look(tile, from, column)     column[] of column tiles `from` on; returns how many
//                                there are
//   finish(tile, first, last, from, tiles, sum)  takes the sums of a tile's batches
//                                [first, last) by column tiles `from` on
template <int kHeld, int kTiles, bool kWide, typename From, typename Point, typename Look, typename Finish>
__device__ __forceinline__ void stream(int begin, int end, int steps, const Divisor& by_batches, int depth,
                                       const From& from, Point point, Look look, Finish finish) {
  const int batches = (steps + kSteps<kHeld> - 1) / kSteps<kHeld>;
  int tile = by_batches.quotient(begin), first = begin - tile * batches, left = end - begin;
  if (left <= 0) return;
  const auto batch_at = [&](int b) {
    return Batch{b * kSteps<kHeld>, (b + 1) * kSteps<kHeld> * kDepth<kHeld> <= depth};
  };
  Ahead at = {};
  Batch next = batch_at(first);
  Slot slot[kSteps<kHeld>];
  point(tile, 0, next.step, at);
#pragma unroll
  for (int d = 0; d < kSteps<kHeld>; ++d) {
    load_rows<kHeld, kWide>(slot[d], at, d, next, steps, depth);
    load_column<kHeld>(slot[d], at, d, next, steps, from);
  }
  int column_tile = 0;
#pragma unroll 1
  while (left > 0) {
    const int last = min(batches, first + left);
    int column[kTiles];
    const int tiles = look(tile, column_tile, column);
    const bool again = kTiles > 1 && tiles > kTiles;
    float sum[kTiles][4];
#pragma unroll
    for (int n = 0; n < kTiles; ++n) sum[n][0] = sum[n][1] = sum[n][2] = sum[n][3] = 0.0f;
    bool more;
    int batch = first;
#pragma unroll 1
    do {
      const Batch now = next;
      more = ++batch < last;
      const bool any = more || again || left > last - first;
      if (more) {
        next = batch_at(batch);
        move_on<kHeld, From>(at);
      } else if (any) {
        next = batch_at(again ? first : 0);
        point(again ? tile : tile + 1, again ? column_tile + kTiles : 0, next.step, at);
      }
      multiply<kHeld, kTiles>(slot, now, steps, tiles, column, from, sum, [&](int d) {
        if (!any) return;
        load_rows<kHeld, kWide>(slot[d], at, d, next, steps, depth);
        load_column<kHeld>(slot[d], at, d, next, steps, from);
      });
    } while (more);
    finish(tile, first, last, column_tile, min(tiles, kTiles), sum);
    if (again) {
      column_tile += kTiles;
      continue;
    }
    left -= last - first;
    first = column_tile = 0;
    ++tile;
  }
}

__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// A tile of h: the active expert, the tile's first row, its rows.
struct Place {
  int expert, row, count;
};

// A tile's sums to h.  v holds columns 2t and 2t + 1 of column tile n, rows g and g
// + 8 of the weights (with a gate: of the gate and of up).
template <int kHeld>
__device__ __noinline__ void to_h(const LayerArgs& a, const Routing& routing, Place p, int n, float4 v) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int first_row = routing.start[p.expert], columns = routing.rows_of[p.expert];
#pragma unroll 1
  for (int j = 0; j < 2; ++j, v.x = v.y, v.z = v.w) {
    const int col = n * 8 + t * 2 + j;
    if (col >= columns) continue;
    const int row = first_row + col;
    uint16_t* h = a.h + static_cast<int64_t>(row) * 2 * a.h_pitch;
#pragma unroll 1
    for (int k = 0; k < (a.gated ? 1 : 2); ++k) {
      const float f = k ? v.z : v.x;
      const float act = a.silu ? f / (1.0f + expf(-f)) : (f > 0.0f || f != f ? f : 0.0f);
      const float value = routing.weight[row] * (a.gated ? act * v.z : act);
      const int at = g + 8 * k;
      if (at >= p.count) continue;
      FromH<kHeld>::put(h, p.row + at, value);
    }
    // Zeros behind the end of each row, up to a whole step.
    if (p.row + p.count == a.hidden)
      for (int c = a.hidden + g; c < a.h_pitch; c += 8) FromH<kHeld>::put(h, c, 0.0f);
  }
}

// The rows of h of all active experts laid end to end, each CTA an equal share
// of them.  A tile is 16 rows of weights: 8 rows of h with a gate (rows g of the
// gate beside rows g of up, so one lane ends up with both), 16 without.  The
// tiles' batches are again laid end to end, and each warp takes an equal share of
// these.  Parts of tiles go to shared memory and are joined in order when all
// warps are done.
template <int kHeld, int kTiles, bool kWide>
__global__ void __launch_bounds__(kWarps * 32, 1)
    up_kernel(const __grid_constant__ LayerArgs a) {
  __shared__ Routing routing;
  extern __shared__ float4 parts[];  // [warp][first, last][tile of columns][lane]
  const int most_tiles = (a.tokens + 7) >> 3;
  launch_dependents();
  const int active = route_all(a, routing, reinterpret_cast<Choice*>(parts));
  if (blockIdx.x == 0) pass_on(a.routing, routing);

  const int lane = threadIdx.x & 31, g = lane >> 2, warp = threadIdx.x >> 5;
  const int high = a.gated ? 8 : 16;  // rows of h of a tile
  const int steps = (a.width + kDepth<kHeld> - 1) / kDepth<kHeld>;
  const int batches = (steps + kSteps<kHeld> - 1) / kSteps<kHeld>;
  const int rows = active * a.hidden, each = a.by_ctas.quotient(rows), over = rows - each * gridDim.x;
  const int begin = each * blockIdx.x + min(static_cast<int>(blockIdx.x), over);
  const int here = each + (static_cast<int>(blockIdx.x) < over);
  if (here == 0) return;

  // Tiles do not reach over the end of an expert: those of the first expert
  // here, then as many of each other one.
  const int expert0 = a.by_hidden.quotient(begin), row0 = begin - expert0 * a.hidden;
  const int per_expert = (a.hidden + high - 1) / high;
  const int rows_first = min(a.hidden - row0, here), in_first = (rows_first + high - 1) / high;
  const int experts_whole = a.by_hidden.quotient(here - rows_first);
  const int rows_last = here - rows_first - experts_whole * a.hidden;
  const int total = (in_first + experts_whole * per_expert + (rows_last + high - 1) / high) * batches;
  const auto place = [&](int tile) {
    Place p{expert0, row0 + tile * high, 0};
    if (tile >= in_first) {
      const int other = a.by_tiles.quotient(tile - in_first);
      p.expert = expert0 + 1 + other;
      p.row = (tile - in_first - other * per_expert) * high;
    }
    p.count = min(min(high, a.hidden - p.row), begin + here - (p.expert * a.hidden + p.row));
    return p;
  };
  const auto share = [&](int w) { return static_cast<int>(static_cast<int64_t>(total) * w / kWarps); };
  const int mine = share(warp), my_end = share(warp + 1);
  const FromX<kHeld, kWide> from{static_cast<const uint16_t*>(a.x), a.x_stride, a.width};
  // A warp's part of the tile that it ends in, or else begins in.
  const auto part = [&](int w, bool last) { return parts + (w * 2 + last) * (most_tiles * 32) + lane; };
  // Rows and columns beyond the tile's are read as its last ones and left out of h.
  const auto point = [&](int tile, int column_tile, int step, Ahead& at) {
    const Place p = place(tile);
    const int e = routing.active[p.expert], last = p.row + p.count - 1;
    point_at<kHeld>(a.gated ? a.gate : a.up, e, min(p.row + g, last), step, at, 0);
    point_at<kHeld>(a.up, e, min(p.row + (a.gated ? g : 8 + g), last), step, at, 1);
    if (!kIsMx4<kHeld>) {
      const int column = min(column_tile * 8 + g, routing.rows_of[p.expert] - 1);
      at.column = from.row(routing.token[routing.start[p.expert] + column]) + from.at(step, 0);
    }
  };
  const auto look = [&](int tile, int column_tile, int (&column)[kTiles]) {
    const int expert = place(tile).expert, first_row = routing.start[expert], columns = routing.rows_of[expert];
#pragma unroll
    for (int n = 0; n < kTiles; ++n)
      column[n] = routing.token[first_row + min((column_tile + n) * 8 + g, columns - 1)];
    return ((columns + 7) >> 3) - column_tile;
  };
  const auto finish = [&](int tile, int first, int last, int column_tile, int tiles,
                          const float (&sum)[kTiles][4]) {
    const bool whole = first == 0 && last == batches;
    const Place p = place(tile);
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
      if (kTiles > 1 && n >= tiles) break;
      const float4 v = make_float4(sum[n][0], sum[n][1], sum[n][2], sum[n][3]);
      if (whole) to_h<kHeld>(a, routing, p, column_tile + n, v);
      else part(warp, first == 0)[(column_tile + n) * 32] = v;
    }
  };
  stream<kHeld, kTiles, kWide>(mine, my_end, steps, a.by_up_batches, a.width, from, point, look, finish);
  __syncthreads();
  // Each warp joins the tile that ends in its share having begun before it.
  const int tile = a.by_up_batches.quotient(mine), tile_begin = tile * batches;
  if (mine == my_end || tile_begin == mine || tile_begin + batches > my_end) return;
  int from_warp = warp;
  while (share(from_warp) > tile_begin) --from_warp;
  const Place p = place(tile);
#pragma unroll 1
  for (int n = 0; n * 8 < routing.rows_of[p.expert]; ++n) {
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
    for (int w = from_warp; w <= warp; ++w) {
      if (share(w) == share(w + 1)) continue;
      const float4 o = part(w, share(w) <= tile_begin)[n * 32];
      v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
    }
    to_h<kHeld>(a, routing, p, n, v);
  }
}

// h beside f16 matrices, a CTA to a row: from floats to two f16 numbers an element,
// times the power of two that brings the row's largest finite magnitude into [2^14,
// 2^15).  So an element is held to 22 bits, or to 2^-39 of its row's largest, whatever
// the row's size; the down kernel takes the power back out of its 32-bit sums.  Eight
// elements keep their 32 bytes.
// A launch of its own costs 2 us for one token and 4 of 230 for 32 of 128 experts of
// 2048 x 1024.  (With both sides as tf32 none is needed, but what is worked on between
// its load and the matrix instruction is waited for early: 277 us.)
constexpr int kScaleThreads = 256;
template <int kHeld>
__global__ void __launch_bounds__(kScaleThreads) scale_kernel(const __grid_constant__ LayerArgs a) {
  static_assert(kHeld == kF16, "others need none");
  __shared__ uint32_t of_warp[kScaleThreads / 32];
  launch_dependents();
  wait_for_previous();
  Routing& routing = *static_cast<Routing*>(a.routing);
  const int row = blockIdx.x, last = routing.count - 1;
  if (last < 0 || row >= routing.start[last] + routing.rows_of[last]) return;
  uint4* h = reinterpret_cast<uint4*>(a.h + static_cast<int64_t>(row) * 2 * a.h_pitch);
  const int pieces = a.h_pitch / 8;
  uint32_t most = 0;
  const auto look = [&](uint32_t bits) {
    bits &= 0x7fffffffu;
    if (bits < 0x7f800000u) most = max(most, bits);
  };
  for (int i = threadIdx.x; i < 2 * pieces; i += kScaleThreads) {
    const uint4 v = h[i];
    look(v.x), look(v.y), look(v.z), look(v.w);
  }
  most = __reduce_max_sync(kFullWarp, most);
  if (threadIdx.x % 32 == 0) of_warp[threadIdx.x / 32] = most;
  __syncthreads();
  most = __reduce_max_sync(kFullWarp, of_warp[threadIdx.x % (kScaleThreads / 32)]);
  // Both powers are normal floats.
  const uint32_t exponent = max(most >> 23, 15u);
  const float factor = __uint_as_float((268u - exponent) << 23);
  for (int i = threadIdx.x; i < pieces; i += kScaleThreads) {
    const uint4 v[2] = {h[2 * i], h[2 * i + 1]};
    uint32_t high[4], low[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint4& w = v[j / 2];
      const float2 f = mul2(make_float2(__uint_as_float(j % 2 ? w.z : w.x), __uint_as_float(j % 2 ? w.w : w.y)),
                            make_float2(factor, factor));
      high[j] = floats_to_pair(f, __half());
      const float2 first = pair_to_floats(high[j], __half());
      // An infinity's rest is 0, not inf - inf.
      low[j] = floats_to_pair(make_float2(isinf(first.x) ? 0.0f : f.x - first.x,
                                          isinf(first.y) ? 0.0f : f.y - first.y), __half());
    }
    h[2 * i] = make_uint4(high[0], high[1], high[2], high[3]);
    h[2 * i + 1] = make_uint4(low[0], low[1], low[2], low[3]);
  }
  if (threadIdx.x == 0) routing.weight[row] = __uint_as_float((exponent - 14u) << 23);
}

// Each CTA an equal share of y's channels, 16 at a time, over all active
// experts: with their rows of h end to end the layer's second half is one
// product of great depth, so no two CTAs add to one sum.  The warps split that
// depth evenly; each adds an expert's columns to its tokens' sums in shared
// memory when it has passed the expert, and at the end the warps' sums are
// added in order.  More than 16 channels a CTA are more passes, each over all of the
// depth and of h, the last for what is left: on 152 SMs 8 tokens of 32 experts of width
// x 768, 4 a token, take 75 us at a width of 2432 and 87 at 2560 (in 4 bits 62 and 74),
// 132 at 4864 and 189 at 7168 (102 and 141).
template <int kHeld, int kTiles, bool kWide>
__global__ void __launch_bounds__(kWarps * 32, 1)
    down_kernel(const __grid_constant__ LayerArgs a) {
  __shared__ Routing routing;
  extern __shared__ float sums[];  // [warp][token][16]
  wait_for_previous();
  take_over(routing, a.routing);
  const int active = routing.count;

  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, warp = threadIdx.x >> 5;
  const int steps = (a.hidden + kDepth<kHeld> - 1) / kDepth<kHeld>;
  const int batches = (steps + kSteps<kHeld> - 1) / kSteps<kHeld>;
  const int total = active * batches;
  const int begin = total * warp / kWarps, end = total * (warp + 1) / kWarps;
  const int each = a.by_ctas.quotient(a.width), over = a.width - each * gridDim.x;
  const int first = each * blockIdx.x + min(static_cast<int>(blockIdx.x), over);
  const int last = first + each + (static_cast<int>(blockIdx.x) < over);
  const FromH<kHeld> from{a.h, a.h_pitch};
  float* mine = sums + warp * a.tokens * 16;

  for (int channel = first; channel < last; channel += 16) {
    const int count = min(16, last - channel);
    for (int i = lane; i < a.tokens * 16; i += 32) mine[i] = 0.0f;
    __syncwarp();
    // Channels and columns beyond the tile's are read as its last ones and left out of y.
    const auto point = [&](int tile, int column_tile, int step, Ahead& at) {
      const int e = routing.active[tile], last_channel = channel + count - 1;
      point_at<kHeld>(a.down, e, min(channel + g, last_channel), step, at, 0);
      point_at<kHeld>(a.down, e, min(channel + 8 + g, last_channel), step, at, 1);
      if (!kIsMx4<kHeld>)
        at.column =
            from.row(routing.start[tile] + min(column_tile * 8 + g, routing.rows_of[tile] - 1)) + from.at(step, 0);
    };
    const auto look = [&](int tile, int column_tile, int (&column)[kTiles]) {
      const int first_row = routing.start[tile], columns = routing.rows_of[tile];
#pragma unroll
      for (int n = 0; n < kTiles; ++n) column[n] = first_row + min((column_tile + n) * 8 + g, columns - 1);
      return ((columns + 7) >> 3) - column_tile;
    };
    const auto finish = [&](int tile, int, int, int column_tile, int tiles, const float (&sum)[kTiles][4]) {
      const int first_row = routing.start[tile], columns = routing.rows_of[tile];
#pragma unroll
      for (int n = 0; n < kTiles; ++n) {
        if (kTiles > 1 && n >= tiles) break;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int col = (column_tile + n) * 8 + t * 2 + j;
          if (col < columns) {
            float* p = mine + routing.token[first_row + col] * 16 + g;
            // scale_kernel's power of two, back out of the sum
            const float scale = kHeld == kF16 ? routing.weight[first_row + col] : 1.0f;
            p[0] += scale * sum[n][j];
            p[8] += scale * sum[n][j + 2];
          }
        }
      }
      __syncwarp();
    };
    stream<kHeld, kTiles, kWide>(begin, end, steps, a.by_down_batches, a.hidden, from, point, look, finish);
    __syncthreads();
    for (int i = threadIdx.x; i < a.tokens * 16; i += kWarps * 32) {
      float v = sums[i];
#pragma unroll 4
      for (int w = 1; w < kWarps; ++w) v += sums[w * a.tokens * 16 + i];
      const int token = i >> 4, c = i & 15;
      if (c >= count) continue;
      const int64_t at = static_cast<int64_t>(token) * a.width + channel + c;
      if (a.dtype == DSMEM_F16) static_cast<__half*>(a.out)[at] = from_float<__half>(v);
      else static_cast<__nv_bfloat16*>(a.out)[at] = from_float<__nv_bfloat16>(v);
    }
    __syncthreads();
  }
}

template <int kHeld, int kTiles, bool kWide>
cudaError_t launch_up(const LayerArgs& a, const CallContext& ctx, cudaStream_t stream) {
  static SmemLimit limit;
  const auto kernel = up_kernel<kHeld, kTiles, kWide>;
  const int bytes = kWarps * 2 * ((a.tokens + 7) / 8) * 32 * static_cast<int>(sizeof(float4));
  const cudaError_t e = limit.need(reinterpret_cast<const void*>(kernel), ctx.device, bytes);
  if (e != cudaSuccess) return e;
  kernel<<<ctx.sm_count, kWarps * 32, bytes, stream>>>(a);
  return cudaGetLastError();
}

// A launch that begins while the one before it runs, and waits for it itself.
template <typename Kernel>
cudaError_t launch_behind(Kernel kernel, int ctas, int threads, int bytes, const LayerArgs& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(bytes);
  cfg.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int kHeld, int kTiles, bool kWide>
cudaError_t launch_down(const LayerArgs& a, const CallContext& ctx, cudaStream_t stream) {
  static SmemLimit limit;
  const auto kernel = down_kernel<kHeld, kTiles, kWide>;
  const int bytes = kWarps * a.tokens * 16 * static_cast<int>(sizeof(float));
  cudaError_t e = limit.need(reinterpret_cast<const void*>(kernel), ctx.device, bytes);
  if constexpr (kHeld == kF16) {
    if (e == cudaSuccess) e = launch_behind(scale_kernel<kHeld>, a.tokens * a.top_k, kScaleThreads, 0, a, stream);
  }
  return e == cudaSuccess ? launch_behind(kernel, ctx.sm_count, kWarps * 32, bytes, a, stream) : e;
}

// Whether rows of a 16-bit matrix are whole 16-byte vectors.  Others are loaded by
// words and shifted: 16 tokens, 16 experts of 1023 x 511 in 43 us, of 1024 x 512 in 21.
bool whole_vectors(const LayerMatrix& m, int columns) {
  return reinterpret_cast<uintptr_t>(m.values) % 16 == 0 && m.row_stride % 8 == 0 && m.group_stride % 8 == 0 &&
         columns % 8 == 0;
}

template <int kHeld, int kTiles>
cudaError_t launch_ups(const LayerArgs& a, const CallContext& ctx, cudaStream_t stream) {
  const bool wide = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && a.x_stride % 8 == 0 && a.width % 8 == 0 &&
                    (kIsMx4<kHeld> || (whole_vectors(a.up, a.width) && (!a.gated || whole_vectors(a.gate, a.width))));
  return wide ? launch_up<kHeld, kTiles, true>(a, ctx, stream) : launch_up<kHeld, kTiles, false>(a, ctx, stream);
}

template <int kHeldUp, int kHeldDown, int kTiles>
cudaError_t launch_with(const LayerArgs& a, const CallContext& ctx, cudaStream_t stream) {
  const cudaError_t e = launch_ups<kHeldUp, kTiles>(a, ctx, stream);
  if (e != cudaSuccess) return e;
  if constexpr (!kIsMx4<kHeldDown>) {
    if (!whole_vectors(a.down, a.hidden)) return launch_down<kHeldDown, kTiles, false>(a, ctx, stream);
  }
  return launch_down<kHeldDown, kTiles, true>(a, ctx, stream);
}
// Up to 8 tokens have one column tile.  (With 4 tiles for any number, 8 tokens took
// 54.0 us, not 51.1, and in 4 bits 44.6, not 43.0; 64 experts of 2048 x 768, 4 a token.)
// For more the kernels hold the sums of 2, or of 4 where the matrices would have to be
// decoded again for each 2: with 4 the 16-bit ones, whose columns of a step wait in
// registers too, took 100 us, not 96, for 32 tokens and 139, not 128, for 64; with 2
// the 4-bit ones 38, not 33, for 32 tokens of 8 experts (80 and 78 of 64).  8 tiles, for
// 64 tokens, spilled registers: 33 tokens took 122 us and in 4 bits 112, not 82.
template <int kHeldUp, int kHeldDown>
cudaError_t launch_both(const LayerArgs& a, const CallContext& ctx, cudaStream_t stream) {
  if (a.tokens <= 8) return launch_with<kHeldUp, kHeldDown, 1>(a, ctx, stream);
  return launch_with<kHeldUp, kHeldDown, kIsMx4<kHeldDown> ? 4 : 2>(a, ctx, stream);
}

}  // namespace
}  // namespace dsmh
