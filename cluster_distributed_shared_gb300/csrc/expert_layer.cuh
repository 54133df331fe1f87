// A whole expert layer for a few tokens, in two kernels.
//
// With e = ids[t, j] and w = weights[t, j] of a token's routing,
//   up kernel    h[t, j] = w act(up[e] x[t]),  or  w act(gate[e] x[t]) * (up[e] x[t])
//   down kernel  y[t]    = sum over j of down[e] h[t, j]
// A few tokens do little arithmetic on many weights, so both kernels are bound
// by reading the chosen experts' matrices once, and everything follows from
// keeping loads of them in flight:
//   * Rows of the matrices go from global memory straight to the registers of
//     mma.sync fragments.  The depth may be summed in any order, so lane
//     (g, t) = (lane / 4, lane % 4) takes 16 consecutive bytes of rows g and
//     g + 8 and the same elements of the rows' side: no shared memory, no
//     transposition, one load for two (16-bit) or eight (4-bit) instructions.
//     (A tcgen05 tile would be 128 rows high, of which one token's share of an
//     SM fills 27, and would pass every byte through shared memory.)
//   * Every SM reads the same number of rows, every warp the same number of
//     steps of depth, kSteps of them in flight.
//   * Each CTA routes all tokens for itself instead of waiting for a launch
//     that does; the down kernel is launched while the up kernel runs
//     (programmatic dependent launch) and waits for it only after its own
//     routing and first loads of weights.
// Sums are 32-bit: in the fragments along a warp's part of the depth, then over
// the warps through shared memory in their order.  Nothing is added atomically.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "dtypes.cuh"
#include "experts.h"
#include "mx4.cuh"
#include "route.cuh"

namespace dsmh {
namespace layer {

constexpr int kLayerWarps = 16;
constexpr int kLayerThreads = kLayerWarps * 32;
constexpr int kSteps = 4;  // steps of depth a warp has in flight
constexpr int kMaxTokens = DSMEM_LAYER_MAX_TOKENS;
constexpr int kMaxRows = kMaxTokens * DSMEM_ROUTE_MAX_TOP_K;

// How the matrices are held, and with them the type of the fragments: 16-bit
// matrices have x's type; 4-bit ones become bf16, which holds every value they
// stand for exactly.
enum Held { kBf16, kF16, kMx4Bf16, kMx4F16 };
template <int kHeld>
constexpr bool kIsMx4 = kHeld == kMx4Bf16 || kHeld == kMx4F16;
template <int kHeld>
constexpr int kDepth = kIsMx4<kHeld> ? 128 : 32;  // elements of a step

// Everything a CTA knows about the routing.  Rows are (token, expert) pairs,
// expert after expert, an expert's rows by token.
struct Routing {
  unsigned long long tokens_of[DSMEM_ROUTE_MAX_EXPERTS];  // a bit for each token
  uint16_t start[DSMEM_ROUTE_MAX_EXPERTS + 1];            // of active experts: first row
  uint16_t active[DSMEM_ROUTE_MAX_EXPERTS + 1];           // experts that any token chose, by number
  uint16_t rows_of[DSMEM_ROUTE_MAX_EXPERTS];              // of active experts
  float weight[kMaxRows];                                 // of each row
  uint8_t token[kMaxRows];
  float chosen_weight[kMaxRows];                          // of each token's choices
  int16_t chosen[kMaxRows];
  int count;                                              // active experts
};

// One token's choices by one warp; experts in lane l are l, l + 32, ...
template <int R>
__device__ __forceinline__ void choose(const LayerArgs& a, int token, Routing& r) {
  const int lane = threadIdx.x & 31;
  const int64_t row = token * a.logits_stride;
  uint32_t key[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int e = i * 32 + lane;
    float v = -INFINITY;
    if (e < a.experts) {
      if (a.logits_dtype == DSMEM_F32) v = static_cast<const float*>(a.logits)[row + e];
      else if (a.logits_dtype == DSMEM_F16) v = to_float(static_cast<const __half*>(a.logits)[row + e]);
      else v = to_float(static_cast<const __nv_bfloat16*>(a.logits)[row + e]);
    }
    key[i] = rank_key(v);
  }
  uint32_t best = 0;
#pragma unroll
  for (int i = 0; i < R; ++i) best = max(best, key[i]);
  const float top = rank_value(__reduce_max_sync(kFullWarp, best));
  float all = 0.0f;
  if (!a.renormalize) {
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (key[i]) all += raised(rank_value(key[i]), top);
    all = warp_sum(all);
  }
  int my_id = -1;
  uint32_t my_key = 0;
  for (int j = 0; j < a.top_k; ++j) {
    best = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) best = max(best, key[i]);
    const uint32_t m = __reduce_max_sync(kFullWarp, best);
    if (m == 0u) break;
    uint32_t id = 0xffffffffu;
#pragma unroll
    for (int i = R - 1; i >= 0; --i)
      if (key[i] == m) id = i * 32 + lane;
    id = __reduce_min_sync(kFullWarp, id);
    if (lane == j) my_id = static_cast<int>(id), my_key = m;
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (i * 32 + lane == static_cast<int>(id)) key[i] = 0u;
  }
  const float mine = my_id >= 0 ? raised(rank_value(my_key), top) : 0.0f;
  if (a.renormalize) all = warp_sum(mine);
  if (lane < a.top_k) {
    r.chosen[token * a.top_k + lane] = static_cast<int16_t>(my_id);
    r.chosen_weight[token * a.top_k + lane] = my_id >= 0 ? mine / all : 0.0f;
    if (my_id >= 0) atomicOr(&r.tokens_of[my_id], 1ull << token);
  }
}

// Fills `r`; all threads of the CTA.
__device__ __forceinline__ void route_all(const LayerArgs& a, Routing& r) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < a.experts; e += kLayerThreads) r.tokens_of[e] = 0ull;
  __syncthreads();
  for (int token = warp; token < a.tokens; token += kLayerWarps) {
    if (a.experts <= 128) choose<4>(a, token, r);
    else choose<DSMEM_ROUTE_MAX_EXPERTS / 32>(a, token, r);
  }
  __syncthreads();
  if (warp == 0) {
    int count = 0, rows = 0;
    for (int e0 = 0; e0 < a.experts; e0 += 32) {
      const int e = e0 + lane;
      const int mine = e < a.experts ? __popcll(r.tokens_of[e]) : 0;
      const uint32_t some = __ballot_sync(kFullWarp, mine > 0);
      int before = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(kFullWarp, before, d);
        if (lane >= d) before += up;
      }
      if (mine > 0) {
        const int i = count + __popc(some & ((1u << lane) - 1u));
        r.active[i] = static_cast<uint16_t>(e);
        r.start[i] = static_cast<uint16_t>(rows + before - mine);
        r.rows_of[i] = static_cast<uint16_t>(mine);
      }
      count += __popc(some);
      rows += __shfl_sync(kFullWarp, before, 31);
    }
    if (lane == 0) r.count = count;
  }
  __syncthreads();
  // Each choice to its row.  An active expert's place is found by bisection.
  for (int i = threadIdx.x; i < a.tokens * a.top_k; i += kLayerThreads) {
    const int e = r.chosen[i];
    if (e < 0) continue;
    int low = 0, high = r.count - 1;
    while (low < high) {
      const int mid = (low + high) >> 1;
      if (r.active[mid] < e) low = mid + 1;
      else high = mid;
    }
    const int token = i / a.top_k;
    const int row = r.start[low] + __popcll(r.tokens_of[e] & ((1ull << token) - 1ull));
    r.token[row] = static_cast<uint8_t>(token);
    r.weight[row] = r.chosen_weight[i];
  }
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

// A lane's part of a step: 16 bytes of two rows, and for 4-bit elements (32 of
// them, one block) their scales.
struct Slot {
  uint4 row[2];
  uint32_t scale[2];
};

// Where a lane's part of the next batch of steps lies in two rows of a matrix.
struct TwoRows {
  const uint8_t* row[2];
  const uint8_t* scale[2];
};
// Row `row` of expert `e`, at the batch that begins with step `step`.
template <int kHeld>
__device__ __forceinline__ void point_at(const LayerMatrix& m, int e, int row, int step, TwoRows& to, int i) {
  const int t = threadIdx.x & 3;
  const int64_t size = kIsMx4<kHeld> ? 1 : 2;
  to.row[i] = static_cast<const uint8_t*>(m.values) + (e * m.group_stride + row * m.row_stride) * size + step * 64 + t * 16;
  if (kIsMx4<kHeld>)
    to.scale[i] = m.scales + (static_cast<int64_t>(e) * m.rows + row) * m.scale_stride + step * 4 + t;
}

// The part of a matrix's rows that a batch of kSteps steps takes.
struct Batch {
  int step;    // its first step
  bool whole;  // all of its steps lie inside the rows
};

// Step d of a batch.  kWide: rows of 16-bit matrices begin at 16-byte boundaries
// and are whole vectors.  (4-bit rows always do and are.)
template <int kHeld, bool kWide>
__device__ __forceinline__ void load_slot(Slot& s, const TwoRows& from, int d, const Batch& b, int steps, int depth) {
  const int at = d * 64;
  if constexpr (kIsMx4<kHeld>) {
    if (b.whole || b.step + d < steps) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        s.row[i] = load_once(from.row[i] + at);
        s.scale[i] = __ldg(from.scale[i] + d * 4);
      }
    }
  } else if (kWide && b.whole) {
#pragma unroll
    for (int i = 0; i < 2; ++i) s.row[i] = load_once(from.row[i] + at);
  } else if (b.step + d < steps) {
    const int t = threadIdx.x & 3, c = (b.step + d) * 32 + t * 8;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      s.row[i] = make_uint4(0, 0, 0, 0);
      if constexpr (kWide) {
        if (c < depth) s.row[i] = load_once(from.row[i] + at);
      } else {
        const uint16_t* row = reinterpret_cast<const uint16_t*>(from.row[i] + at) - c;
        s.row[i] = aligned_piece(row, c, depth, (reinterpret_cast<uintptr_t>(row) & 2u) != 0);
      }
    }
  }
}

// Eight 4-bit elements as bf16 pairs (0,4), (1,5), (2,6), (3,7), scaled.  An
// element's sign, exponent and fraction bits at those of a bf16 make its value
// times 2^-126; `factor` (twice, in a pair) makes up for it with the scale.
// Both products are exact.  `again` is the second factor where one bf16 cannot
// hold both, which a whole warp takes together.
__device__ __forceinline__ uint32_t times_bf16(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void decode8(uint32_t w, uint32_t factor, bool twice, uint32_t again, uint32_t (&r)[4]) {
  constexpr uint32_t kSign = 0x80008000u, kRest = 0x01c001c0u;
  r[0] = ((w << 6) & kRest) | ((w << 12) & kSign);
  r[1] = ((w << 2) & kRest) | ((w << 8) & kSign);
  r[2] = ((w >> 2) & kRest) | ((w << 4) & kSign);
  r[3] = ((w >> 6) & kRest) | (w & kSign);
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = times_bf16(r[i], factor);
  if (twice) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = times_bf16(r[i], again);
  }
}
// 2^(byte - 1) = 2^126 2^(byte - 127) as a bf16 pair where it is one, else
// 2^126, with 2^(byte - 127) (or NaN) for `again`.
__device__ __forceinline__ uint32_t factor_of(uint32_t byte, bool twice) {
  return (twice ? 253u : byte + 126u) * 0x00800080u;
}
__device__ __forceinline__ uint32_t again_of(uint32_t byte) {
  const uint32_t bits = byte == 0u ? 0x0040u : (byte == 255u ? 0x7fc0u : byte << 7);
  return bits | bits << 16;
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) {
  return i == 0 ? v.x : (i == 1 ? v.y : (i == 2 ? v.z : v.w));
}

// Eight elements of the rows' side as fragments' words: pairs in the order of
// the matrices', and for values that one 16-bit number does not hold a second
// one, the rest.
struct Eight {
  uint32_t high[4], low[4];
};

// Where the rows' side comes from; `row` is an element's row there and c its
// place.  x: a token's vector, 16-bit, any alignment, read again and again.
template <int kHeld, bool kWide>
struct FromX {
  static constexpr bool kTwo = kHeld == kMx4F16;  // f16 is the sum of two bf16
  const uint16_t* x;
  int64_t stride;
  int depth;
  __device__ __forceinline__ void get(int row, int c, bool whole, Eight& e) const {
    const uint16_t* p = x + row * stride;
    uint4 v = make_uint4(0, 0, 0, 0);
    if constexpr (kWide) {
      if (whole || c < depth) v = __ldg(reinterpret_cast<const uint4*>(p + c));
    } else {
      v = aligned_piece(p, c, depth, (reinterpret_cast<uintptr_t>(p) & 2u) != 0);
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
// h: the up kernel's rows, two numbers an element, in the fragments' order, with
// zeros up to whole steps; each row is read once by a CTA.
struct FromH {
  static constexpr bool kTwo = true;
  const uint16_t* h;  // [rows][2][pitch]
  int pitch;
  __device__ __forceinline__ void get(int row, int c, bool, Eight& e) const {
    const uint16_t* p = h + static_cast<int64_t>(row) * 2 * pitch + c;
    const uint4 high = __ldcg(reinterpret_cast<const uint4*>(p));
    const uint4 low = __ldcg(reinterpret_cast<const uint4*>(p + pitch));
    e.high[0] = high.x, e.high[1] = high.y, e.high[2] = high.z, e.high[3] = high.w;
    e.low[0] = low.x, e.low[1] = low.y, e.low[2] = low.z, e.low[3] = low.w;
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
__device__ __forceinline__ void multiply(Slot (&slot)[kSteps], const Batch& b, int steps, int tiles,
                                         const int (&column)[kTiles], const From& from, float (&sum)[kTiles][4],
                                         Reload reload) {
  const int t = threadIdx.x & 3;
  if constexpr (kIsMx4<kHeld>) {
#pragma unroll
    for (int d = 0; d < kSteps; ++d) {
      if (b.whole || b.step + d < steps) {
        const Slot& s = slot[d];
        const bool twice = __any_sync(kFullWarp, max(s.scale[0], s.scale[1]) > 128u);
        const uint32_t f0 = factor_of(s.scale[0], twice), f1 = factor_of(s.scale[1], twice);
        const uint32_t g0 = again_of(s.scale[0]), g1 = again_of(s.scale[1]);
        const int c = (b.step + d) * 128 + t * 32;
        Eight first[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) from.get(column[0], c + q * 8, b.whole, first[q]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t v[4], w[4];
          decode8(word_of(s.row[0], q), f0, twice, g0, v);
          decode8(word_of(s.row[1], q), f1, twice, g1, w);
          mma_eight<kHeld, From::kTwo>(sum[0], v[0], w[0], v[1], w[1], v[2], w[2], v[3], w[3], first[q]);
#pragma unroll
          for (int n = 1; n < kTiles; ++n) {
            if (n >= tiles) break;
            Eight e;
            from.get(column[n], c + q * 8, b.whole, e);
            mma_eight<kHeld, From::kTwo>(sum[n], v[0], w[0], v[1], w[1], v[2], w[2], v[3], w[3], e);
          }
        }
      }
      reload(d);
    }
  } else {
    constexpr int kAtOnce = From::kTwo ? 2 : 4;  // steps whose columns are loaded together
#pragma unroll
    for (int n = kTiles - 1; n >= 0; --n) {
      if (n > 0 && n >= tiles) continue;
#pragma unroll
      for (int d0 = 0; d0 < kSteps; d0 += kAtOnce) {
        Eight e[kAtOnce];
#pragma unroll
        for (int d = 0; d < kAtOnce; ++d)
          if (b.whole || b.step + d0 + d < steps)
            from.get(column[n], (b.step + d0 + d) * 32 + t * 8, b.whole, e[d]);
#pragma unroll
        for (int d = 0; d < kAtOnce; ++d) {
          const Slot& s = slot[d0 + d];
          if (b.whole || b.step + d0 + d < steps)
            mma_eight<kHeld, From::kTwo>(sum[n], s.row[0].x, s.row[1].x, s.row[0].y, s.row[1].y, s.row[0].z,
                                         s.row[1].z, s.row[0].w, s.row[1].w, e[d]);
          if (n == 0) reload(d0 + d);
        }
      }
    }
  }
}

__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Whether rows of a 16-bit matrix are whole 16-byte vectors.
inline bool whole_vectors(const LayerMatrix& m, int columns) {
  return reinterpret_cast<uintptr_t>(m.values) % 16 == 0 && m.row_stride % 8 == 0 && m.group_stride % 8 == 0 &&
         columns % 8 == 0;
}

}  // namespace layer
}  // namespace dsmh
