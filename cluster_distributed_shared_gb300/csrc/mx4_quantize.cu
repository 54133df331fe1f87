// Microscaled 4-bit quantisation and its way back.
//
// Both read every byte once and write every byte once, and memory bounds them
// where rows are many: bf16 rows 57 us there and 55 us back at 65536 x 2048
// (5.9 and 6.1 TB/s), f32 rows 96 and 92 us (6.3 and 6.6 TB/s).  For that a
// thread has kPieces loads in flight before it uses the first, and the arithmetic
// an element is kept to about four instructions: magnitudes are compared as
// packed bits, products and conversions work on pairs.  With a thread to a block
// of 32, and elements looked at one by one, 16384 x 2048 there and back took 42 us,
// not 27.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "divisor.h"
#include "dtypes.cuh"
#include "experts.h"
#include "mx4.cuh"

namespace dsmh {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kEach = 8;     // elements of a piece, which one thread takes at a time
constexpr int kPieces = 4;   // pieces of a thread, all in flight together

struct Rows {
  const void* in;    // quantise: rows of floats; the way back: 4-bit values
  void* out;
  uint8_t* scales;
  int64_t stride;    // quantise: elements between rows of floats
  int total;         // pieces of all rows
  int columns;       // elements of a row
  int pieces;        // pieces of a padded row
  Divisor by_pieces;
};

// Eight elements of a row as words of their type, zeros behind its end.  kWide:
// rows are whole 16-byte vectors; others are loaded by words and shifted (16384 x
// 2048 in 14 us, 16384 x 2047 in 20).
template <typename T>
struct Piece {
  static constexpr int kVectors = kEach * static_cast<int>(sizeof(T)) / 16;
  Vector16<T> v[kVectors];
  template <bool kWide>
  __device__ __forceinline__ void load(const T* row, int first, int columns) {
#pragma unroll
    for (int i = 0; i < kVectors; ++i) {
      const int at = first + i * Vector16<T>::kPairs * 2;
      if constexpr (kWide) {
        v[i].words(at < columns ? __ldcs(reinterpret_cast<const uint4*>(row + at)) : make_uint4(0, 0, 0, 0));
      } else if constexpr (sizeof(T) == 2) {
        v[i].words(aligned_piece(reinterpret_cast<const uint16_t*>(row), at, columns,
                                 (reinterpret_cast<uintptr_t>(row) & 2u) != 0));
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i].w[j] = at + j < columns ? __float_as_uint(row[at + j]) : 0u;
      }
    }
  }
  // Bits, as a float, of the largest magnitude: bits of magnitudes are in their
  // order, and those of NaN the largest.
  __device__ __forceinline__ uint32_t largest() const {
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < kVectors; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 2) most = __vmaxu2(most, v[i].w[j] & 0x7fff7fffu);
        else most = max(most, v[i].w[j] & 0x7fffffffu);
      }
    if constexpr (sizeof(T) == 2) most = max(most & 0xffffu, most >> 16);
    return most;
  }
  // Those bits of the type's as bits of a float.
  __device__ __forceinline__ static uint32_t as_float(uint32_t bits) {
    if constexpr (sizeof(T) == 4) return bits;
    else return __float_as_uint(pair_to_floats(bits, T()).x);
  }
  __device__ __forceinline__ float2 pair(int i) const {
    return v[i / Vector16<T>::kPairs].get(i % Vector16<T>::kPairs);
  }
};

// Four neighbouring lanes hold a block of 32 elements: the largest magnitude is
// the maximum of their bits, and gives the scale; every product with the
// scale's inverse is exact.
template <typename T, bool kWide>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const Rows r) {
  const int first = blockIdx.x * (kThreads * kPieces) + threadIdx.x;
  Piece<T> piece[kPieces];
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    const int i = min(first + u * kThreads, r.total - 1);
    const int row = r.by_pieces.quotient(i);
    piece[u].template load<kWide>(static_cast<const T*>(r.in) + row * r.stride, (i - row * r.pieces) * kEach,
                                  r.columns);
  }
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    const int i = first + u * kThreads;
    uint32_t most = piece[u].largest();
    most = max(most, __shfl_xor_sync(kFull, most, 1));
    most = max(most, __shfl_xor_sync(kFull, most, 2));
    const uint32_t byte = mx_scale_byte(Piece<T>::as_float(most));
    const float inverse = mx_inverse(byte);
    float2 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = mul2(piece[u].pair(j), make_float2(inverse, inverse));
    const uint32_t word = byte == 255u ? 0u : e2m1_word(v);
    if (i < r.total) {
      static_cast<uint32_t*>(r.out)[i] = word;
      if (threadIdx.x % 4 == 0) r.scales[i / 4] = static_cast<uint8_t>(byte);
    }
  }
}

// A piece as pairs of bf16, which hold all these values exactly, in order.
__device__ __forceinline__ void decode_in_order(uint32_t word, uint32_t byte, uint32_t (&pair)[4]) {
  const bool twice = byte > 128u;
  uint32_t r[4];
  decode8(word, factor_of(byte, twice), r);
  if (twice) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = times_bf16(r[i], again_of(byte));
  }
  pair[0] = __byte_perm(r[0], r[1], 0x5410);
  pair[1] = __byte_perm(r[2], r[3], 0x5410);
  pair[2] = __byte_perm(r[0], r[1], 0x7632);
  pair[3] = __byte_perm(r[2], r[3], 0x7632);
}

// How rows of the output may be written: element by element, by 16 bytes, or by
// whole sectors of 32 (which floats fill: by halves they took 127 us where whole
// ones take 92, 65536 rows of 2048).
enum Width { kElements, kVectors, kSectors };

template <typename T, int kWidth>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const Rows r) {
  const int first = blockIdx.x * (kThreads * kPieces) + threadIdx.x;
  uint32_t word[kPieces], byte[kPieces];
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    const int i = min(first + u * kThreads, r.total - 1);
    word[u] = __ldcs(static_cast<const uint32_t*>(r.in) + i);
    byte[u] = r.scales[i / 4];
  }
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    const int i = first + u * kThreads;
    if (i >= r.total) break;
    const int row = r.by_pieces.quotient(i);
    const int at = (i - row * r.pieces) * kEach;
    if (at >= r.columns) continue;
    uint32_t pair[4];
    decode_in_order(word[u], byte[u], pair);
    T* out = static_cast<T*>(r.out) + static_cast<int64_t>(row) * r.columns + at;
    if constexpr (kWidth == kSectors) {
      float v[kEach];
#pragma unroll
      for (int j = 0; j < kEach / 2; ++j) {
        const float2 f = pair_to_floats(pair[j], __nv_bfloat16());
        v[2 * j] = f.x, v[2 * j + 1] = f.y;
      }
      asm volatile("st.global.cs.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(out), "f"(v[0]), "f"(v[1]),
                   "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                   : "memory");
    } else if constexpr (kWidth == kVectors) {
      constexpr int kPairs = Vector16<T>::kPairs;
#pragma unroll
      for (int j = 0; j < kEach / 2; j += kPairs) {
        Vector16<T> p;
#pragma unroll
        for (int q = 0; q < kPairs; ++q) {
          if constexpr (std::is_same<T, __nv_bfloat16>::value) p.w[q] = pair[j + q];
          else p.set(q, pair_to_floats(pair[j + q], __nv_bfloat16()));
        }
        if (at + 2 * j < r.columns) __stcs(reinterpret_cast<uint4*>(out + 2 * j), p.words());
      }
    } else {
      T v[kEach];
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        const float2 f = pair_to_floats(pair[j / 2], __nv_bfloat16());
        v[j] = from_float<T>(j % 2 ? f.y : f.x);
      }
      if (sizeof(T) == 2 && at + kEach <= r.columns) {
        // By words, where they begin.
        const int odd = reinterpret_cast<uintptr_t>(out) / 2 % 2;
        if (odd) out[0] = v[0];
#pragma unroll
        for (int j = 0; j < kEach / 2; ++j) {
          Pack<T, 2> p;
          p.v[0] = odd ? v[(2 * j + 1) % kEach] : v[2 * j], p.v[1] = odd ? v[(2 * j + 2) % kEach] : v[2 * j + 1];
          if (!odd || j + 1 < kEach / 2) *reinterpret_cast<Pack<T, 2>*>(out + 2 * j + odd) = p;
        }
        if (odd) out[kEach - 1] = v[kEach - 1];
      } else {
#pragma unroll
        for (int j = 0; j < kEach; ++j)
          if (at + j < r.columns) out[j] = v[j];
      }
    }
  }
}

bool rows_of_vectors(const void* p, int64_t stride, int64_t columns, int size) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * size % 16 == 0 && columns * size % 16 == 0;
}

// Launches over at most 2^30 pieces, whose numbers are divided in 31 bits.
template <typename Launch>
cudaError_t in_parts(const Mx4Args& a, Launch launch) {
  Rows r = {};
  r.columns = a.columns;
  r.pieces = mx4_padded(a.columns) / kEach;
  r.by_pieces = Divisor(static_cast<uint32_t>(r.pieces));
  const int64_t most = std::max<int64_t>((int64_t{1} << 30) / r.pieces, 1);
  cudaError_t e = cudaSuccess;
  for (int64_t row = 0; row < a.rows && e == cudaSuccess; row += most) {
    r.total = static_cast<int>(std::min(most, a.rows - row) * r.pieces);
    launch(r, row, static_cast<unsigned>((r.total + kThreads * kPieces - 1) / (kThreads * kPieces)));
    e = cudaGetLastError();
  }
  return e;
}

template <typename T>
cudaError_t quantize(const Mx4Args& a, cudaStream_t stream) {
  const bool wide = rows_of_vectors(a.x, a.rows > 1 ? a.stride : 0, a.columns, sizeof(T));
  return in_parts(a, [&](Rows& r, int64_t row, unsigned ctas) {
    r.in = static_cast<const T*>(a.x) + row * a.stride;
    r.stride = a.stride;
    r.out = a.values + row * r.pieces * 4;
    r.scales = a.scales + row * (r.pieces / 4);
    if (wide) quantize_kernel<T, true><<<ctas, kThreads, 0, stream>>>(r);
    else quantize_kernel<T, false><<<ctas, kThreads, 0, stream>>>(r);
  });
}
template <typename T>
cudaError_t dequantize(const Mx4Args& a, cudaStream_t stream) {
  const bool wide = rows_of_vectors(a.out, a.columns, a.columns, sizeof(T));
  return in_parts(a, [&](Rows& r, int64_t row, unsigned ctas) {
    r.in = a.values + row * r.pieces * 4;
    r.scales = a.scales + row * (r.pieces / 4);
    r.out = static_cast<T*>(a.out) + row * a.columns;
    if constexpr (sizeof(T) == 4) {
      if (reinterpret_cast<uintptr_t>(a.out) % 32 == 0 && a.columns % kEach == 0) {
        dequantize_kernel<T, kSectors><<<ctas, kThreads, 0, stream>>>(r);
        return;
      }
    }
    if (wide) dequantize_kernel<T, kVectors><<<ctas, kThreads, 0, stream>>>(r);
    else dequantize_kernel<T, kElements><<<ctas, kThreads, 0, stream>>>(r);
  });
}

}  // namespace

cudaError_t launch_quantize(const Mx4Args& a, cudaStream_t stream) {
  if (a.dtype == DSMEM_F32) return quantize<float>(a, stream);
  if (a.dtype == DSMEM_F16) return quantize<__half>(a, stream);
  return quantize<__nv_bfloat16>(a, stream);
}
cudaError_t launch_dequantize(const Mx4Args& a, cudaStream_t stream) {
  if (a.dtype == DSMEM_F32) return dequantize<float>(a, stream);
  if (a.dtype == DSMEM_F16) return dequantize<__half>(a, stream);
  return dequantize<__nv_bfloat16>(a, stream);
}

}  // namespace dsmh
