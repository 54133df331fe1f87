// Microscaled 4-bit quantisation and its way back.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

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
  int64_t total;     // pieces of all rows
  int columns;       // elements of a row
  int pieces;        // pieces of a padded row
  Divisor by_pieces;
};

// Eight elements of a row from `first` on, zeros behind its end.  kWide: rows
// are whole 16-byte vectors.
template <typename T, bool kWide>
__device__ __forceinline__ void load8(const T* row, int first, int columns, float (&v)[kEach]) {
  if constexpr (kWide) {
    constexpr int kVectors = kEach * static_cast<int>(sizeof(T)) / 16;
#pragma unroll
    for (int i = 0; i < kVectors; ++i) {
      Vector16<T> p;
      const int at = first + i * Vector16<T>::kPairs * 2;
      p.words(at < columns ? __ldcs(reinterpret_cast<const uint4*>(row + at)) : make_uint4(0, 0, 0, 0));
#pragma unroll
      for (int q = 0; q < Vector16<T>::kPairs; ++q) {
        const float2 f = p.get(q);
        v[(i * Vector16<T>::kPairs + q) * 2] = f.x;
        v[(i * Vector16<T>::kPairs + q) * 2 + 1] = f.y;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kEach; ++i) v[i] = first + i < columns ? to_float(row[first + i]) : 0.0f;
  }
}

// Four neighbouring lanes hold a block of 32 elements: the largest magnitude is
// the maximum of their bits, and gives the scale; every product with the
// scale's inverse is exact.
template <typename T, bool kWide>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const Rows r) {
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kThreads * kPieces) + threadIdx.x;
  float v[kPieces][kEach];
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    const int64_t piece = first + u * kThreads;
    if (piece >= r.total) continue;
    const int row = r.by_pieces.quotient(static_cast<int>(piece));
    const int at = (static_cast<int>(piece) - row * r.pieces) * kEach;
    load8<T, kWide>(static_cast<const T*>(r.in) + row * r.stride, at, r.columns, v[u]);
  }
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    const int64_t piece = first + u * kThreads;
    uint32_t largest = 0;
    if (piece < r.total) {
#pragma unroll
      for (int i = 0; i < kEach; ++i) largest = max(largest, __float_as_uint(v[u][i]) & 0x7fffffffu);
    }
    largest = max(largest, __shfl_xor_sync(kFull, largest, 1));
    largest = max(largest, __shfl_xor_sync(kFull, largest, 2));
    if (piece >= r.total) continue;
    const uint32_t byte = mx_scale_byte(largest);
    uint32_t word = 0;
    if (byte != 255u) {
      const float inverse = mx_inverse(byte);
#pragma unroll
      for (int i = 0; i < kEach; i += 2)
        word |= e2m1_pair(v[u][i] * inverse, v[u][i + 1] * inverse) << (4 * i);
    }
    static_cast<uint32_t*>(r.out)[piece] = word;
    if (threadIdx.x % 4 == 0) r.scales[piece / 4] = static_cast<uint8_t>(byte);
  }
}

template <typename T, bool kWide>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const Rows r) {
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kThreads * kPieces) + threadIdx.x;
  uint32_t word[kPieces], byte[kPieces];
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    const int64_t piece = first + u * kThreads;
    if (piece >= r.total) continue;
    word[u] = __ldcs(static_cast<const uint32_t*>(r.in) + piece);
    byte[u] = r.scales[piece / 4];
  }
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    const int64_t piece = first + u * kThreads;
    if (piece >= r.total) continue;
    const int row = r.by_pieces.quotient(static_cast<int>(piece));
    const int at = (static_cast<int>(piece) - row * r.pieces) * kEach;
    if (at >= r.columns) continue;
    const float scale = mx_scale(byte[u]);
    T* out = static_cast<T*>(r.out) + static_cast<int64_t>(row) * r.columns + at;
    if constexpr (kWide) {
      constexpr int kPairs = Vector16<T>::kPairs;
#pragma unroll
      for (int i = 0; i < kEach / 2; i += kPairs) {
        Vector16<T> p;
#pragma unroll
        for (int q = 0; q < kPairs; ++q)
          p.set(q, make_float2(e2m1_value(word[u], 2 * (i + q)) * scale,
                               e2m1_value(word[u], 2 * (i + q) + 1) * scale));
        if (at + 2 * i < r.columns) __stcs(reinterpret_cast<uint4*>(out + 2 * i), p.words());
      }
    } else {
#pragma unroll
      for (int i = 0; i < kEach; ++i)
        if (at + i < r.columns) out[i] = from_float<T>(e2m1_value(word[u], i) * scale);
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
    r.total = std::min(most, a.rows - row) * r.pieces;
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
    if (wide) dequantize_kernel<T, true><<<ctas, kThreads, 0, stream>>>(r);
    else dequantize_kernel<T, false><<<ctas, kThreads, 0, stream>>>(r);
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
