// Rows of bf16 or fp32 read and written 16 bytes a lane, wherever they begin.
#pragma once

#include "common.hpp"

namespace twell {

// 16 bytes at any element's address: global memory takes such an access at any
// alignment (unaligned access mode), so odd widths keep the wide loads.
typedef uint32_t u32x4_any_t __attribute__((ext_vector_type(4), aligned(2)));

__device__ __forceinline__ u32x4_t load16(const void* p) { return *static_cast<const u32x4_any_t*>(p); }
__device__ __forceinline__ void store16(void* p, u32x4_t v) { *static_cast<u32x4_any_t*>(p) = v; }

// Two fp32 values as bf16, rounded to nearest even; NaN stays NaN.
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, bf16x2_t{static_cast<__bf16>(lo), static_cast<__bf16>(hi)});
}

template <class E>
struct Piece;  // 16 bytes as fp32 values
template <>
struct Piece<EBf16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void unpack(const u32x4_t& v, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(v[i] << 16);
      f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ u32x4_t pack(const float* f) {
    u32x4_t v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = bf16_pair(f[2 * i], f[2 * i + 1]);
    return v;
  }
};
template <>
struct Piece<EF32> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void unpack(const u32x4_t& v, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(v[i]);
  }
  static __device__ __forceinline__ u32x4_t pack(const float* f) {
    u32x4_t v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __float_as_uint(f[i]);
    return v;
  }
};

// Elements [c, c + kN) of a row of n elements; what is past its end reads as
// zero and is not written.  c is a multiple of kN.
template <class E>
__device__ __forceinline__ u32x4_t load_piece(const typename E::storage* row, int c, int n) {
  if (c + Piece<E>::kN <= n) return load16(row + c);
  u32x4_t v{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < Piece<E>::kN; ++i) {
    if (c + i >= n) continue;
    if constexpr (E::kBytes == 2) v[i / 2] |= static_cast<uint32_t>(row[c + i]) << (16 * (i % 2));
    else v[i] = __float_as_uint(row[c + i]);
  }
  return v;
}
template <class E>
__device__ __forceinline__ void store_piece(typename E::storage* row, int c, int n, const u32x4_t& v) {
  if (c + Piece<E>::kN <= n) {
    store16(row + c, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < Piece<E>::kN; ++i) {
    if (c + i >= n) continue;
    if constexpr (E::kBytes == 2) row[c + i] = static_cast<uint16_t>(v[i / 2] >> (16 * (i % 2)));
    else row[c + i] = __uint_as_float(v[i]);
  }
}

}  // namespace twell
