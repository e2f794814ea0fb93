// Rows of bf16 or fp32 read and written 16 bytes a lane, wherever they begin.
#pragma once

#include "common.hpp"

namespace twell {

// 16 bytes at any element's address: global memory takes such an access at any
// alignment (unaligned access mode), so odd widths keep the wide loads.
typedef uint32_t u32x4_any_t __attribute__((ext_vector_type(4), aligned(2)));

__device__ __forceinline__ u32x4_t load16(const void* p) { return *static_cast<const u32x4_any_t*>(p); }
__device__ __forceinline__ void store16(void* p, u32x4_t v) { *static_cast<u32x4_any_t*>(p) = v; }
// The same past the caches.
__device__ __forceinline__ void store16_past(void* p, u32x4_t v) {
  __builtin_nontemporal_store(static_cast<u32x4_any_t>(v), static_cast<u32x4_any_t*>(p));
}

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

// v's bytes moved down by `bytes` (1 .. 15), zeros from above.
__device__ __forceinline__ u32x4_t shifted_down(const u32x4_t& v, int bytes) {
  uint64_t lo = v[0] | static_cast<uint64_t>(v[1]) << 32, hi = v[2] | static_cast<uint64_t>(v[3]) << 32;
  const int s = 8 * (bytes & 7);
  if (bytes & 8) {
    lo = hi;
    hi = 0;
  }
  lo = lo >> s | hi << 1 << (63 - s);
  hi >>= s;
  return u32x4_t{static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32), static_cast<uint32_t>(hi),
                 static_cast<uint32_t>(hi >> 32)};
}

// Elements [c, c + kN) of a row of n elements; what is past its end reads as
// zero and is not written.  c is a multiple of kN.  The last piece of a row is read
// as its last 16 bytes and moved down: one load (element by element it was eight,
// one after another; layer norm's gradients of 16384 rows of 4099 in bf16 took 226 us).
template <class E>
__device__ __forceinline__ u32x4_t load_piece(const typename E::storage* row, int c, int n) {
  constexpr int kN = Piece<E>::kN;
  if (c + kN <= n) return load16(row + c);
  u32x4_t v{0, 0, 0, 0};
  if (c >= n) return v;
  if (n >= kN) return shifted_down(load16(row + n - kN), (c + kN - n) * E::kBytes);
#pragma unroll
  for (int i = 0; i < kN; ++i) {  // a row of less than 16 bytes
    if (i >= n) continue;
    if constexpr (E::kBytes == 2) v[i / 2] |= static_cast<uint32_t>(row[i]) << (16 * (i % 2));
    else v[i] = __float_as_uint(row[i]);
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
