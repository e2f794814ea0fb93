// Matrices in 8-bit floating point (e4m3) with a power-of-two scale for each
// row and 128 of its inputs, laid out for the matrix core.
//
// A block is 16 rows x 128 inputs, 2048 bytes, [tile of 16 rows][128 inputs]:
// lane l of a wave holds row l % 16 and inputs 32 s + 8 (l / 16) + 0..7 for
// s = 0..3, steps 0 and 1 in 16 bytes at 16 l, steps 2 and 3 at 1024 + 16 l.  So
// a fragment goes from memory, or from LDS, to v_mfma_scale_f32_16x16x128_f8f6f4
// in two 16-byte loads a lane, whole lines each, without bank conflicts; which
// 32 inputs a lane has does not matter as long as both operands agree.
// Scales are bytes b, standing for 2^(b - 127), [tile][ceil(blocks / 4)][16
// rows][4]: the four blocks' scales of a row in one word.  The matrix
// instruction applies them itself.
#pragma once

#include "common.hpp"
#include "internal.hpp"
#include "rows.hpp"

namespace twell {

typedef int32_t i32x8_t __attribute__((ext_vector_type(8)));
typedef short i16x2_t __attribute__((ext_vector_type(2)));

constexpr int kF8Block = 128;    // inputs of a block
constexpr int kF8Bytes = 2048;   // of a block
constexpr int kF8Scales = 64;    // bytes of four blocks' scales

// The scale byte of values up to `most` (bits of a finite float): of the
// smallest power of two, from 2^-126 on, that takes them into e4m3's range, up
// to 448 = 1.75 2^8.
__device__ __forceinline__ uint32_t f8_scale_byte(uint32_t most) {
  const int e = static_cast<int>(most >> 23) - 8 + ((most & 0x7fffffu) > 0x600000u ? 1 : 0);
  return static_cast<uint32_t>(e > 1 ? e : 1);
}
__device__ __forceinline__ float f8_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// The largest of a value over the four lanes that hold a row's block.
__device__ __forceinline__ uint32_t max_over_row(uint32_t m) {
  const auto a = __builtin_amdgcn_permlane32_swap(m, m, false, false);
  m = max(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane16_swap(m, m, false, false);
  return max(b[0], b[1]);
}

// One lane's 32 inputs of a row's block, from memory to codes.  An infinity or a
// NaN has no part in the scale and becomes a NaN code.
template <class E>
struct F8Inputs;
template <>
struct F8Inputs<EBf16> {
  u32x4_t raw[4];  // of each step
  __device__ __forceinline__ void load(const uint16_t* row, int c0, int lane, int K) {
#pragma unroll
    for (int s = 0; s < 4; ++s) raw[s] = load_piece<EBf16>(row, c0 + 32 * s + 8 * (lane >> 4), K);
  }
  // Bits of the largest magnitude, as fp32.
  __device__ __forceinline__ uint32_t most() const {
    typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
    u16x2_t m{0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i)
      m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, raw[i / 4][i % 4] & 0x7fff7fffu));
    if (__any(m[0] >= 0x7f80 || m[1] >= 0x7f80)) {
      m = u16x2_t{0, 0};
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        u16x2_t v = __builtin_bit_cast(u16x2_t, raw[i / 4][i % 4] & 0x7fff7fffu);
        v[0] = v[0] < 0x7f80 ? v[0] : 0;
        v[1] = v[1] < 0x7f80 ? v[1] : 0;
        m = __builtin_elementwise_max(m, v);
      }
    }
    return static_cast<uint32_t>(max(m[0], m[1])) << 16;
  }
  // Over the scale, rounded to nearest even: the only rounding there is.
  __device__ __forceinline__ void codes(float scale, u32x4_t (&c)[2]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      i16x2_t r{0, 0};
      r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, pair(2 * i), scale, false);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, pair(2 * i + 1), scale, true);
      c[i / 4][i % 4] = __builtin_bit_cast(uint32_t, r);
    }
  }

 private:
  __device__ __forceinline__ bf16x2_t pair(int i) const {
    const bf16x8_t v = __builtin_bit_cast(bf16x8_t, raw[i / 4]);  // whole, as above (AxpyCoef)
    return bf16x2_t{v[2 * (i % 4)], v[2 * (i % 4) + 1]};
  }
};
template <>
struct F8Inputs<EF32> {
  float f[32];
  __device__ __forceinline__ void load(const float* row, int c0, int lane, int K) {
#pragma unroll
    for (int i = 0; i < 32; i += 4)
      Piece<EF32>::unpack(load_piece<EF32>(row, c0 + 32 * (i / 8) + 8 * (lane >> 4) + i % 8, K), f + i);
  }
  __device__ __forceinline__ uint32_t most() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const uint32_t u = __float_as_uint(f[i]) & 0x7fffffffu;
      m = max(m, u < 0x7f800000u ? u : 0u);
    }
    return m;
  }
  __device__ __forceinline__ void codes(float scale, u32x4_t (&c)[2]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      i16x2_t r{0, 0};
      r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, f[4 * i], f[4 * i + 1], scale, false);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, f[4 * i + 2], f[4 * i + 3], scale, true);
      c[i / 4][i % 4] = __builtin_bit_cast(uint32_t, r);
    }
  }
};

// Where the rows of tile `index` are: tiles of `unit` rows, numbered expert by
// expert, the last of each expert short.  Called by whole waves; every result is
// wave-uniform.  Offsets that do not ascend or leave 0 .. T are cut to what does.
struct F8Place {
  int expert;      // -1: there is no such tile
  int64_t row0;    // first row
  int rows;        // 1 .. unit
  int64_t tile16;  // tiles of 16 rows before row0, as the codes of rows are laid out
  int tiles16;     // of its expert from row0 on
};
__device__ __forceinline__ F8Place f8_locate(const int32_t* offsets, int experts, int64_t T, int unit, int64_t index) {
  F8Place p{-1, 0, 0, 0, 0};
  if (!offsets) {
    const int64_t row0 = index * unit;
    if (row0 >= T) return p;
    const int64_t left = T - row0;
    return {0, row0, static_cast<int>(left < unit ? left : unit), row0 / 16, static_cast<int>((left + 15) / 16)};
  }
  const int lane = threadIdx.x & 63;
  int tiles = 0, tiles16 = 0;  // of the experts before; index and 16-row tiles fit 32 bits
  for (int e0 = 0; e0 < experts; e0 += 64) {
    const int e = e0 + lane;
    int a = 0, b = 0;
    if (e < experts) {
      const int top = static_cast<int>(T);
      a = min(max(offsets[e], 0), top);
      b = min(max(offsets[e + 1], a), top);
    }
    const int n = (b - a + unit - 1) / unit, n16 = (b - a + 15) / 16;
    const int in = wave_incl_scan(n), in16 = wave_incl_scan(n16);
    const uint64_t past = __ballot(tiles + in > index);
    if (past) {
      const int l = __builtin_amdgcn_readfirstlane(__builtin_ctzll(past));
      const int k = static_cast<int>(index) - tiles - __builtin_amdgcn_readlane(in - n, l);
      const int first = __builtin_amdgcn_readlane(a, l), last = __builtin_amdgcn_readlane(b, l);
      p.expert = e0 + l;
      p.row0 = first + static_cast<int64_t>(k) * unit;
      p.rows = static_cast<int>(min(static_cast<int64_t>(unit), last - p.row0));
      p.tile16 = tiles16 + __builtin_amdgcn_readlane(in16 - n16, l) + k * (unit / 16);
      p.tiles16 = (last - static_cast<int>(p.row0) + 15) / 16;
      return p;
    }
    tiles += wave_last(in);
    tiles16 += wave_last(in16);
  }
  return p;
}

// `bytes` of memory from base on, for the loads below: a base in scalar registers
// and 32-bit offsets, so that a loop of loads needs no vector registers for
// addresses.  Loads past the bytes give zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t f8_buffer(const uint8_t* base, uint32_t bytes = 0xffffffffu) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, bytes, 0x00027000);
}
// 16 bytes a lane straight to LDS: from base + lane_offset + offset (wave-uniform);
// lane l's go to lds + 16 l (lds wave-uniform).
__device__ __forceinline__ void direct16(__amdgpu_buffer_rsrc_t base, uint32_t lane_offset, uint32_t offset, uint8_t* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(base, lds, 16, lane_offset, offset, 0, 0);
}

// 16 bytes a lane to registers, from the same place.
__device__ __forceinline__ u32x4_t buffer16(__amdgpu_buffer_rsrc_t base, uint32_t lane_offset, uint32_t offset) {
  return __builtin_amdgcn_raw_buffer_load_b128(base, lane_offset, offset, 0);
}

__device__ __forceinline__ uint32_t buffer4(__amdgpu_buffer_rsrc_t base, uint32_t lane_offset, uint32_t offset) {
  return __builtin_amdgcn_raw_buffer_load_b32(base, lane_offset, offset, 0);
}

// Workgroup id to tile: ids go round-robin to the 8 XCDs, each of which gets a
// run of tiles here, so that workgroups that share operands share an L2.
__device__ __forceinline__ int xcd_run(int id, int n) {
  const int xcd = id & 7, per = n >> 3, more = n & 7;
  return xcd * per + (xcd < more ? xcd : more) + (id >> 3);
}

}  // namespace twell
