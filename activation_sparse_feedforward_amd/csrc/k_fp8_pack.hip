// Weights and rows to e4m3 (fp8.hpp), and weights back.
#include "fp8.hpp"
#include "launch.hpp"
#include "rows.hpp"

namespace twell {
namespace {

constexpr int kPackWaves = 4;

// The scale of block b of `blocks` to a row's four; the last block's workgroup fills what is left of them with zeros.
__device__ __forceinline__ void put_scale(uint8_t* four, uint32_t byte, int b, int blocks) {
  four[b % 4] = static_cast<uint8_t>(byte);
  if (b + 1 == blocks)
    for (int i = b % 4 + 1; i < 4; ++i) four[i] = 0;
}

// One workgroup per 128 x 128 weights, which share a scale, so that the codes of
// the transposed matrix are the same numbers.  Reading and writing bound it; the
// transposed codes go through LDS byte by byte, a tenth of that time.  16 fp32
// matrices of 1024 x 2048 with both planes: 32.8 us, 6.1 TB/s.
constexpr int kLdsRow = kF8Block + 4;
template <class E>
__global__ __launch_bounds__(kPackWaves* kWave) void f8_pack_kernel(F8PackArgs a) {
  using S = typename E::storage;
  __shared__ uint32_t most[kPackWaves];
  __shared__ __align__(16) uint8_t lds[kF8Block * kLdsRow];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int cb = blockIdx.x, rb = blockIdx.y;
  const int64_t e = blockIdx.z;
  const S* w = static_cast<const S*>(a.w) + e * a.N * a.K;
  F8Inputs<E> in[2];
  uint32_t m = 0;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int r = rb * 128 + (2 * wave + t) * 16 + (lane & 15);
    // rows past the matrix are zeros: none of their inputs exists
    in[t].load(w + static_cast<int64_t>(min(r, a.N - 1)) * a.K, cb * 128, lane, r < a.N ? a.K : 0);
  }
#pragma unroll
  for (int t = 0; t < 2; ++t) m = max(m, in[t].most());
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), x)));
  if (lane == 0) most[wave] = m;
  __syncthreads();
  m = max(max(most[0], most[1]), max(most[2], most[3]));
  const uint32_t byte = f8_scale_byte(m);
  const float scale = f8_scale(byte);
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    u32x4_t c[2];
    in[t].codes(scale, c);
    const int tile = rb * 8 + 2 * wave + t;
    if (tile < a.tiles) {
      uint8_t* to = a.codes + ((e * a.tiles + tile) * a.blocks + cb) * kF8Bytes + lane * 16;
      *reinterpret_cast<u32x4_t*>(to) = c[0];
      *reinterpret_cast<u32x4_t*>(to + 1024) = c[1];
    }
    if (a.codes_t) {
      uint8_t* row = lds + ((2 * wave + t) * 16 + (lane & 15)) * kLdsRow + 8 * (lane >> 4);
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        *reinterpret_cast<uint32_t*>(row + 32 * s) = c[s / 2][2 * (s % 2)];
        *reinterpret_cast<uint32_t*>(row + 32 * s + 4) = c[s / 2][2 * (s % 2) + 1];
      }
    }
  }
  if (threadIdx.x < 128) {
    const int tile = rb * 8 + threadIdx.x / 16;
    if (tile < a.tiles)
      put_scale(a.scales + ((e * a.tiles + tile) * a.quads + cb / 4) * kF8Scales + (threadIdx.x % 16) * 4, byte, cb,
                a.blocks);
  } else if (a.codes_t) {
    const int i = threadIdx.x - 128, tile = cb * 8 + i / 16;
    if (tile < a.tiles_t)
      put_scale(a.scales_t + ((e * a.tiles_t + tile) * a.quads_t + rb / 4) * kF8Scales + (i % 16) * 4, byte, rb,
                a.blocks_t);
  }
  if (!a.codes_t) return;
  __syncthreads();
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int tile = cb * 8 + 2 * wave + t;
    if (tile >= a.tiles_t) continue;
    const uint8_t* col = lds + (2 * wave + t) * 16 + (lane & 15);
    u32x4_t c[2];
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t v = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v |= static_cast<uint32_t>(col[(32 * s + 8 * (lane >> 4) + 4 * h + i) * kLdsRow]) << (8 * i);
        c[s / 2][2 * (s % 2) + h] = v;
      }
    uint8_t* to = a.codes_t + ((e * a.tiles_t + tile) * a.blocks_t + rb) * kF8Bytes + lane * 16;
    *reinterpret_cast<u32x4_t*>(to) = c[0];
    *reinterpret_cast<u32x4_t*>(to + 1024) = c[1];
  }
}

// Codes times scales, exact in fp32 (but for scales whose products leave its
// range), rounded once to bf16.  One wave a block.
template <class E>
__global__ __launch_bounds__(kPackWaves* kWave) void f8_unpack_kernel(F8PackArgs a) {
  using S = typename E::storage;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kPackWaves + wave;
  const int64_t tile = id / a.blocks;  // of all experts
  const int b = static_cast<int>(id % a.blocks);
  if (tile >= static_cast<int64_t>(a.experts) * a.tiles) return;
  const int64_t e = tile / a.tiles;
  const int r = static_cast<int>(tile % a.tiles) * 16 + (lane & 15);
  const uint8_t* from = a.codes + (tile * a.blocks + b) * kF8Bytes + lane * 16;
  const u32x4_t c[2] = {*reinterpret_cast<const u32x4_t*>(from), *reinterpret_cast<const u32x4_t*>(from + 1024)};
  const float scale = f8_scale(a.scales[(tile * a.quads + b / 4) * kF8Scales + (lane & 15) * 4 + b % 4]);
  if (r >= a.N) return;
  S* out = static_cast<S*>(a.out) + (e * a.N + r) * a.K;
  constexpr int kN = Piece<E>::kN;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    float f[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int v = static_cast<int>(c[s / 2][2 * (s % 2) + h]);
      const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(v, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(v, true);
      f[4 * h] = lo[0] * scale;
      f[4 * h + 1] = lo[1] * scale;
      f[4 * h + 2] = hi[0] * scale;
      f[4 * h + 3] = hi[1] * scale;
    }
#pragma unroll
    for (int i = 0; i < 8; i += kN)
      store_piece<E>(out, b * 128 + 32 * s + 8 * (lane >> 4) + i, a.K, Piece<E>::pack(f + i));
  }
}

// Rows to codes: a wave has four blocks of 16 rows, whose scales make whole words.
// 16384 rows of 2048 in bf16 take 31 us from memory (3.3 TB/s, where a copy reaches
// 4.9: a load takes 64 bytes of each of 16 rows, half lines), 20 from the caches; of
// 1024 12 us.
template <class E>
__global__ __launch_bounds__(kPackWaves* kWave) void f8_rows_kernel(F8RowsArgs a) {
  using S = typename E::storage;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int quad = blockIdx.y * kPackWaves + wave;
  if (quad >= a.quads) return;
  const F8Place p = f8_locate(a.offsets, a.experts, a.T, 16, blockIdx.x);
  if (p.expert < 0 || p.tile16 >= a.most_tiles) return;
  const int r = lane & 15;
  const S* row = static_cast<const S*>(a.x) + (p.row0 + (r < p.rows ? r : 0)) * a.ldx;
  F8Inputs<E> in[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) in[j].load(row, (quad * 4 + j) * 128, lane, a.K);  // past the row: zeros
  uint32_t word = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int b = quad * 4 + j;
    if (b >= a.blocks) break;
    const uint32_t byte = f8_scale_byte(max_over_row(in[j].most()));
    word |= byte << (8 * j);
    u32x4_t c[2];
    in[j].codes(f8_scale(byte), c);
    uint8_t* to = a.codes + (p.tile16 * a.blocks + b) * kF8Bytes + lane * 16;
    *reinterpret_cast<u32x4_t*>(to) = c[0];
    *reinterpret_cast<u32x4_t*>(to + 1024) = c[1];
  }
  if (lane < 16)
    *reinterpret_cast<uint32_t*>(a.scales + (p.tile16 * a.quads + quad) * kF8Scales + lane * 4) = word;
}

}  // namespace

hipError_t launch_f8_pack(const F8PackArgs& a, int dtype, hipStream_t s) {
  const dim3 grid(a.blocks, (a.N + 127) / 128, a.experts);
  return dtype == 1 ? launch(f8_pack_kernel<EBf16>, grid, kPackWaves * kWave, 0, s, a)
                    : launch(f8_pack_kernel<EF32>, grid, kPackWaves * kWave, 0, s, a);
}
hipError_t launch_f8_unpack(const F8PackArgs& a, int dtype, hipStream_t s) {
  const int64_t n = static_cast<int64_t>(a.experts) * a.tiles * a.blocks;
  const dim3 grid(static_cast<unsigned>((n + kPackWaves - 1) / kPackWaves));
  return dtype == 1 ? launch(f8_unpack_kernel<EBf16>, grid, kPackWaves * kWave, 0, s, a)
                    : launch(f8_unpack_kernel<EF32>, grid, kPackWaves * kWave, 0, s, a);
}
hipError_t launch_f8_rows(const F8RowsArgs& a, int dtype, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(a.offsets ? a.most_tiles : (a.T + 15) / 16),
                  (a.quads + kPackWaves - 1) / kPackWaves);
  return dtype == 1 ? launch(f8_rows_kernel<EBf16>, grid, kPackWaves * kWave, 0, s, a)
                    : launch(f8_rows_kernel<EF32>, grid, kPackWaves * kWave, 0, s, a);
}

}  // namespace twell
