// Laying out weights for the few-token products (few_token.hpp), and reading
// them back.  4 bits: each group of 32, 64 or 128 consecutive inputs of a row
// has one scale s = bf16(max|w| * r), r = 1/7 in fp32; codes are
// q = rne(w / s) clamped to -7 .. 7 and stored as q + 8.  A group that holds an
// infinity or a NaN gets a NaN scale, so that every value of it reads back as
// NaN instead of as something plausible.
#include "few_token.hpp"
#include "internal.hpp"

namespace twell {
namespace {

constexpr int kPackWaves = 4;

template <int BITS, int GROUP>
constexpr int scales_per_block() { return BITS == 4 ? kBlockK / GROUP : 1; }

__device__ __forceinline__ uint32_t umax32(uint32_t a, uint32_t b) { return a > b ? a : b; }

// w / s, correctly rounded, for s with 8 significant bits, inv = 1 / s correctly
// rounded, and nothing near the ends of the exponent range: the product with
// inv, corrected once by its exact rest.  (Checked against the division for
// every mantissa of s and w.)  A third of the division's operations, and 16
// divisions' worth of them was half of the pack kernel's time.
__device__ __forceinline__ float divided(float w, float s, float inv) {
  const float t = w * inv;
  return fmaf(fmaf(-t, s, w), inv, t);
}

// Writes one block of 16 rows x 128 inputs; lane's 32 values in f[step][8].
template <int BITS, int GROUP>
__device__ __forceinline__ void store_block(const float (&f)[4][8], uint8_t* codes, uint16_t* scales, int lane) {
  if constexpr (BITS == 16) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      u32x4_t v;
#pragma unroll
      for (int j = 0; j < 4; ++j)  // bf16 in, bf16 out: the upper halves are the values
        v[j] = (__float_as_uint(f[s][2 * j]) >> 16) | (__float_as_uint(f[s][2 * j + 1]) & 0xffff0000u);
      *reinterpret_cast<u32x4_t*>(codes + (s * 64 + lane) * 16) = v;
    }
  } else {
    constexpr int G = scales_per_block<BITS, GROUP>();
    constexpr int kSteps = 4 / G;
    u32x4_t words;
    uint16_t sc[G];
#pragma unroll
    for (int gr = 0; gr < G; ++gr) {
      // largest magnitude of the group as bits: infinities and NaN compare above
      // every finite value
      uint32_t m = 0;
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int i = 0; i < 8; ++i) m = umax32(m, __float_as_uint(f[gr * kSteps + s][i]) & 0x7fffffffu);
      m = umax32(m, __shfl_xor(m, 16));
      m = umax32(m, __shfl_xor(m, 32));
      const bool finite = m < 0x7f800000u;
      sc[gr] = finite ? bf16_of(__uint_as_float(m) * (1.0f / 7.0f)) : static_cast<uint16_t>(0x7fc0);
      const float sf = bf16_bits_to_f32(sc[gr]);
      const bool live = finite && sf > 0.f;
      const float div = live ? sf : 1.f;
      const float inv = 1.0f / div;
      // the rests of quotients below 1/4 may be lost without harm: they round to 0
      const bool plain = div >= 0x1p-100f && div <= 0x1p100f;
      float q[kSteps][8];
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int i = 0; i < 8; ++i) q[s][i] = divided(f[gr * kSteps + s][i], div, inv);
      if (!plain) {
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
          for (int i = 0; i < 8; ++i) q[s][i] = f[gr * kSteps + s][i] / div;
      }
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          // adding 2^23 + 8 rounds to the nearest even whole number and leaves u = q + 8
          // in the lowest bits
          const float c = __builtin_amdgcn_fmed3f(q[s][i], -7.f, 7.f) + 8388616.f;
          w |= (__float_as_uint(c) & 15u) << (4 * (i >> 1) + 16 * (i & 1));
        }
        words[gr * kSteps + s] = __builtin_rotateleft32(live ? w : 0x88888888u, 3);
      }
    }
    *reinterpret_cast<u32x4_t*>(codes + lane * 16) = words;
    if (lane < 16) {
#pragma unroll
      for (int gr = 0; gr < G; ++gr) scales[lane * G + gr] = sc[gr];
    }
  }
}

// w [E][N][K], one wave per block.  Like tokens, rows are read by rows and go
// through LDS.  Bound by reading w: 8192 x 2048 in bf16 to 4 bits 12.0 us, 42 MB
// at 3.5 TB/s; the quotients take about as long.
template <class E, int BITS, int GROUP>
__global__ __launch_bounds__(kPackWaves* kWave) void weights_pack_kernel(WeightsArgs a) {
  using Src = std::conditional_t<E::kBytes == 2, SourceBf16, SourceF32>;
  using X = Tokens<Src, 4>;
  __shared__ __align__(16) char lds[kPackWaves * X::kLdsBytes];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kPackWaves + wave;
  if (id >= static_cast<int64_t>(a.tiles) * a.blocks) return;
  const int tile = static_cast<int>(id / a.blocks), b = static_cast<int>(id % a.blocks);
  const int64_t e = blockIdx.y;
  const int row0 = tile * kTileRows, left = a.N - row0;
  const X x({a.K},
            [&](int r) {
              return static_cast<const typename Src::Elem*>(a.w) + (e * a.N + row0 + (r < left ? r : 0)) * a.K;
            },
            lds + wave * X::kLdsBytes, lane);
  typename X::Loaded q;
  x.fetch(q, b, (b + 1) * kBlockK <= a.K, lane);
  x.store(q, lane);
  const int r = lane & 15;
  float f[4][8];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    u32x4_t v[Src::kReads];
#pragma unroll
    for (int i = 0; i < Src::kReads; ++i)
      v[i] = *reinterpret_cast<const u32x4_t*>(x.lds + X::piece_at(r, Src::place(s, lane >> 4, i)));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t u;
      if constexpr (E::kBytes == 2) u = i & 1 ? v[0][i >> 1] & 0xffff0000u : v[0][i >> 1] << 16;
      else u = v[i >> 2][i & 3];
      f[s][i] = __uint_as_float(r < left ? u : 0u);
    }
  }
  const int64_t blk = (e * a.tiles + tile) * a.blocks + b;
  constexpr int G = scales_per_block<BITS, GROUP>();
  store_block<BITS, GROUP>(f, a.codes + blk * Block<BITS>::kBytes, a.scales + blk * (16 * G), lane);
}

// w [E][K][N] (one row per input): 64 rows x 128 inputs through LDS per
// workgroup, read along N and handed out along K, one element of padding a row
// against bank conflicts.  Bound by reading w: 6 matrices of 1001 x 1407 in fp32
// 11.6 us, 38 MB at 3.3 TB/s.
template <class E, int BITS, int GROUP>
__global__ __launch_bounds__(kPackWaves* kWave) void weights_pack_t_kernel(WeightsArgs a) {
  __shared__ float tile_f[64][kBlockK + 1];
  using Elem = typename E::storage;
  constexpr int kPer = E::kPer16B;      // rows of the result in one load
  constexpr int kAcross = 64 / kPer;    // lanes along N
  constexpr int kDown = 64 / kAcross;   // inputs per load
  constexpr int kLoads = kBlockK / kDown / kPackWaves;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n_groups = (a.tiles + 3) / 4;
  const int tg = static_cast<int>(blockIdx.x % n_groups), b = static_cast<int>(blockIdx.x / n_groups);
  const int64_t e = blockIdx.y;
  const int in = (lane % kAcross) * kPer, n = tg * 64 + in;
  const Elem* w = static_cast<const Elem*>(a.w) + e * a.K * a.N;
  if (tg * 64 + 64 <= a.N && (b + 1) * kBlockK <= a.K) {
    u32x4_t v[kLoads];
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int64_t k = b * kBlockK + (j * kPackWaves + wave) * kDown + lane / kAcross;
      if constexpr (E::kBytes == 2) v[j] = *reinterpret_cast<const u32x4_a2_t*>(w + k * a.N + n);
      else v[j] = *reinterpret_cast<const u32x4_a4_t*>(w + k * a.N + n);
    }
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int i = (j * kPackWaves + wave) * kDown + lane / kAcross;
#pragma unroll
      for (int c = 0; c < kPer; ++c) {
        uint32_t u;
        if constexpr (E::kBytes == 2) u = c & 1 ? v[j][c >> 1] & 0xffff0000u : v[j][c >> 1] << 16;
        else u = v[j][c];
        tile_f[in + c][i] = __uint_as_float(u);
      }
    }
  } else {
    const int m = tg * 64 + lane;
#pragma unroll
    for (int j = 0; j < kBlockK / kPackWaves; ++j) {  // no branch: all loads at once
      const int i = j * kPackWaves + wave, k = b * kBlockK + i;
      const float v = load_elem<E>(w, static_cast<int64_t>(k < a.K ? k : a.K - 1) * a.N + (m < a.N ? m : a.N - 1));
      tile_f[lane][i] = (k < a.K) & (m < a.N) ? v : 0.f;
    }
  }
  __syncthreads();
  const int tile = tg * 4 + wave;
  if (tile >= a.tiles) return;
  float f[4][8];
#pragma unroll
  for (int s = 0; s < 4; ++s)
#pragma unroll
    for (int i = 0; i < 8; ++i) f[s][i] = tile_f[wave * 16 + (lane & 15)][32 * s + 8 * (lane >> 4) + i];
  const int64_t blk = (e * a.tiles + tile) * a.blocks + b;
  constexpr int G = scales_per_block<BITS, GROUP>();
  store_block<BITS, GROUP>(f, a.codes + blk * Block<BITS>::kBytes, a.scales + blk * (16 * G), lane);
}

// The values the planes stand for, into w [E][N][K]; one wave per block, by rows
// through LDS, since a lane's own eight values would be written 16 lines at a
// time.  Bound by writing w: 8192 x 2048 to fp32 12.8 us, 76 MB at 5.9 TB/s.
template <class E, int BITS, int GROUP>
__global__ __launch_bounds__(kPackWaves* kWave) void weights_unpack_kernel(WeightsArgs a) {
  using Elem = typename E::storage;
  constexpr int kPieces = kBlockK / E::kPer16B;  // of 16 bytes in a row of the block
  constexpr int kWaveBytes = 16 * kPieces * 16;
  __shared__ __align__(16) char lds[kPackWaves * kWaveBytes];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kPackWaves + wave;
  if (id >= static_cast<int64_t>(a.tiles) * a.blocks) return;
  const int tile = static_cast<int>(id / a.blocks), b = static_cast<int>(id % a.blocks);
  const int64_t e = blockIdx.y;
  const int64_t blk = (e * a.tiles + tile) * a.blocks + b;
  constexpr int G = scales_per_block<BITS, GROUP>();
  Block<BITS> q;
  q.template load<false>(a.codes + blk * Block<BITS>::kBytes, lane);
  Scales<G> sc;
  if constexpr (BITS == 4) sc.load(a.scales + blk * (16 * G), lane);
  char* mine = lds + wave * kWaveBytes;
  auto piece_at = [&](int r, int c) { return mine + r * kPieces * 16 + ((c ^ r) << 4); };
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int r = lane & 15, g = lane >> 4;
    if constexpr (BITS == 16) {
      *reinterpret_cast<u32x4_t*>(piece_at(r, 4 * s + g)) = q.c[s];
    } else {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int u = static_cast<int>(__builtin_rotateright32(q.c[s], 3 + 4 * (i >> 1) + 16 * (i & 1)) & 15u);
        f[i] = static_cast<float>(u - 8) * sc.at(s * G / 4);
      }
      if constexpr (E::kBytes == 4) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          u32x4_t v;
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = __float_as_uint(f[4 * h + i]);
          *reinterpret_cast<u32x4_t*>(piece_at(r, 8 * s + 2 * g + h)) = v;
        }
      } else {
        u32x4_t v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = bf16_of(f[2 * j]) | (static_cast<uint32_t>(bf16_of(f[2 * j + 1])) << 16);
        *reinterpret_cast<u32x4_t*>(piece_at(r, 4 * s + g)) = v;
      }
    }
  }
  lds_handoff();
  const int row0 = tile * kTileRows;
#pragma unroll
  for (int j = 0; j < kPieces / 4; ++j) {  // 64 pieces are 64 / kPieces rows
    const int r = (j * 64 + lane) / kPieces, c = lane % kPieces;
    const u32x4_t v = *reinterpret_cast<const u32x4_t*>(piece_at(r, c));
    const int k = b * kBlockK + c * E::kPer16B;
    if (row0 + r >= a.N) continue;
    Elem* p = static_cast<Elem*>(a.out) + (e * a.N + row0 + r) * a.K + k;
    if (k + E::kPer16B <= a.K) {
      if constexpr (E::kBytes == 2) *reinterpret_cast<u32x4_a2_t*>(p) = v;
      else *reinterpret_cast<u32x4_a4_t*>(p) = v;
    } else {
#pragma unroll
      for (int i = 0; i < E::kPer16B; ++i) {
        if (k + i >= a.K) break;
        if constexpr (E::kBytes == 2) p[i] = static_cast<uint16_t>(v[i >> 1] >> (16 * (i & 1)));
        else p[i] = __uint_as_float(v[i]);
      }
    }
  }
}

// Launches the instance of K for (element type, bits, group).
template <template <class, int, int> class K>
hipError_t dispatch(const WeightsArgs& a, int dtype, dim3 grid, hipStream_t s) {
  auto go = [&](void (*kernel)(WeightsArgs)) { return launch(kernel, grid, kPackWaves * kWave, 0, s, a); };
  const bool f32 = dtype == 0;
  if (a.bits == 16) return go(K<EBf16, 16, 128>::kernel());
  if (a.group == 32) return go(f32 ? K<EF32, 4, 32>::kernel() : K<EBf16, 4, 32>::kernel());
  if (a.group == 64) return go(f32 ? K<EF32, 4, 64>::kernel() : K<EBf16, 4, 64>::kernel());
  return go(f32 ? K<EF32, 4, 128>::kernel() : K<EBf16, 4, 128>::kernel());
}
template <class E, int B, int G>
struct Pack {
  static auto kernel() { return &weights_pack_kernel<E, B, G>; }
};
template <class E, int B, int G>
struct PackT {
  static auto kernel() { return &weights_pack_t_kernel<E, B, G>; }
};
template <class E, int B, int G>
struct Unpack {
  static auto kernel() { return &weights_unpack_kernel<E, B, G>; }
};

dim3 block_grid(const WeightsArgs& a) {
  const int64_t n = static_cast<int64_t>(a.tiles) * a.blocks;
  return dim3(static_cast<unsigned>((n + kPackWaves - 1) / kPackWaves), static_cast<unsigned>(a.experts));
}

}  // namespace

hipError_t launch_weights_pack(const WeightsArgs& a, int dtype, bool transposed, hipStream_t s) {
  if (!transposed) return dispatch<Pack>(a, dtype, block_grid(a), s);
  const int64_t n = static_cast<int64_t>((a.tiles + 3) / 4) * a.blocks;
  return dispatch<PackT>(a, dtype, dim3(static_cast<unsigned>(n), static_cast<unsigned>(a.experts)), s);
}

hipError_t launch_weights_unpack(const WeightsArgs& a, int dtype, hipStream_t s) {
  return dispatch<Unpack>(a, dtype, block_grid(a), s);
}

}  // namespace twell
