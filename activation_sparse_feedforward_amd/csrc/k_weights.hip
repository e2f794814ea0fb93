// Laying out weights for the few-token products (few_token.hpp), and reading
// them back.  4 bits: each group of 32, 64 or 128 consecutive inputs of a row
// has one scale s = bf16(max|w| / 7), the quotient in fp32; codes are
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

// Inputs k .. k+7 of one row as fp32, zeros from K on (p: the row).
template <class E>
__device__ __forceinline__ void row8(const void* base, int64_t row_off, int k, int K, bool whole, float (&f)[8]) {
  if constexpr (E::kBytes == 2) {
    const uint16_t* p = static_cast<const uint16_t*>(base) + row_off + k;
    if (whole) {
      const u32x4_t v = *reinterpret_cast<const u32x4_a2_t*>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(v[i] << 16);
        f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = k + i < K ? bf16_bits_to_f32(p[i]) : 0.f;
    }
  } else {
    const float* p = static_cast<const float*>(base) + row_off + k;
    if (whole) {
      const u32x4_t a = *reinterpret_cast<const u32x4_a4_t*>(p);
      const u32x4_t b = *reinterpret_cast<const u32x4_a4_t*>(p + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[i] = __uint_as_float(a[i]);
        f[4 + i] = __uint_as_float(b[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = k + i < K ? p[i] : 0.f;
    }
  }
}

__device__ __forceinline__ uint32_t umax32(uint32_t a, uint32_t b) { return a > b ? a : b; }

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
      sc[gr] = finite ? bf16_of(__uint_as_float(m) / 7.0f) : static_cast<uint16_t>(0x7fc0);
      const float sf = bf16_bits_to_f32(sc[gr]);
      const bool live = finite && sf > 0.f;
      const float div = live ? sf : 1.f;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float q = fminf(fmaxf(rintf(f[gr * kSteps + s][i] / div), -7.f), 7.f);
          const uint32_t u = live ? static_cast<uint32_t>(static_cast<int>(q) + 8) : 8u;
          w |= u << (4 * (i >> 1) + 16 * (i & 1));
        }
        words[gr * kSteps + s] = __builtin_rotateleft32(w, 3);
      }
    }
    *reinterpret_cast<u32x4_t*>(codes + lane * 16) = words;
    if (lane < 16) {
#pragma unroll
      for (int gr = 0; gr < G; ++gr) scales[lane * G + gr] = sc[gr];
    }
  }
}

// w [E][N][K], one wave per block.
template <class E, int BITS, int GROUP>
__global__ __launch_bounds__(kPackWaves* kWave) void weights_pack_kernel(WeightsArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kPackWaves + (threadIdx.x >> 6);
  if (id >= static_cast<int64_t>(a.tiles) * a.blocks) return;
  const int tile = static_cast<int>(id / a.blocks), b = static_cast<int>(id % a.blocks);
  const int64_t e = blockIdx.y;
  const int row = tile * kTileRows + (lane & 15);
  const int64_t row_off = (e * a.N + row) * a.K;
  const bool whole = (b + 1) * kBlockK <= a.K;
  float f[4][8];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    if (row < a.N) {
      row8<E>(a.w, row_off, b * kBlockK + 32 * s + 8 * (lane >> 4), a.K, whole, f[s]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[s][i] = 0.f;
    }
  }
  const int64_t blk = (e * a.tiles + tile) * a.blocks + b;
  constexpr int G = scales_per_block<BITS, GROUP>();
  store_block<BITS, GROUP>(f, a.codes + blk * Block<BITS>::kBytes, a.scales + blk * (16 * G), lane);
}

// w [E][K][N] (one row per input): 64 rows x 128 inputs through LDS per
// workgroup, read along N and handed out along K.
template <class E, int BITS, int GROUP>
__global__ __launch_bounds__(kPackWaves* kWave) void weights_pack_t_kernel(WeightsArgs a) {
  __shared__ float tile_f[64][kBlockK + 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n_groups = (a.tiles + 3) / 4;
  const int tg = static_cast<int>(blockIdx.x % n_groups), b = static_cast<int>(blockIdx.x / n_groups);
  const int64_t e = blockIdx.y;
  const int n = tg * 64 + lane;
  for (int i = wave; i < kBlockK; i += kPackWaves) {
    const int k = b * kBlockK + i;
    tile_f[lane][i] = (k < a.K && n < a.N) ? load_elem<E>(a.w, (e * a.K + k) * a.N + n) : 0.f;
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

// The values the planes stand for, into w [E][N][K]; one wave per block.
template <class E, int BITS, int GROUP>
__global__ __launch_bounds__(kPackWaves* kWave) void weights_unpack_kernel(WeightsArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kPackWaves + (threadIdx.x >> 6);
  if (id >= static_cast<int64_t>(a.tiles) * a.blocks) return;
  const int tile = static_cast<int>(id / a.blocks), b = static_cast<int>(id % a.blocks);
  const int64_t e = blockIdx.y;
  const int row = tile * kTileRows + (lane & 15);
  const int64_t blk = (e * a.tiles + tile) * a.blocks + b;
  constexpr int G = scales_per_block<BITS, GROUP>();
  Block<BITS> q;
  q.template load<false>(a.codes + blk * Block<BITS>::kBytes, lane);
  Scales<G> sc;
  if constexpr (BITS == 4) sc.load(a.scales + blk * (16 * G), lane);
  if (row >= a.N) return;
  const int64_t row_off = (e * a.N + row) * a.K;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    float f[8];
    if constexpr (BITS == 16) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = bf16_bits_to_f32(i & 1 ? q.c[s][i >> 1] >> 16 : q.c[s][i >> 1] & 0xffffu);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int u = static_cast<int>(__builtin_rotateright32(q.c[s], 3 + 4 * (i >> 1) + 16 * (i & 1)) & 15u);
        f[i] = static_cast<float>(u - 8) * sc.at(s * G / 4);
      }
    }
    const int k = b * kBlockK + 32 * s + 8 * (lane >> 4);
    const bool whole = k + 8 <= a.K;
    if constexpr (E::kBytes == 4) {
      float* p = static_cast<float*>(a.out) + row_off + k;
      if (whole) {
        u32x4_t lo, hi;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          lo[i] = __float_as_uint(f[i]);
          hi[i] = __float_as_uint(f[4 + i]);
        }
        *reinterpret_cast<u32x4_a4_t*>(p) = lo;
        *reinterpret_cast<u32x4_a4_t*>(p + 4) = hi;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (k + i < a.K) p[i] = f[i];
      }
    } else {
      uint16_t* p = static_cast<uint16_t*>(a.out) + row_off + k;
      if (whole) {
        u32x4_t v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = bf16_of(f[2 * j]) | (static_cast<uint32_t>(bf16_of(f[2 * j + 1])) << 16);
        *reinterpret_cast<u32x4_a2_t*>(p) = v;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (k + i < a.K) p[i] = bf16_of(f[i]);
      }
    }
  }
}

// Calls fn with the kernel instance of (element type, bits, group).
template <template <class, int, int> class K>
void dispatch(const WeightsArgs& a, int dtype, dim3 grid, hipStream_t s) {
  const dim3 block(kPackWaves * kWave);
  const bool f32 = dtype == 0;
  if (a.bits == 16) {
    K<EBf16, 16, 128>::go(a, grid, block, s);
  } else if (a.group == 32) {
    f32 ? K<EF32, 4, 32>::go(a, grid, block, s) : K<EBf16, 4, 32>::go(a, grid, block, s);
  } else if (a.group == 64) {
    f32 ? K<EF32, 4, 64>::go(a, grid, block, s) : K<EBf16, 4, 64>::go(a, grid, block, s);
  } else {
    f32 ? K<EF32, 4, 128>::go(a, grid, block, s) : K<EBf16, 4, 128>::go(a, grid, block, s);
  }
}
template <class E, int B, int G>
struct GoPack {
  static void go(const WeightsArgs& a, dim3 g, dim3 b, hipStream_t s) { weights_pack_kernel<E, B, G><<<g, b, 0, s>>>(a); }
};
template <class E, int B, int G>
struct GoPackT {
  static void go(const WeightsArgs& a, dim3 g, dim3 b, hipStream_t s) {
    weights_pack_t_kernel<E, B, G><<<g, b, 0, s>>>(a);
  }
};
template <class E, int B, int G>
struct GoUnpack {
  static void go(const WeightsArgs& a, dim3 g, dim3 b, hipStream_t s) {
    weights_unpack_kernel<E, B, G><<<g, b, 0, s>>>(a);
  }
};

dim3 block_grid(const WeightsArgs& a) {
  const int64_t n = static_cast<int64_t>(a.tiles) * a.blocks;
  return dim3(static_cast<unsigned>((n + kPackWaves - 1) / kPackWaves), static_cast<unsigned>(a.experts));
}

}  // namespace

hipError_t launch_weights_pack(const WeightsArgs& a, int dtype, bool transposed, hipStream_t s) {
  if (transposed) {
    const int64_t n = static_cast<int64_t>((a.tiles + 3) / 4) * a.blocks;
    dispatch<GoPackT>(a, dtype, dim3(static_cast<unsigned>(n), static_cast<unsigned>(a.experts)), s);
  } else {
    dispatch<GoPack>(a, dtype, block_grid(a), s);
  }
  return hipGetLastError();
}

hipError_t launch_weights_unpack(const WeightsArgs& a, int dtype, hipStream_t s) {
  dispatch<GoUnpack>(a, dtype, block_grid(a), s);
  return hipGetLastError();
}

}  // namespace twell
