// dW_e = dy^T x over expert e's rows, from the values themselves, fp32 sums.
//
// Both operands are wanted along their rows (tokens), which memory has apart:
// bf16 tiles stay in LDS as they come, [token][column], and ds_read_b64_tr_b16
// reads them across: 16 lanes give the addresses of 4 tokens x 16 columns, lane i
// gets column i of the 4 tokens.  fp32 needs one value a lane, which any LDS
// read gives.
#include "fp8.hpp"
#include "launch.hpp"
#include "rows.hpp"

namespace twell {
namespace {

constexpr int kGradWaves = 4;  // 2 x 2

// One operand's tile of kTokens x kCols in LDS.
template <class E>
struct GradTile;
template <>
struct GradTile<EBf16> {
  static constexpr int kTokens = 32, kCols = 128, kRow = kCols * 2;
  static constexpr int kBytes = kTokens * kRow;
  // 32-byte pieces of a row are permuted by its token: a read takes 4 tokens a
  // lane group, and those of two groups then lie in different banks
  static __device__ __forceinline__ int at(int token, int col) {
    const int byte = col * 2;
    return token * kRow + ((byte >> 5) ^ (token & 7)) * 32 + (byte & 31);
  }
  struct Frag {
    bf16x8_t v;
  };
  // 16 columns from col0, 32 tokens: slot g of a lane group g has tokens 4 g .. 4 g + 3 and 16 + those
  static __device__ __forceinline__ void read(Frag& f, const char* lds, int col0, int, int lane) {
    typedef short i16x4_t __attribute__((ext_vector_type(4)));
    const int i = lane & 15, g = lane >> 4;
    i16x4_t h[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const char* p = lds + at(16 * s + 4 * g + (i >> 2), col0 + 4 * (i & 3));
      h[s] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4_t*)(p));
    }
    struct Both {
      i16x4_t a, b;
    };
    f.v = __builtin_bit_cast(bf16x8_t, Both{h[0], h[1]});
  }
  static constexpr int kSteps = 1;  // matrix instructions per tile of tokens
  static __device__ __forceinline__ void mfma(f32x4_t& acc, const Frag& a, const Frag& b) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, acc, 0, 0, 0);
  }
};
template <>
struct GradTile<EF32> {
  static constexpr int kTokens = 32, kCols = 128, kRow = (kCols + 16) * 4;  // 4 tokens in 4 x 16 banks
  static constexpr int kBytes = kTokens * kRow;
  static __device__ __forceinline__ int at(int token, int col) { return token * kRow + col * 4; }
  struct Frag {
    float v;
  };
  static __device__ __forceinline__ void read(Frag& f, const char* lds, int col0, int step, int lane) {
    f.v = *reinterpret_cast<const float*>(lds + at(4 * step + (lane >> 4), col0 + (lane & 15)));
  }
  static constexpr int kSteps = 8;
  static __device__ __forceinline__ void mfma(f32x4_t& acc, const Frag& a, const Frag& b) {
    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v, b.v, acc, 0, 0, 0);
  }
};

// A 128 x 128 tile of dW per workgroup, 64 x 64 a wave.
template <class E>
__global__ __launch_bounds__(kGradWaves* kWave) void wgrad_kernel(WgradArgs a) {
  using S = typename E::storage;
  using Tl = GradTile<E>;
  __shared__ __align__(16) char lds[2][2 * Tl::kBytes];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = blockIdx.y;
  const int tiles_k = (a.K + 127) / 128;
  const int id = xcd_run(blockIdx.x, gridDim.x);
  const int n0 = id / tiles_k * 128, k0 = id % tiles_k * 128;
  int64_t first = 0, last = a.T;
  if (a.offsets) {
    const int top = static_cast<int>(a.T);
    const int b = min(max(a.offsets[e], 0), top);
    first = b;
    last = min(max(a.offsets[e + 1], b), top);
  }
  const S* dy = static_cast<const S*>(a.dy);
  const S* x = static_cast<const S*>(a.x);
  constexpr int kN = Piece<E>::kN, kPieces = Tl::kCols / kN;  // of a row
  constexpr int kEach = Tl::kTokens * kPieces / (kGradWaves * kWave);
  u32x4_t v[2][kEach];
  auto fetch = [&](int64_t t0) {
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int q = i * kGradWaves * kWave + threadIdx.x;
      const int64_t t = t0 + q / kPieces;
      const int c = q % kPieces * kN;
      v[0][i] = v[1][i] = u32x4_t{0, 0, 0, 0};
      if (t < last) {
        v[0][i] = load_piece<E>(dy + t * a.ldy, n0 + c, a.N);
        v[1][i] = load_piece<E>(x + t * a.ldx, k0 + c, a.K);
      }
    }
  };
  auto put = [&](char* stage) {
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int q = i * kGradWaves * kWave + threadIdx.x;
      const int at = Tl::at(q / kPieces, q % kPieces * kN);
      *reinterpret_cast<u32x4_t*>(stage + at) = v[0][i];
      *reinterpret_cast<u32x4_t*>(stage + Tl::kBytes + at) = v[1][i];
    }
  };
  f32x4_t acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int cn = (wave >> 1) * 64, ck = (wave & 1) * 64;
  fetch(first);
  int turn = 0;
  for (int64_t t0 = first; t0 < last; t0 += Tl::kTokens, turn ^= 1) {
    char* stage = lds[turn];
    put(stage);  // what was read from it two turns ago was read before the last barrier
    __syncthreads();
    if (t0 + Tl::kTokens < last) fetch(t0 + Tl::kTokens);
#pragma unroll
    for (int s = 0; s < Tl::kSteps; ++s) {
      typename Tl::Frag fx[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) Tl::read(fx[j], stage + Tl::kBytes, ck + 16 * j, s, lane);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        typename Tl::Frag fy;
        Tl::read(fy, stage, cn + 16 * i, s, lane);
        // rows of the result are x's columns, so that a lane has four of them next to each other
#pragma unroll
        for (int j = 0; j < 4; ++j) Tl::mfma(acc[i][j], fx[j], fy);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = n0 + cn + 16 * i + (lane & 15);
    if (n >= a.N) continue;
    float* row = a.dw + (static_cast<int64_t>(e) * a.N + n) * a.K;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = k0 + ck + 16 * j + 4 * (lane >> 4);
      if (k < a.K) store_piece<EF32>(row, k, a.K, __builtin_bit_cast(u32x4_t, acc[i][j]));
    }
  }
}

}  // namespace

hipError_t launch_wgrad(const WgradArgs& a, int dtype, hipStream_t s) {
  const dim3 grid(((a.N + 127) / 128) * ((a.K + 127) / 128), a.experts);
  return dtype == 1 ? launch(wgrad_kernel<EBf16>, grid, kGradWaves * kWave, 0, s, a)
                    : launch(wgrad_kernel<EF32>, grid, kGradWaves * kWave, 0, s, a);
}

}  // namespace twell
