// Layer norm, forward and backward:
//   h = (x - mean) rstd, rstd = 1 / sqrt(var + eps);  y = h w + b
//   g = dy w;  dx = rstd (g - mean(g) - h mean(g h));  dw = sum_t dy h;  db = sum_t dy
//
// Bound by reading and writing rows once.  A row stays in registers between its
// sums and its result, so the variance is the mean of (x - mean)^2 itself, not a
// difference of two large sums.  W waves share a row, each lane holding U pieces
// of 16 bytes.  16384 rows of 2048 in bf16: forward 24.7 us (5.4 TB/s, a copy's 4.9
// and more, since part of y stays in the caches), backward 32.5 (6.2) and 5.7 for the
// sums over rows; 1999 rows of 4099 in fp32 16.7, 21.6 and 4.4.
#include "internal.hpp"
#include "launch.hpp"
#include "rows.hpp"

namespace twell {
namespace {

// Sums of the W waves' values, the same bits in every wave; one barrier.  lds
// holds W * N floats and is not reused before another barrier.
template <int W, int N>
__device__ __forceinline__ void across_waves(float (&v)[N], float* lds) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if constexpr (W > 1) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) lds[wave * N + i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) s += lds[w * N + i];
      v[i] = s;
    }
  }
}

// Weights are read as fp32 or bf16, kN of them for one piece of a row.
template <class E, class EW>
__device__ __forceinline__ void load_weights(const void* w, int c, int d, float none, float* f) {
  if (!w) {
#pragma unroll
    for (int j = 0; j < Piece<E>::kN; ++j) f[j] = none;
    return;
  }
  constexpr int kPieces = Piece<E>::kN / Piece<EW>::kN;
  const auto* p = static_cast<const typename EW::storage*>(w);
  if constexpr (kPieces >= 1) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int at = c + i * Piece<EW>::kN;
      Piece<EW>::unpack(at < d ? load_piece<EW>(p, at, d) : u32x4_t{0, 0, 0, 0}, f + i * Piece<EW>::kN);
    }
  } else {  // four fp32 elements of a row, eight bf16 weights in a piece
#pragma unroll
    for (int j = 0; j < Piece<E>::kN; ++j) f[j] = c + j < d ? load_elem<EW>(w, c + j) : 0.f;
  }
}

template <class E, class EW, int W, int U>
__global__ __launch_bounds__((W == 1 ? 4 : W) * kWave) void norm_fwd_kernel(NormArgs a) {
  using S = typename E::storage;
  using P = Piece<E>;
  constexpr int kN = P::kN;
  __shared__ float lds[2 * W];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t t = W == 1 ? static_cast<int64_t>(blockIdx.x) * 4 + wave : blockIdx.x;
  if (t >= a.T) return;
  const int part = W == 1 ? 0 : wave;
  const S* x = static_cast<const S*>(a.x) + t * a.ldx;
  const int c0 = (part * U * kWave + lane) * kN;
  constexpr int kStep = kWave * kN;
  u32x4_t raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u) raw[u] = load_piece<E>(x, c0 + u * kStep, a.d);
  float f[U][kN];
  float s[1] = {0.f};
#pragma unroll
  for (int u = 0; u < U; ++u) {
    P::unpack(raw[u], f[u]);
#pragma unroll
    for (int j = 0; j < kN; ++j) s[0] += f[u][j];
  }
  across_waves<W>(s, lds);
  const float inv_d = 1.0f / static_cast<float>(a.d);
  const float mean = s[0] * inv_d;
  float q[1] = {0.f};
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      f[u][j] = c0 + u * kStep + j < a.d ? f[u][j] - mean : 0.f;
      q[0] = fmaf(f[u][j], f[u][j], q[0]);
    }
  across_waves<W>(q, lds + W);
  const float rstd = 1.0f / sqrtf(q[0] * inv_d + a.eps);
  if (a.stats && threadIdx.x % (W * kWave) == 0) {
    a.stats[2 * t] = mean;
    a.stats[2 * t + 1] = rstd;
  }
  S* y = static_cast<S*>(a.y) + t * a.ldy;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = c0 + u * kStep;
    float w[kN], b[kN];
    load_weights<E, EW>(a.w, c, a.d, 1.f, w);
    load_weights<E, EW>(a.b, c, a.d, 0.f, b);
#pragma unroll
    for (int j = 0; j < kN; ++j) f[u][j] = fmaf(f[u][j] * rstd, w[j], b[j]);
    store_piece<E>(y, c, a.d, P::pack(f[u]));
  }
}

// A workgroup takes rows blockIdx.x, + gridDim.x, ... and keeps its share of dw
// and db in registers, which it writes to part[blockIdx.x][2][d] at the end:
// sums over tokens then take a fixed order.  The next row is on its way while one
// is summed and written.
template <class E, class EW, int W, int U>
__global__ __launch_bounds__(W* kWave) void norm_bwd_kernel(NormArgs a) {
  using S = typename E::storage;
  using P = Piece<E>;
  constexpr int kN = P::kN;
  constexpr bool kWeights = U * kN <= 12;  // kept in registers; else read again for each row, from the caches
  constexpr bool kValues = W * U < 48;     // likewise h and dy w, else worked out twice from the row's pieces
  __shared__ float lds[2][2 * W];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int c0 = (wave * U * kWave + lane) * kN;
  constexpr int kStep = kWave * kN;
  float w[kWeights ? U : 1][kN], dw[U][kN], db[U][kN];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if constexpr (kWeights) load_weights<E, EW>(a.w, c0 + u * kStep, a.d, 1.f, w[u]);
#pragma unroll
    for (int j = 0; j < kN; ++j) dw[u][j] = db[u][j] = 0.f;
  }
  const float inv_d = 1.0f / static_cast<float>(a.d);
  struct Row {
    u32x4_t x[U], g[U];
    float mean, rstd;
  };
  Row row;
  auto fetch = [&](Row& r, int64_t t) {
    if (t >= a.T) return;
    const S* x = static_cast<const S*>(a.x) + t * a.ldx;
    const S* dy = static_cast<const S*>(a.dy) + t * a.ldy;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      r.x[u] = load_piece<E>(x, c0 + u * kStep, a.d);
      r.g[u] = load_piece<E>(dy, c0 + u * kStep, a.d);
    }
    r.mean = a.stats_in[2 * t];
    r.rstd = a.stats_in[2 * t + 1];
  };
  // h and dy of piece u of a row
  auto values = [&](const Row& r, int u, float* h, float* g) {
    P::unpack(r.x[u], h);
    P::unpack(r.g[u], g);
    if constexpr (!kWeights) load_weights<E, EW>(a.w, c0 + u * kStep, a.d, 1.f, w[0]);
#pragma unroll
    for (int j = 0; j < kN; ++j) h[j] = c0 + u * kStep + j < a.d ? (h[j] - r.mean) * r.rstd : 0.f;
  };
  fetch(row, blockIdx.x);
  int turn = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1) {
    constexpr int kHeld = kValues ? U : 1;
    float h[kHeld][kN], g[kHeld][kN];
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int q = kValues ? u : 0;
      values(row, u, h[q], g[q]);
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        dw[u][j] = fmaf(g[q][j], h[q][j], dw[u][j]);
        db[u][j] += g[q][j];
        g[q][j] *= w[kWeights ? u : 0][j];
        s[0] += g[q][j];
        s[1] = fmaf(g[q][j], h[q][j], s[1]);
      }
    }
    const float r = row.rstd;
    const Row same = row;
    fetch(row, t + gridDim.x);
    across_waves<W>(s, lds[turn]);  // two turns: a wave may be one row ahead of another
    S* dx = static_cast<S*>(a.dx) + t * a.lddx;
    const float m0 = s[0] * inv_d, m1 = s[1] * inv_d;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int q = kValues ? u : 0;
      if constexpr (!kValues) {
        values(same, u, h[0], g[0]);
#pragma unroll
        for (int j = 0; j < kN; ++j) g[0][j] *= w[kWeights ? u : 0][j];
      }
#pragma unroll
      for (int j = 0; j < kN; ++j) g[q][j] = r * (g[q][j] - m0 - h[q][j] * m1);
      store_piece<E>(dx, c0 + u * kStep, a.d, P::pack(g[q]));
    }
  }
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.d;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = c0 + u * kStep;
#pragma unroll
    for (int i = 0; i < kN; i += 4) {
      if (c + i >= a.d) continue;
      store_piece<EF32>(part, c + i, a.d, Piece<EF32>::pack(dw[u] + i));
      store_piece<EF32>(part + a.d, c + i, a.d, Piece<EF32>::pack(db[u] + i));
    }
  }
}

// dw and db: column sums of part, parts in a fixed order.
constexpr int kSumWaves = 16;
__global__ __launch_bounds__(kSumWaves* kWave) void norm_sum_kernel(NormArgs a) {
  __shared__ float lds[kSumWaves][kWave];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t width = 2 * static_cast<int64_t>(a.d);
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kWave + lane;
  float s = 0.f;
  if (c < width) {
#pragma unroll 8
    for (int b = wave; b < a.blocks; b += kSumWaves) s += a.part[b * width + c];
  }
  lds[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < width) {
    s = 0.f;
#pragma unroll
    for (int w = 0; w < kSumWaves; ++w) s += lds[w][lane];
    float* out = c < a.d ? a.dw : a.db;
    if (out) out[c < a.d ? c : c - a.d] = s;
  }
}

template <class E, class EW>
hipError_t go_fwd(const NormArgs& a, hipStream_t s) {
  constexpr int kOne = kWave * Piece<E>::kN;  // elements of one wave's 1 KB
  const unsigned T = static_cast<unsigned>(a.T);
  if (a.d <= 4 * kOne) {
    if (a.d <= kOne) return launch(norm_fwd_kernel<E, EW, 1, 1>, dim3((T + 3) / 4), 4 * kWave, 0, s, a);
    if (a.d <= 2 * kOne) return launch(norm_fwd_kernel<E, EW, 1, 2>, dim3((T + 3) / 4), 4 * kWave, 0, s, a);
    return launch(norm_fwd_kernel<E, EW, 1, 4>, dim3((T + 3) / 4), 4 * kWave, 0, s, a);
  }
  if (a.d <= 8 * kOne) return launch(norm_fwd_kernel<E, EW, 4, 2>, dim3(T), 4 * kWave, 0, s, a);
  if (a.d <= 16 * kOne) return launch(norm_fwd_kernel<E, EW, 4, 4>, dim3(T), 4 * kWave, 0, s, a);
  if constexpr (32 * kOne < kNormMostWidth)
    if (a.d > 32 * kOne) return launch(norm_fwd_kernel<E, EW, 16, 4>, dim3(T), 16 * kWave, 0, s, a);
  return launch(norm_fwd_kernel<E, EW, 16, 2>, dim3(T), 16 * kWave, 0, s, a);
}
template <class E, class EW>
hipError_t go_rows_bwd(const NormArgs& a, hipStream_t s) {
  constexpr int kOne = kWave * Piece<E>::kN;
  const dim3 grid(a.blocks);
  if (a.d <= kOne) return launch(norm_bwd_kernel<E, EW, 1, 1>, grid, 1 * kWave, 0, s, a);
  if (a.d <= 2 * kOne) return launch(norm_bwd_kernel<E, EW, 2, 1>, grid, 2 * kWave, 0, s, a);
  if (a.d <= 4 * kOne) return launch(norm_bwd_kernel<E, EW, 4, 1>, grid, 4 * kWave, 0, s, a);
  if (a.d <= 8 * kOne) return launch(norm_bwd_kernel<E, EW, 8, 1>, grid, 8 * kWave, 0, s, a);
  if (a.d <= 16 * kOne) return launch(norm_bwd_kernel<E, EW, 16, 1>, grid, 16 * kWave, 0, s, a);
  if constexpr (E::kBytes == 2) {  // 16 waves have too few registers for two pieces of bf16
    if (a.d <= 24 * kOne) return launch(norm_bwd_kernel<E, EW, 8, 3>, grid, 8 * kWave, 0, s, a);
    return launch(norm_bwd_kernel<E, EW, 8, 4>, grid, 8 * kWave, 0, s, a);
  } else {
    if (a.d <= 32 * kOne) return launch(norm_bwd_kernel<E, EW, 16, 2>, grid, 16 * kWave, 0, s, a);
    if (a.d <= 48 * kOne) return launch(norm_bwd_kernel<E, EW, 16, 3>, grid, 16 * kWave, 0, s, a);
    return launch(norm_bwd_kernel<E, EW, 16, 4>, grid, 16 * kWave, 0, s, a);
  }
}
template <class E, class EW>
hipError_t go_bwd(const NormArgs& a, hipStream_t s) {
  const hipError_t e = a.blocks ? go_rows_bwd<E, EW>(a, s) : hipSuccess;  // no rows: dw and db are zeros
  if (e != hipSuccess || (!a.dw && !a.db)) return e;
  return launch(norm_sum_kernel, dim3((2 * a.d + kWave - 1) / kWave), kSumWaves * kWave, 0, s, a);
}

}  // namespace

// Workgroups of the backward kernel.  Each writes 2 d sums, which norm_sum_kernel
// reads: more of them cost more there, fewer have fewer loads under way.  (16384
// rows in bf16 with 256, 512, 1024 and 2048, us: 600 wide, 2 waves a row, 79, 46, 29.6,
// 26; 1024 wide 44, 31, 25, 28.5; 1500 wide, 3 waves, 114, 65, 44, 49; 2048 wide, 4 waves,
// 48.6, 37.1, 38.9, 46; of 4096, 8 waves: 79 with 256, 81 with 512.  2000 rows of 2048: 12.8
// with 256, 14.8 with 512.)
int norm_blocks(int64_t T, int d, int dtype) {
  const int waves = (d + (dtype == 1 ? 511 : 255)) / (dtype == 1 ? 512 : 256);  // of a row, with one piece a lane
  const int64_t most = waves == 1 ? 2048 : waves <= 4 ? 1024 : 256, wanted = waves <= 4 ? (T + 3) / 4 : (T + 1) / 2;
  return static_cast<int>(wanted < most ? wanted : most);
}

hipError_t launch_norm_fwd(const NormArgs& a, int dtype, int w_dtype, hipStream_t s) {
  if (dtype == 1) return w_dtype == 1 ? go_fwd<EBf16, EBf16>(a, s) : go_fwd<EBf16, EF32>(a, s);
  return w_dtype == 1 ? go_fwd<EF32, EBf16>(a, s) : go_fwd<EF32, EF32>(a, s);
}
hipError_t launch_norm_bwd(const NormArgs& a, int dtype, int w_dtype, hipStream_t s) {
  if (dtype == 1) return w_dtype == 1 ? go_bwd<EBf16, EBf16>(a, s) : go_bwd<EBf16, EF32>(a, s);
  return w_dtype == 1 ? go_bwd<EF32, EBf16>(a, s) : go_bwd<EF32, EF32>(a, s);
}

}  // namespace twell
