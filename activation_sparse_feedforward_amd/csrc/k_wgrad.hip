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

// The rows of a workgroup: part blockIdx.z of gridDim.z of an expert's.  The
// experts with most rows go first (up to 64 experts; among more of them one weighs
// less), so that what is left at the end is short.
struct GradRows {
  int expert;
  int64_t first, last;
  float* out;  // the expert's dW, or this part's share of it
};
__device__ __forceinline__ GradRows grad_rows(const WgradArgs& a, int unit) {
  GradRows r{static_cast<int>(blockIdx.y), 0, a.T, nullptr};
  if (a.offsets) {
    const int top = static_cast<int>(a.T);
    int b = 0, n = -1;
    const int lane = threadIdx.x & 63;
    auto rows_of = [&](int e) {
      b = min(max(a.offsets[e], 0), top);
      n = min(max(a.offsets[e + 1], b), top) - b;
    };
    if (a.experts <= 64) {
      if (lane < a.experts) rows_of(lane);
      int before = 0;
      for (int e = 0; e < a.experts; ++e) {
        const int m = __builtin_amdgcn_readlane(n, e);
        before += m > n || (m == n && e < lane) ? 1 : 0;
      }
      const uint64_t mine = __ballot(lane < a.experts && before == r.expert);
      r.expert = __builtin_amdgcn_readfirstlane(__builtin_ctzll(mine));
      b = __builtin_amdgcn_readlane(b, r.expert);
      n = __builtin_amdgcn_readlane(n, r.expert);
    } else {
      rows_of(r.expert);
    }
    r.first = b;
    r.last = b + n;
  }
  const int64_t n = r.last - r.first, parts = gridDim.z;
  if (parts > 1) {
    const int64_t each = (n + parts * unit - 1) / (parts * unit) * unit, end = r.last;
    r.first = min(r.first + blockIdx.z * each, end);
    r.last = min(r.first + each, end);
  }
  r.out = (parts > 1 ? a.part : a.dw) + (static_cast<int64_t>(blockIdx.z) * a.experts + r.expert) * a.N * a.K;
  return r;
}

constexpr int kGradWaves = 4;  // 2 x 2

// One operand's tile of kTokens x COLS in LDS.
template <class E, int COLS>
struct GradTile;
template <>
struct GradTile<EBf16, 128> {
  static constexpr int kTokens = 32, kRow = 128 * 2;
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
template <int COLS>
struct GradTile<EF32, COLS> {
  static constexpr int kTokens = 32, kRow = (COLS + 16) * 4;  // 4 tokens in 4 x 16 banks
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

// fp32, and bf16 rows of less than 16 bytes: a tile of 32 F x 32 F of dW per
// workgroup, 16 F x 16 F a wave.  Many rows of fp32 are bound by its matrix
// instructions, at a sixteenth of bf16's rate (16384 rows, 2048 x 2048: 1143 us, 120
// TFLOP/s, where a library's product reaches 153; 8192 rows of 8 experts of 1024 x 2048:
// 308 us, 111), few by their starts: 777 rows of 5 experts of 1001 x 707 take 20 to 22
// us, 50 TFLOP/s, 1024 x 704 in whole tiles 20; an expert is some five steps, each
// fetched one ahead, behind the offsets.
template <class E, int F>
__global__ __launch_bounds__(kGradWaves* kWave) void wgrad_kernel(WgradArgs a) {
  using S = typename E::storage;
  constexpr int kCols = 32 * F;
  using Tl = GradTile<E, kCols>;
  __shared__ __align__(16) char lds[2][2 * Tl::kBytes];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int tiles_k = (a.K + kCols - 1) / kCols;
  const int id = xcd_run(blockIdx.x, gridDim.x);
  const int n0 = id / tiles_k * kCols, k0 = id % tiles_k * kCols;
  const GradRows r = grad_rows(a, Tl::kTokens);
  const int64_t first = r.first, last = r.last;
  const S* dy = static_cast<const S*>(a.dy);
  const S* x = static_cast<const S*>(a.x);
  constexpr int kN = Piece<E>::kN, kPieces = kCols / kN;  // of a row
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
  f32x4_t acc[F][F];
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int j = 0; j < F; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int cn = (wave >> 1) * 16 * F, ck = (wave & 1) * 16 * F;
  fetch(first);
  int turn = 0;
  for (int64_t t0 = first; t0 < last; t0 += Tl::kTokens, turn ^= 1) {
    char* stage = lds[turn];
    put(stage);  // what was read from it two turns ago was read before the last barrier
    __syncthreads();
    if (t0 + Tl::kTokens < last) fetch(t0 + Tl::kTokens);
#pragma unroll
    for (int s = 0; s < Tl::kSteps; ++s) {
      typename Tl::Frag fx[F];
#pragma unroll
      for (int j = 0; j < F; ++j) Tl::read(fx[j], stage + Tl::kBytes, ck + 16 * j, s, lane);
#pragma unroll
      for (int i = 0; i < F; ++i) {
        typename Tl::Frag fy;
        Tl::read(fy, stage, cn + 16 * i, s, lane);
        // rows of the result are x's columns, so that a lane has four of them next to each other
#pragma unroll
        for (int j = 0; j < F; ++j) Tl::mfma(acc[i][j], fx[j], fy);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < F; ++i) {
    const int n = n0 + cn + 16 * i + (lane & 15);
    if (n >= a.N) continue;
    float* row = r.out + static_cast<int64_t>(n) * a.K;
#pragma unroll
    for (int j = 0; j < F; ++j) {
      const int k = k0 + ck + 16 * j + 4 * (lane >> 4);
      if (k < a.K) store_piece<EF32>(row, k, a.K, __builtin_bit_cast(u32x4_t, acc[i][j]));
    }
  }
}

// ------------------------------------------------------------------ 256 x 256 tiles, bf16
// Steps of 32 tokens x 256 columns of dy and of x;
// a wave fetches a quarter of a step to registers four steps ahead, writes it to
// LDS two steps ahead, and reads its fragments one step ahead.  128 x 128 a wave,
// one wave a SIMD: a fragment feeds eight matrix instructions, so that LDS carries
// 96 bytes a cycle (64 x 64 a wave take 192, which bounds the kernel above).
// (Direct loads to LDS would save the registers, but the compiler waits for all of
// them before every transposed read.)  16384 rows, 8192 x 2048: 414 to 440 us, 1.25 to
// 1.33 PFLOP/s, where a library's bf16 product of 8192^3 reaches 1.38; 8191 wide, rows
// not aligned, 569 us; 16 uneven experts of 1024 x 2048 97 us: two workgroups a CU one
// after the other, each with a start and 256 KB to store that nothing overlaps.
constexpr int kWide = 256, kWideTokens = 32, kWideRow = kWide * 2;
constexpr int kWideTile = kWideTokens * kWideRow, kWideStage = 2 * kWideTile, kWideStages = 4;
constexpr int kWideLds = kWideStages * kWideStage;
constexpr int kWideLoads = kWideStage / (kGradWaves * 1024);  // of a wave and step

struct WideFrags {
  bf16x8_t y[8], x[8];
};

// WHOLE: 16 bytes of a row never cross its end, and 32 rows fit 31 bits.  Else
// they may reach into the row behind, whose values land in columns that are not
// stored; the last row, which has none behind it, is a step of its own.
template <bool WHOLE>
struct WideWork {
  const char* rows;  // what this wave fetches: the expert's first row of dy or x (WHOLE: from the tile's first column on)
  int64_t ld;        // bytes
  int n;             // tokens
  int left;          // WHOLE: bytes from the tile's first column to the end of a row
  int wave;
  uint32_t from, to;  // of a lane's 16 bytes: in a row (WHOLE: in two rows) of memory, and in a stage
  uint32_t at[8];     // of a lane's fragments in a tile, for the first 128 columns
  char* lds;

  // Memory of a step: past the last token, and past the end of its row, loads give zeros.
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t step_rows(int step) const {
    const int t0 = min(step * kWideTokens, n), count = min(n - t0, kWideTokens);
    const uint32_t bytes = count > 0 ? static_cast<uint32_t>((count - 1) * ld + left) : 0u;
    return f8_buffer(reinterpret_cast<const uint8_t*>(rows + t0 * ld), __builtin_amdgcn_readfirstlane(bytes));
  }
  // Token of a lane's load q of a wave: 2 p and 2 p + 1, p = 8 (wave % 2) + q; waves 0 and 1 of dy, 2 and 3 of x.
  __device__ __forceinline__ int token(int q, int step) const {
    return step * kWideTokens + ((wave & 1) * kWideLoads + q) * 2 + ((threadIdx.x >> 5) & 1);
  }
  __device__ __forceinline__ u32x4_t fetch(__amdgpu_buffer_rsrc_t r, int q, int step) const {
    if constexpr (WHOLE) return buffer16(r, from, ((wave & 1) * kWideLoads + q) * 2 * static_cast<uint32_t>(ld));
    else return load16(rows + min(token(q, step), n - 1) * ld + from);
  }
  // The 32-byte pieces of a row are permuted by its token (GradTile), here by 2 p modulo 8.
  template <bool ALL = WHOLE>
  __device__ __forceinline__ void put(u32x4_t v, int q, int step) const {
    if constexpr (!ALL) {
      const bool there = token(q, step) < n;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = there ? v[i] : 0;
    }
    char* p = lds + (step & (kWideStages - 1)) * kWideStage + q * 1024;
    *reinterpret_cast<u32x4_t*>(p + (to ^ (((2 * q) & 7) * 32))) = v;
  }
  // Fragment f of 8: dy's for f < 8, else x's; half h has 16 tokens.
  __device__ __forceinline__ void read(WideFrags& frags, int f, int h, int step) const {
    typedef short i16x4_t __attribute__((ext_vector_type(4)));
    struct Halves {
      i16x4_t h[2];
    };
    const int side = f < 8 ? wave >> 1 : wave & 1;
    const char* p = lds + (step & (kWideStages - 1)) * kWideStage + (f < 8 ? 0 : kWideTile) + side * 256 +
                    h * 16 * kWideRow + at[f & 7];
    bf16x8_t& v = f < 8 ? frags.y[f] : frags.x[f - 8];
    Halves b = __builtin_bit_cast(Halves, v);
    b.h[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4_t*)(p));
    v = __builtin_bit_cast(bf16x8_t, b);
  }
};

// One step: products of this one's fragments; between them the next one's are read, the one after that, fetched two
// steps ago, is written, and the one two further on is fetched.
template <bool WHOLE>
__device__ __forceinline__ void wide_step(const WideWork<WHOLE>& w, int step, const WideFrags& now, WideFrags& next,
                                          u32x4_t (&fetched)[kWideLoads], f32x4_t (&acc)[8][8]) {
  __amdgpu_buffer_rsrc_t rows;
  if constexpr (WHOLE) rows = w.step_rows(step + 4);
  // the next step's tiles are written, by all waves
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // rows of the result are x's columns, so that a lane has four of them next to each other
      acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(now.x[j], now.y[i], acc[i][j], 0, 0, 0);
      const int m = i * 8 + j;
      if (m < 32) {
        w.read(next, m / 2, m % 2, step + 1);
      } else if (m < 32 + 2 * kWideLoads) {
        const int q = (m - 32) / 2;
        if (m % 2 == 0) w.put(fetched[q], q, step + 2);
        else fetched[q] = w.fetch(rows, q, step + 4);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
}

template <bool WHOLE>
__global__ __launch_bounds__(256) void wgrad_wide_kernel(WgradArgs a) {
  extern __shared__ __align__(16) char lds_stages[];
  const int lane = threadIdx.x & 63;
  const int tiles_k = (a.K + kWide - 1) / kWide;
  const int id = xcd_run(blockIdx.x, gridDim.x);
  const int n0 = id / tiles_k * kWide, k0 = id % tiles_k * kWide;
  const GradRows r = grad_rows(a, kWideTokens);
  const int64_t first = r.first, last = r.last;
  WideWork<WHOLE> w;
  w.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool of_x = w.wave >= 2;
  w.ld = (of_x ? a.ldx : a.ldy) * 2;
  w.rows = static_cast<const char*>(of_x ? a.x : a.dy) + first * w.ld;
  w.n = static_cast<int>(last - first);
  const int width = of_x ? a.K : a.N, c0 = of_x ? k0 : n0, c = c0 + (lane & 31) * 8;
  if constexpr (WHOLE) {
    w.rows += c0 * 2;
    w.left = (width - c0) * 2;
    w.from = (lane >> 5) * static_cast<uint32_t>(w.ld) + (lane & 31) * 16;
  } else {
    w.n = max(w.n - 1, 0);
    w.from = (c < width ? c : 0) * 2;
  }
  w.lds = lds_stages;
  w.to = (of_x ? kWideTile : 0) + (w.wave & 1) * kWideLoads * 1024 + (lane >> 5) * kWideRow +
         (((lane & 31) * 16) ^ ((lane >> 5) * 32));
  const int token = 4 * (lane >> 4) + ((lane & 15) >> 2);
#pragma unroll
  for (int f = 0; f < 8; ++f) w.at[f] = token * kWideRow + (f ^ (token & 7)) * 32 + 8 * (lane & 3);

  f32x4_t acc[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int steps = (w.n + kWideTokens - 1) / kWideTokens;
  if (steps > 0) {
    WideFrags fa, fb;
    u32x4_t ra[kWideLoads], rb[kWideLoads];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      __amdgpu_buffer_rsrc_t rows;
      if constexpr (WHOLE) rows = w.step_rows(s);
#pragma unroll
      for (int q = 0; q < kWideLoads; ++q) {
        u32x4_t& v = s & 1 ? rb[q] : ra[q];
        if (s >= 2) w.put(v, q, s - 2);
        v = w.fetch(rows, q, s);
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
    for (int f = 0; f < 16; ++f)
#pragma unroll
      for (int h = 0; h < 2; ++h) w.read(fa, f, h, 0);
    for (int s = 0; s < steps; s += 2) {  // a step past the end adds zeros
      wide_step(w, s, fa, fb, ra, acc);
      wide_step(w, s + 1, fb, fa, rb, acc);
    }
  }
  if (!WHOLE && last > first) {  // the last token, alone in a step
    const uint16_t* row = reinterpret_cast<const uint16_t*>(w.rows + w.n * w.ld);
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kWideLoads; ++q) {
      u32x4_t v{0, 0, 0, 0};
      if (w.token(q, 0) == 0) v = load_piece<EBf16>(row, c, width);
      w.template put<true>(v, q, 0);
    }
    __syncthreads();
    WideFrags f;
#pragma unroll
    for (int i = 0; i < 32; ++i) w.read(f, i / 2, i % 2, 0);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.x[j], f.y[i], acc[i][j], 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int n = n0 + (w.wave >> 1) * 128 + 16 * i + (lane & 15);
    if (n >= a.N) continue;
    float* row = r.out + static_cast<int64_t>(n) * a.K;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int k = k0 + (w.wave & 1) * 128 + 16 * j + 4 * (lane >> 4);
      if (k < a.K) store_piece<EF32>(row, k, a.K, __builtin_bit_cast(u32x4_t, acc[i][j]));
    }
  }
}

// dW from its parts, in their order.
__global__ __launch_bounds__(256) void wgrad_sum_kernel(WgradArgs a) {
  const int64_t n = static_cast<int64_t>(a.experts) * a.N * a.K;
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  if (i + 4 > n) {
    for (int64_t j = i; j < n; ++j) {
      float s = 0.f;
      for (int p = 0; p < a.parts; ++p) s += a.part[p * n + j];
      a.dw[j] = s;
    }
    return;
  }
  f32x4_t s{0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int p = 0; p < a.parts; ++p) s += __builtin_bit_cast(f32x4_t, load16(a.part + p * n + i));
  store16(a.dw + i, __builtin_bit_cast(u32x4_t, s));
}

template <class E, int F>
hipError_t go_tiles(const WgradArgs& a, hipStream_t s) {
  const dim3 grid(((a.N + 32 * F - 1) / (32 * F)) * ((a.K + 32 * F - 1) / (32 * F)), a.experts, a.parts);
  return launch(wgrad_kernel<E, F>, grid, kGradWaves * kWave, 0, s, a);
}

bool whole_pieces(const void* p, int64_t ld, int width) {  // no 16 bytes cross the end of a row; 32 rows stay in 31 bits
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 8 == 0 && width % 8 == 0 && ld <= 1 << 24;
}

}  // namespace

// Parts of each expert's rows: as many as leave a workgroup for every CU, of 256
// rows at the least on average; a part costs writing and reading dW once more.
int wgrad_parts(int64_t T, int N, int K, int experts) {
  const int64_t tiles = static_cast<int64_t>((N + kWide - 1) / kWide) * ((K + kWide - 1) / kWide) * experts;
  const int64_t by_cus = 256 / tiles, by_rows = T / (256 * static_cast<int64_t>(experts));
  const int64_t n = by_cus < by_rows ? by_cus : by_rows;
  return static_cast<int>(n < 1 ? 1 : n > 16 ? 16 : n);
}

hipError_t launch_wgrad(const WgradArgs& a, int dtype, hipStream_t s) {
  hipError_t e;
  if (dtype == 1 && a.N >= 8 && a.K >= 8) {
    const dim3 grid(((a.N + kWide - 1) / kWide) * ((a.K + kWide - 1) / kWide), a.experts, a.parts);
    if (whole_pieces(a.dy, a.ldy, a.N) && whole_pieces(a.x, a.ldx, a.K))
      e = launch_lds<&wgrad_wide_kernel<true>, kWideLds>(grid, kGradWaves * kWave, kWideLds, s, a);
    else
      e = launch_lds<&wgrad_wide_kernel<false>, kWideLds>(grid, kGradWaves * kWave, kWideLds, s, a);
  } else if (dtype == 1) {
    e = go_tiles<EBf16, 4>(a, s);
  } else {
    // fp32 is bound by its matrix instructions: small tiles while there are few workgroups
    // (777 rows of 5 experts of 1001 x 707: 30 us with 128 x 128, 20 with 64 x 64)
    const int64_t tiles = static_cast<int64_t>((a.N + 127) / 128) * ((a.K + 127) / 128) * a.experts * a.parts;
    e = tiles < 1024 ? go_tiles<EF32, 2>(a, s) : go_tiles<EF32, 4>(a, s);
  }
  if (e != hipSuccess || a.parts == 1) return e;
  const int64_t n = static_cast<int64_t>(a.experts) * a.N * a.K;
  return launch(wgrad_sum_kernel, dim3(static_cast<unsigned>((n + 1023) / 1024)), 256, 0, s, a);
}

}  // namespace twell
