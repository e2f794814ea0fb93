// y = Q(x) Q(W)^T: rows and weights in e4m3 (fp8.hpp), one matrix or one per
// expert over sorted rows.
#include "fp8.hpp"
#include "launch.hpp"
#include "rows.hpp"

namespace twell {
namespace {

// A fragment: one lane's 32 codes.
struct F8Frag {
  u32x4_t v[2];
  __device__ __forceinline__ void read(const uint8_t* at) {  // the block + 16 lane
    v[0] = *reinterpret_cast<const u32x4_t*>(at);
    v[1] = *reinterpret_cast<const u32x4_t*>(at + 1024);
  }
};

// acc += a b over 128 inputs, w = weights (rows of the result), x = tokens
// (columns).  sw, sx: scale bytes in bits 0..7.
__device__ __forceinline__ void f8_mfma(f32x4_t& acc, const F8Frag& w, uint32_t sw, const F8Frag& x, uint32_t sx) {
  i32x8_t a, b;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a[i] = static_cast<int>(w.v[i / 4][i % 4]);
    b[i] = static_cast<int>(x.v[i / 4][i % 4]);
  }
  acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, 0, 0, 0, static_cast<int>(sw), 0,
                                                         static_cast<int>(sx));
}

// The codes as bf16 values, scales and all: exact, but below 2^-126.
struct Bf16Frag {
  bf16x8_t v[4];
  __device__ __forceinline__ void from(const F8Frag& f, uint32_t byte) {
    const float scale = f8_scale(byte & 255u);
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t c = f.v[s / 2][2 * (s % 2) + i / 2];
        const bf16x2_t p = i % 2 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, scale, true)
                                 : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, scale, false);
        v[s][2 * i] = p[0];
        v[s][2 * i + 1] = p[1];
      }
  }
};
__device__ __forceinline__ void bf16_mfma(f32x4_t& acc, const Bf16Frag& w, const Bf16Frag& x) {
#pragma unroll
  for (int s = 0; s < 4; ++s) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[s], x.v[s], acc, 0, 0, 0);
}

// Register r of lane l of an accumulator: weight row 4 (l / 16) + r, token l % 16.
template <class E, class Args>
__device__ __forceinline__ void store_acc(const Args& a, int64_t row, int n, const f32x4_t& acc) {
  using S = typename E::storage;
  S* y = static_cast<S*>(a.y) + row * a.ldy + n;
  if (n + 4 <= a.N) {
    if constexpr (E::kBytes == 2) {
      typedef uint32_t u32x2_any_t __attribute__((ext_vector_type(2), aligned(2)));
      *reinterpret_cast<u32x2_any_t*>(y) = u32x2_any_t{bf16_pair(acc[0], acc[1]), bf16_pair(acc[2], acc[3])};
    } else {
      store16(y, __builtin_bit_cast(u32x4_t, acc));
    }
    return;
  }
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if (n + r < a.N) {
      if constexpr (E::kBytes == 2) y[r] = static_cast<uint16_t>(bf16_pair(acc[r], 0.f));
      else y[r] = acc[r];
    }
}

// The same for four tiles of weights next to each other, all in the matrix, in bf16:
// lane group g gives its quarter of every tile for tile g whole, so that a lane has 16
// outputs in a row, two stores, and four lanes a line of 128 bytes (16384 x 8192 of
// 512 and 2048 inputs: 130 and 291 us with four stores of 8 bytes, 112 and 272 so).
template <bool PAST, class Args>
__device__ __forceinline__ void store_four_acc(const Args& a, int64_t row, int n, const f32x4_t (&acc)[4], bool live) {
  u32x4_t out[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = bf16_pair(acc[i][2 * h], acc[i][2 * h + 1]);
    const auto even = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
    const auto odd = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
    const auto low = __builtin_amdgcn_permlane16_swap(even[0], odd[0], false, false);
    const auto high = __builtin_amdgcn_permlane16_swap(even[1], odd[1], false, false);
    out[0][h] = low[0];
    out[0][2 + h] = low[1];
    out[1][h] = high[0];
    out[1][2 + h] = high[1];
  }
  if (!live) return;  // lanes without a row took part above
  uint16_t* y = static_cast<uint16_t*>(a.y) + row * a.ldy + n + 16 * ((threadIdx.x & 63) >> 4);
  if constexpr (PAST) {
    store16_past(y, out[0]);
    store16_past(y + 8, out[1]);
  } else {
    store16(y, out[0]);
    store16(y + 8, out[1]);
  }
}

// ------------------------------------------------------------------ many rows
// What a workgroup of four waves works on: tiles of 16 kW weight rows x 16 kX rows.
template <int kW, int kX>
struct F8Work {
  F8Place p;
  int w0;                          // first tile of weight rows
  int w_last, x_last;              // last tiles that exist, of the matrix and of the rows from p.row0 on
  const uint8_t *w_codes, *w_scales;  // of the expert's tile 0
  const uint8_t *x_codes, *x_scales;  // of p.tile16

  __device__ __forceinline__ bool init(const F8GemmArgs& a) {
    // groups of 8 tiles of rows, all tiles of weights of a group in a row
    const int nt = (a.tiles + kW - 1) / kW;
    const int id = xcd_run(blockIdx.x, gridDim.x);
    const int mts = gridDim.x / nt, group = id / (8 * nt), first = group * 8, size = min(8, mts - first);
    const int in = id - group * 8 * nt, mt = first + in % size;
    p = f8_locate(a.offsets, a.experts, a.T, 16 * kX, mt);
    if (p.expert < 0 || p.tile16 + min(p.tiles16, kX) > a.most_tiles) return false;
    w0 = in / size * kW;
    w_last = a.tiles - 1;
    x_last = p.tiles16 - 1;
    w_codes = a.w_codes + static_cast<int64_t>(p.expert) * a.tiles * a.blocks * kF8Bytes;
    w_scales = a.w_scales + static_cast<int64_t>(p.expert) * a.tiles * a.quads * kF8Scales;
    x_codes = a.x_codes + p.tile16 * a.blocks * kF8Bytes;
    x_scales = a.x_scales + p.tile16 * a.quads * kF8Scales;
    return true;
  }
  // tiles past the matrix or the expert's rows are the last one again; their results are not stored
  __device__ __forceinline__ int w_tile(int i) const { return min(w0 + i, w_last); }
  __device__ __forceinline__ int x_tile(int i) const { return min(i, x_last); }
  template <class E, bool PAST = false, int FW, int FX>
  __device__ __forceinline__ void store(const F8GemmArgs& a, int fw0, int fx0, const f32x4_t (&acc)[FW][FX]) const {
    const int lane = threadIdx.x & 63;
    if constexpr (E::kBytes == 2 && FW == 4) {
      if ((w0 + fw0 + 4) * 16 <= a.N) {
#pragma unroll
        for (int j = 0; j < FX; ++j) {
          const f32x4_t four[4] = {acc[0][j], acc[1][j], acc[2][j], acc[3][j]};
          const int r = (fx0 + j) * 16 + (lane & 15);
          store_four_acc<PAST>(a, p.row0 + r, (w0 + fw0) * 16, four, r < p.rows);
        }
        return;
      }
    }
#pragma unroll
    for (int j = 0; j < FX; ++j) {
      const int r = (fx0 + j) * 16 + (lane & 15);
      if (r >= p.rows) continue;
#pragma unroll
      for (int i = 0; i < FW; ++i) {
        const int n = (w0 + fw0 + i) * 16 + 4 * (lane >> 4);
        if (n < a.N) store_acc<E>(a, p.row0 + r, n, acc[i][j]);
      }
    }
  }
};

// bf16 results.  A wave has 64 weight rows of its own, whose codes go from memory to
// registers, one block (128 inputs) ahead, and all 16 FX rows of the workgroup,
// whose codes go to LDS with direct loads, three blocks ahead, and from there to
// registers three fragments ahead.  So a fragment from LDS feeds four matrix
// instructions and LDS carries 2 KB for 131 k operations of each wave: with both
// operands in LDS and 64 x 64 a wave it would be twice that, which bounds it (16384
// rows of 2048 through 8192 x 2048, with rounding the rows: 352 us so, 249 to 258 as
// it is; 256 x 256 tiles with one workgroup a CU 367).  The product alone takes some
// 230 us, 2.4 PFLOP/s, of 8192 inputs 825, 2.7; the matrix cores are busy for two
// thirds of the time, at a clock of 1.5 to 1.8 GHz that their power sets, and
// with all loads in an L2 it would be 7 % faster.
template <int FX, bool PAST>  // PAST: results past the caches
struct F8Gemm {
  static constexpr int kStages = 4, kStage = FX * kF8Bytes, kLds = kStages * kStage;
  static constexpr int kLoads = FX / 2;  // direct loads of a wave and block, 1 KB each
  static_assert(kLoads <= 8, "a wait for all but kLoads covers what came before a block's eight loads of weights");

  const F8GemmArgs& a;
  F8Work<16, FX> work;
  int lane, wave;
  __amdgpu_buffer_rsrc_t w_rows, x_rows, w_words, x_words;
  uint32_t w_from[4], x_from[kLoads];  // at block 0
  uint8_t* lds;
  f32x4_t acc[4][FX];
  F8Frag x[4];  // ring

  __device__ __forceinline__ void fetch_x(int q, int kb, uint8_t* stage) {
    direct16(x_rows, lane * 16, x_from[q] + kb * kF8Bytes, stage + (wave * kLoads + q) * 1024);
  }
  __device__ __forceinline__ void fetch_w(F8Frag& w, int i, int half, int kb) {
    w.v[half] = buffer16(w_rows, lane * 16, w_from[i] + kb * kF8Bytes + half * 1024);
  }
  struct Words {
    uint32_t w, x[FX];  // scales of four blocks: 128 rows of weights, which a wave's lie in, share theirs
  };
  __device__ __forceinline__ void fetch_words(Words& s, int q) {
    s.w = buffer4(w_words, (lane & 15) * 4, q * kF8Scales);
#pragma unroll
    for (int j = 0; j < FX; ++j)
      s.x[j] = buffer4(x_words, (lane & 15) * 4, static_cast<uint32_t>(work.x_tile(j)) * a.quads * kF8Scales + q * kF8Scales);
  }
  // One block, with everything else that has to happen meanwhile dealt out between
  // the matrix instructions (sched_barrier pins the order: with one wave a SIMD
  // anything issued in clumps leaves the matrix core idle).  FIRST: of four; it
  // fetches the next four's scales, ahead of what the next block waits for.
  template <bool FIRST>
  __device__ __forceinline__ void block(int kb, const F8Frag (&w)[4], F8Frag (&w_next)[4], const Words& s, Words& s_next) {
    // of what this wave has fetched only the last block's rows may still be under way, so the next block's are
    // there; and all waves are done with the block before this one, whose place is filled now
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(kLoads) : "memory");
    __builtin_amdgcn_sched_barrier(0);
    const uint8_t* here = lds + (kb & 3) * kStage + lane * 16;
    const uint8_t* next = lds + ((kb + 1) & 3) * kStage + lane * 16;
    // past the end: the last block again, not used (a branch here would move matrix instructions)
    const int kw = min(kb + 1, a.blocks - 1), kx = min(kb + 3, a.blocks - 1);
    uint8_t* fill = lds + ((kb + 3) & 3) * kStage;
    if constexpr (FIRST) {
      fetch_words(s_next, min((kb >> 2) + 1, a.quads - 1));
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int j = 0; j < FX; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f8_mfma(acc[i][j], w[i], s.w, x[j % 4], s.x[j]);
        if (i == 0) x[(j + 3) % 4].read(j + 3 < FX ? here + (j + 3) * kF8Bytes : next + (j + 3 - FX) * kF8Bytes);
        else if (j * 3 + i - 1 < 8) fetch_w(w_next[(j * 3 + i - 1) / 2], (j * 3 + i - 1) / 2, (j * 3 + i - 1) % 2, kw);
        else if (j * 3 + i - 9 < kLoads) fetch_x(j * 3 + i - 9, kx, fill);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }

  __device__ __forceinline__ void run() {
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int blocks = a.blocks, quads = a.quads;
    w_rows = f8_buffer(work.w_codes + static_cast<int64_t>(work.w0) * blocks * kF8Bytes);
    x_rows = f8_buffer(work.x_codes);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w_from[i] = static_cast<uint32_t>(work.w_tile(4 * wave + i) - work.w0) * blocks * kF8Bytes;
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      const int half = wave * kLoads + q;
      x_from[q] = static_cast<uint32_t>(work.x_tile(half >> 1)) * blocks * kF8Bytes + (half & 1) * 1024;
    }
    w_words = f8_buffer(work.w_scales + static_cast<int64_t>(work.w_tile(4 * wave)) * quads * kF8Scales);
    x_words = f8_buffer(work.x_scales);
    F8Frag wa[4], wb[4];
    Words words, words_next;
    fetch_words(words_next, 0);
#pragma unroll
    for (int q = 0; q < kLoads; ++q) fetch_x(q, 0, lds);
#pragma unroll
    for (int q = 0; q < 8; ++q) fetch_w(wa[q / 2], q / 2, q % 2, 0);
#pragma unroll
    for (int kb = 1; kb < 3; ++kb)
#pragma unroll
      for (int q = 0; q < kLoads; ++q) fetch_x(q, min(kb, blocks - 1), lds + kb * kStage);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < FX; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
    for (int j = 0; j < 3; ++j) x[j].read(lds + lane * 16 + j * kF8Bytes);
    // four blocks at a time, whose scales share words
    for (int kb0 = 0; kb0 < blocks; kb0 += 4) {
      words = words_next;
      block<true>(kb0, wa, wb, words, words_next);
      const int end = min(kb0 + 4, blocks);
#pragma nounroll
      for (int kb = kb0 + 1; kb < end; ++kb) {
        words.w >>= 8;
#pragma unroll
        for (int j = 0; j < FX; ++j) words.x[j] >>= 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) wa[i] = wb[i];
        block<false>(kb, wa, wb, words, words_next);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) wa[i] = wb[i];
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load is still on its way to LDS when the workgroup ends
    work.template store<EBf16, PAST>(a, 4 * wave, 0, acc);
  }
};

template <int FX, bool PAST>
__global__ __launch_bounds__(256, 2) void f8_gemm_kernel(F8GemmArgs a) {
  extern __shared__ __align__(16) uint8_t lds_tiles[];
  F8Gemm<FX, PAST> g{a};
  if (!g.work.init(a)) return;
  g.lds = lds_tiles;
  g.run();
}

// fp32 results: codes widened to bf16, four instructions a block.  2 x 2 waves of 64 x 64, both operands through
// LDS in two stages.  Widening is 128 conversions beside 64 matrix instructions of a wave and block: 8192 rows of 8
// experts of 1024 x 2048 take 72 us with their rounding.
constexpr int kExactTiles = 8;  // of 16 weight rows, and of 16 rows
constexpr int kExactStage = 2 * kExactTiles * kF8Bytes;
__global__ __launch_bounds__(256) void f8_gemm_exact_kernel(F8GemmArgs a) {
  constexpr int F = kExactTiles / 2, kLoads = kExactStage / 4096;  // of a wave
  extern __shared__ __align__(16) uint8_t lds_tiles[];
  F8Work<kExactTiles, kExactTiles> work;
  if (!work.init(a)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fw0 = (wave >> 1) * F, fx0 = (wave & 1) * F;
  // waves 0 and 1 fetch weights, 2 and 3 rows
  const bool of_w = wave < 2;
  const auto from = f8_buffer(of_w ? work.w_codes + static_cast<int64_t>(work.w0) * a.blocks * kF8Bytes : work.x_codes);
  uint32_t at[kLoads];
#pragma unroll
  for (int q = 0; q < kLoads; ++q) {
    const int half = (wave & 1) * kLoads + q, t = half >> 1;
    at[q] = static_cast<uint32_t>(of_w ? work.w_tile(t) - work.w0 : work.x_tile(t)) * a.blocks * kF8Bytes + (half & 1) * 1024;
  }
  auto fetch = [&](int kb) {
#pragma unroll
    for (int q = 0; q < kLoads; ++q)
      direct16(from, lane * 16, at[q] + kb * kF8Bytes, lds_tiles + (kb & 1) * kExactStage + (wave * kLoads + q) * 1024);
  };
  f32x4_t acc[F][F];
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int j = 0; j < F; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  uint32_t sw = 0, sx[F];
  fetch(0);
  for (int kb = 0; kb < a.blocks; ++kb) {
    const uint8_t* stage = lds_tiles + (kb & 1) * kExactStage + lane * 16;
    if ((kb & 3) == 0) {
      const int q = kb >> 2;
      sw = *reinterpret_cast<const uint32_t*>(work.w_scales +
                                              (static_cast<int64_t>(work.w_tile(fw0)) * a.quads + q) * kF8Scales);
#pragma unroll
      for (int j = 0; j < F; ++j)
        sx[j] = *reinterpret_cast<const uint32_t*>(
            work.x_scales + (static_cast<int64_t>(work.x_tile(fx0 + j)) * a.quads + q) * kF8Scales + (lane & 15) * 4);
    } else {
      sw >>= 8;
#pragma unroll
      for (int j = 0; j < F; ++j) sx[j] >>= 8;
    }
    // this stage is there, and all waves' reads of the one that is filled next have come back
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (kb + 1 < a.blocks) fetch(kb + 1);
    Bf16Frag xb[F];
#pragma unroll
    for (int j = 0; j < F; ++j) {
      F8Frag x;
      x.read(stage + (kExactTiles + fx0 + j) * kF8Bytes);
      xb[j].from(x, sx[j]);
    }
#pragma unroll
    for (int i = 0; i < F; ++i) {
      F8Frag w;
      w.read(stage + (fw0 + i) * kF8Bytes);
      Bf16Frag wb;
      wb.from(w, sw);
#pragma unroll
      for (int j = 0; j < F; ++j) bf16_mfma(acc[i][j], wb, xb[j]);
    }
  }
  work.template store<EF32>(a, fw0, fx0, acc);
}

// ------------------------------------------------------------------ few rows
// With few rows for each expert what counts is reading the weights once, at
// memory's rate, and one trip to memory where they are few too: weights go from
// memory to the matrix core's registers, without LDS.  A workgroup has 16 MT rows
// and 16 NT weight rows; its waves take turns at the blocks of inputs and add
// their sums through LDS, in the order of the waves.  A wave fetches two blocks
// of weights, and the rows' inputs, before it uses the first.
// CODES: rows come as codes; else each wave rounds the inputs that it needs
// itself, which saves a launch and costs each workgroup the rounding again.
constexpr int kFewAhead = 2;

template <class E, int MT, int NT, bool CODES, int WAVES>
__global__ __launch_bounds__(WAVES* kWave) void f8_few_kernel(F8GemmArgs a) {
  using S = typename E::storage;
  extern __shared__ __align__(16) float lds_sums[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const F8Place p = f8_locate(a.offsets, a.experts, a.T, 16 * MT, blockIdx.y);
  if (p.expert < 0 || (CODES && p.tile16 + min(p.tiles16, MT) > a.most_tiles)) return;
  const int tile0 = blockIdx.x * NT, r = lane & 15;
  const S* row[MT];
  const uint8_t *xcodes[MT], *xscales[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    if constexpr (CODES) {
      const int64_t t = p.tile16 + min(m, p.tiles16 - 1);
      xcodes[m] = a.x_codes + t * a.blocks * kF8Bytes + lane * 16;
      xscales[m] = a.x_scales + t * a.quads * kF8Scales + r * 4;
    } else {
      row[m] = static_cast<const S*>(a.x) + (p.row0 + (16 * m + r < p.rows ? 16 * m + r : 0)) * a.ldx;
    }
  }
  const uint8_t *codes[NT], *scales[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    // a tile past the matrix is the last one again; its results are not stored
    const int64_t t = static_cast<int64_t>(p.expert) * a.tiles + min(tile0 + i, a.tiles - 1);
    codes[i] = a.w_codes + t * a.blocks * kF8Bytes + lane * 16;
    scales[i] = a.w_scales + t * a.quads * kF8Scales + r * 4;
  }
  f32x4_t acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[m][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int b0 = wave; b0 < a.blocks; b0 += waves * kFewAhead) {
    F8Frag w[kFewAhead][NT], xc[kFewAhead][MT];
    uint32_t sw[kFewAhead][NT], sx[kFewAhead][MT];
    F8Inputs<E> in[kFewAhead][MT];
#pragma unroll
    for (int u = 0; u < kFewAhead; ++u) {
      const int b = b0 + u * waves;
      if (b < a.blocks) {
        const int64_t at = static_cast<int64_t>(b) * kF8Bytes;
        const int scale = (b >> 2) * kF8Scales + (b & 3);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          w[u][i].read(codes[i] + at);
          sw[u][i] = scales[i][scale];
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          if constexpr (CODES) {
            xc[u][m].read(xcodes[m] + at);
            sx[u][m] = xscales[m][scale];
          } else {
            in[u][m].load(row[m], b * kF8Block, lane, a.K);
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kFewAhead; ++u) {
      if (b0 + u * waves >= a.blocks) break;
      Bf16Frag wb[NT];
      if constexpr (E::kBytes == 4) {
#pragma unroll
        for (int i = 0; i < NT; ++i) wb[i].from(w[u][i], sw[u][i]);
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if constexpr (!CODES) {
          sx[u][m] = f8_scale_byte(max_over_row(in[u][m].most()));
          in[u][m].codes(f8_scale(sx[u][m]), xc[u][m].v);
        }
        if constexpr (E::kBytes == 4) {
          Bf16Frag xb;
          xb.from(xc[u][m], sx[u][m]);
#pragma unroll
          for (int i = 0; i < NT; ++i) bf16_mfma(acc[m][i], wb[i], xb);
        } else {
#pragma unroll
          for (int i = 0; i < NT; ++i) f8_mfma(acc[m][i], w[u][i], sw[u][i], xc[u][m], sx[u][m]);
        }
      }
    }
  }
  constexpr int kSums = MT * NT;
  if (waves > 1) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < NT; ++i)
        *reinterpret_cast<f32x4_t*>(lds_sums + ((wave * kSums + m * NT + i) * kWave + lane) * 4) = acc[m][i];
    __syncthreads();
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int at = m * NT + i;
      if (at % waves != wave) continue;
      f32x4_t sum = acc[m][i];
      if (waves > 1) {
        sum = *reinterpret_cast<const f32x4_t*>(lds_sums + (at * kWave + lane) * 4);
        for (int v = 1; v < waves; ++v)
          sum += *reinterpret_cast<const f32x4_t*>(lds_sums + ((v * kSums + at) * kWave + lane) * 4);
      }
      const int n = (tile0 + i) * 16 + 4 * (lane >> 4);
      if (16 * m + r < p.rows && n < a.N) store_acc<E>(a, p.row0 + 16 * m + r, n, sum);
    }
}

template <class E, int MT, int NT, bool CODES, int WAVES>
hipError_t go_few(const F8GemmArgs& a, hipStream_t s) {
  int waves = WAVES;
  while (waves > 1 && waves > a.blocks) waves >>= 1;
  constexpr int kUnit = 16 * MT;
  const int64_t mt = a.offsets ? a.T / kUnit + a.experts : (a.T + kUnit - 1) / kUnit;
  const dim3 grid((a.tiles + NT - 1) / NT, static_cast<unsigned>(mt));
  constexpr size_t kPerWave = MT * NT * kWave * 16;
  return launch_lds<&f8_few_kernel<E, MT, NT, CODES, WAVES>, WAVES * kPerWave>(grid, waves * kWave, waves * kPerWave, s, a);
}

template <int kW, int kX>
dim3 tile_grid(const F8GemmArgs& a) {
  const int64_t nt = (a.tiles + kW - 1) / kW;
  const int64_t mt = a.offsets ? a.T / (16 * kX) + a.experts : (a.T + 16 * kX - 1) / (16 * kX);
  return dim3(static_cast<unsigned>(nt * mt));
}
template <int FX, bool PAST>
hipError_t go_gemm(const F8GemmArgs& a, hipStream_t s) {
  using G = F8Gemm<FX, PAST>;
  return launch_lds<&f8_gemm_kernel<FX, PAST>, G::kLds>(tile_grid<16, FX>(a), 256, G::kLds, s, a);
}

}  // namespace

// bf16 results: the matrix core multiplies the codes.  It cuts the products of 8
// consecutive inputs to multiples of 2^-13 of the largest one's power of two and
// adds them in fp32, so a sum is off by less than 7 * 2^-13 of the largest product
// of each 8 (1.35e-5 of its norm for Gaussian data); a code's own rounding is 2^-4,
// the result's 2^-8.  fp32 results have the same codes multiplied as bf16 values,
// exactly, with fp32 sums, at half the rate or less.
//
// Which kernel: by the sizes, fitted to 218 calls, each timed with every kernel (1 to
// 32768 rows of 768 x 1024 to 11008 x 4096, 1 to 128 experts, both types): the one
// taken is 3 % behind the fastest on average, by more than 10 % in 13 of them and by
// 21 % at the most.  Replayed, us, bf16:
//                               8192 x 2048                64 experts of 1024 x 2048
//   rows                        1    32   64   256  1024  64    256   1024  4096  8192
//   rounding on the way
//     16 x 16, 16 waves         8.0  16.1 28.5 105  411   35.5  51.6  87.6  256   484
//     16 x 32, 8 waves          6.4  9.4  15.4 50.3 184   21.0  31.5  45.2  121   223
//     16 x 64, 8 waves          6.5  7.6  12.7 43.2 164   21.6  32.3  42.9  105   192
//     16 x 32, 4 waves          7.0  9.3  14.4 43.7 160   19.0  26.8  38.7  96.0  175
//     16 x 64, 4 waves          7.5  8.8  10.5 35.1 131   20.0  28.0  35.6  81.3  145
//   codes from a launch of their own
//     32 x 32, 4 waves          9.8  10.9 12.5 22.5 61.0  23.4  31.8  37.7  58.9  89.9
//     64 x 64, 4 waves          12.8 13.9 14.3 18.2 44.3  28.6  37.9  40.3  52.6  74.0
//     64 x 256, through LDS     17.3 18.7 19.4 19.9 28.3  30.8  36.5  39.4  45.9  66.3
//     128 x 256, through LDS    19.1 20.3 20.8 22.4 28.1  30.2  39.2  42.2  49.9  56.9
// With many workgroups, small ones with few waves follow each other without a gap
// (the waves of one wait for each other at its end); with few, more waves a
// workgroup keep more of the weights on their way.
template <class E>
hipError_t go_few_rows(const F8GemmArgs& a, int64_t groups, hipStream_t s) {
  // At most 256 workgroups, one for each CU, of the narrowest tiles that allow it (16 rows of 2048 inputs, us in tiles of
  // 16 x 16, 16 x 32, 16 x 64: 4096 outputs 5.8, 6.3, 7.2; 5120: 9.0, 6.4, 7.2; 8192: 9.3, 6.8, 7.5; 8224: 12.1, 8.7, 7.5)
  if (groups <= 128) return go_few<E, 1, 1, false, 16>(a, s);
  if (groups <= 256) return go_few<E, 1, 2, false, 8>(a, s);
  if (groups <= 512) return go_few<E, 1, 4, false, 8>(a, s);
  if constexpr (E::kBytes == 2) {  // 16 x 32 suits tiles of few rows; fp32's widening costs less in 16 x 64 everywhere
    if (a.T <= 16 * static_cast<int64_t>(a.experts) && groups <= 2048) return go_few<E, 1, 2, false, 4>(a, s);
  }
  return go_few<E, 1, 4, false, 4>(a, s);
}

hipError_t launch_f8_product(const F8GemmArgs& a, const F8RowsArgs& rows, int dtype, hipStream_t s) {
  const bool bf16 = dtype == 1;
  // tiles of rows: the most there can be, and about how many (an expert's last one is half full on average)
  auto row_tiles = [&](int64_t unit) { return a.offsets ? a.T / unit + a.experts : (a.T + unit - 1) / unit; };
  auto row_work = [&](int unit) {
    return a.offsets ? static_cast<double>(a.T) / unit + 0.5 * a.experts : static_cast<double>(row_tiles(unit));
  };
  const int64_t pairs = (a.tiles + 1) / 2, quads = (a.tiles + 3) / 4, blocks = a.blocks;
  const int64_t groups = row_tiles(16) * pairs;
  // rounding again in every workgroup costs fp32 more: long rows take longer than their codes' launch
  if ((bf16 || a.T == 1 || blocks <= 32) &&
      (a.T <= 16 * static_cast<int64_t>(a.experts) || groups * blocks <= (bf16 ? 16384 : 12288)))
    return bf16 ? go_few_rows<EBf16>(a, groups, s) : go_few_rows<EF32>(a, groups, s);
  const hipError_t e = launch_f8_rows(rows, dtype, s);
  if (e != hipSuccess) return e;
  // estimates in us; those of the tiles through LDS leave a part out that the others have as well
  if (!bf16) {
    const double few = 4.2e-4 * row_work(32) * pairs * blocks;
    const double rounds = 0.5 * row_work(64) * ((a.tiles + 7) / 8) / 512;
    if (1.35 * blocks * (rounds > 1 ? rounds : 1) > few) return go_few<EF32, 2, 2, true, 4>(a, s);
    return launch_lds<&f8_gemm_exact_kernel, 2 * kExactStage>(tile_grid<kExactTiles, kExactTiles>(a), 256,
                                                              2 * kExactStage, s, a);
  }
  const double few32 = 3.8e-4 * row_work(32) * pairs * blocks, few64 = 1.5e-3 * row_work(64) * quads * blocks;
  const double strips = (a.tiles + 15) / 16, rounds = row_work(64) * strips / 512;
  if (1.05 * blocks * (rounds > 1 ? rounds : 1) > (few32 < few64 ? few32 : few64)) {
    // 64 x 64 tiles only where they are enough
    return few64 < few32 && row_tiles(64) * quads >= 256 ? go_few<EBf16, 4, 4, true, 4>(a, s)
                                                         : go_few<EBf16, 2, 2, true, 4>(a, s);
  }
  // While there are few, tiles of 64 rows: up to half as many of 128 rows as CUs they halve each CU's work; past that
  // some CUs have two, as much as one of 128 rows.  One matrix, us with 64 and 128 rows, by tiles of 128: 2048 inputs 128
  // 22.8, 25.5; 144 24.8, 25.4; 160 25.6, 25.7; 192 26.7, 27.8; 224 29.2, 28.7; 272 41.1, 39.3; 4096 inputs 144 36.6,
  // 37.9; 160 37.9, 37.5; 192 39.7, 38.0; 256 43.9, 42.6.  Of experts the last tiles cost as much as full ones: 16 of 2048
  // outputs and inputs 128 31.5, 32.6; 192 35.8, 34.2; 256 38.5, 45.4; 320 56.3, 48.6; 64 of 1024: 256 46.3, 50.1.
  if (row_work(128) * strips <= (a.offsets ? 256 : 160)) return go_gemm<4, false>(a, s);
  // Results of 64 MB and more, unless there is little to read for them, go past the caches, which keep the operands:
  // 16384 x 8192 of 2048 and 8192 inputs 260 -> 248 and 903 -> 868 us, but of 512 inputs 107 -> 111.
  return a.T * a.N >= int64_t(1) << 25 && blocks >= 8 ? go_gemm<8, true>(a, s) : go_gemm<8, false>(a, s);
}

}  // namespace twell
