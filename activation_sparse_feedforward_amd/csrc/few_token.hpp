// Products of a few tokens with laid-out weights: the core shared by the
// 4-bit linear kernel and the mixture-of-experts kernels.
//
// Weights are held in blocks of 16 rows x 128 inputs, the inputs of one tile
// of 16 rows one block after another, so that a wave streams a tile with
// 16-byte loads of 1 KB each and no bounds checks (rows and inputs beyond the
// matrix are stored as zeros).  Lane l of a wave owns row l % 16 and, with
// g = l / 16, the inputs 32 s + 8 g .. + 7 of the block's four steps s = 0..3:
// exactly the operand of one v_mfma_f32_16x16x32_bf16 per step, so weights go
// from memory to the matrix core without a shuffle or LDS.
//   16 bits: step s of lane l is the 16-byte piece (s * 64 + l) of the block (4 KB).
//    4 bits: the 16-byte piece l of the block (1 KB) is lane l's four words,
//            one per step; a word holds the codes u = q + 8 of its eight
//            inputs, input 2j in bits 4j .. 4j+3 and input 2j+1 in bits
//            16+4j .. 16+4j+3.  Scales: bf16, [block][16 rows][128 / group].
//
// The matrix instruction takes tokens as its 16 rows and weight rows as its 16
// columns, so a lane's four results belong to one weight row: the group scale
// is one value per lane.  Matrix row m holds token 4 (m % 4) + m / 4, which
// puts tokens 4i .. 4i+3 into result register i of the four lane groups: up to
// four tokens need one register, and one FMA per group of weights.
#pragma once

#include "common.hpp"

namespace twell {

constexpr int kTileRows = 16;
constexpr int kBlockK = 128;

__device__ __forceinline__ f32x4_t mfma16(bf16x8_t a, bf16x8_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// fp32 -> bf16 bits, round to nearest even, NaN stays NaN.
__device__ __forceinline__ uint16_t bf16_of(float f) { return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f)); }

// Eight 4-bit codes as bf16 values 16 + u: u lands in mantissa bits 3 .. 6 of
// 16.0 (bit pattern 0x4180), so a pair costs one shift and one and-or.  The
// offset 16 + 8 is taken off again by a product with -24 (offset_operand).  For
// bf16 data: its sums are rounded to 8 bits in the end.
__device__ __forceinline__ bf16x8_t codes_operand(uint32_t w) {
  constexpr uint32_t kMask = 0x00780078u, kBase = 0x41804180u;
  u32x4_t r;
  r[0] = ((w << 3) & kMask) | kBase;
  r[1] = ((w >> 1) & kMask) | kBase;
  r[2] = ((w >> 5) & kMask) | kBase;
  r[3] = ((w >> 9) & kMask) | kBase;
  return __builtin_bit_cast(bf16x8_t, r);
}
__device__ __forceinline__ bf16x8_t offset_operand() {
  const u32x4_t r{0xC1C0C1C0u, 0xC1C0C1C0u, 0xC1C0C1C0u, 0xC1C0C1C0u};  // -24
  return __builtin_bit_cast(bf16x8_t, r);
}

// Eight 4-bit codes as bf16 values q.  2.5 operations per code instead of one,
// for fp32 data: the matrix core cuts its sums off at the size of the largest
// term, and with the offset's terms around 5 times the codes' that showed as
// an error of 1.1e-6 of the result's norm (64 x 4096 weights, groups of 32),
// one-sided; fp32 products of the plain kind have 3e-7.
__device__ __forceinline__ bf16x8_t exact_codes_operand(uint32_t w) {
  const int v = static_cast<int>(w ^ 0x88888888u);  // u = q + 8 to two's complement
  u32x4_t r;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float lo = static_cast<float>((v << (28 - 4 * j)) >> 28);
    const float hi = static_cast<float>((v << (12 - 4 * j)) >> 28);
    r[j] = (__float_as_uint(lo) >> 16) | (__float_as_uint(hi) & 0xffff0000u);
  }
  return __builtin_bit_cast(bf16x8_t, r);
}

// 16 bytes from an address aligned to the element only (rows of odd width).
typedef uint32_t u32x4_a2_t __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_a4_t __attribute__((ext_vector_type(4), aligned(4)));

// ---------------------------------------------------------------- token operands
// One row of the token operand per lane: inputs k .. k+7 as kPlanes bf16
// operands whose sum is the value.  `whole` says that k + 8 <= K for every lane
// of the wave; otherwise inputs from K on read as zero.
struct RowBf16 {
  static constexpr int kPlanes = 1;
  const uint16_t* p;  // row, or null for a row without a token
  int K;
  __device__ __forceinline__ void load(int k, bool whole, bf16x8_t (&v)[1]) const {
    u32x4_t r{0, 0, 0, 0};
    if (p != nullptr) {
      if (whole) {
        r = *reinterpret_cast<const u32x4_a2_t*>(p + k);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (k + i < K) r[i >> 1] |= static_cast<uint32_t>(p[k + i]) << (16 * (i & 1));
        }
      }
    }
    v[0] = __builtin_bit_cast(bf16x8_t, r);
  }
};

// An fp32 value is cut (truncated, so that each rest is exact) into three bf16
// values: 24 bits of mantissa, so products with bf16 weights lose nothing
// before the fp32 sum.
struct RowF32 {
  static constexpr int kPlanes = 3;
  const float* p;
  int K;
  __device__ __forceinline__ void load(int k, bool whole, bf16x8_t (&v)[3]) const {
    float f[8] = {};
    if (p != nullptr) {
      if (whole) {
        const u32x4_t a = *reinterpret_cast<const u32x4_a4_t*>(p + k);
        const u32x4_t b = *reinterpret_cast<const u32x4_a4_t*>(p + k + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[i] = __uint_as_float(a[i]);
          f[4 + i] = __uint_as_float(b[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (k + i < K) f[i] = p[k + i];
        }
      }
    }
    u32x4_t out[3];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float a = f[2 * j], b = f[2 * j + 1];
#pragma unroll
      for (int s = 0; s < 3; ++s) {
        const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
        out[s][j] = (ua >> 16) | (ub & 0xffff0000u);
        a -= __uint_as_float(ua & 0xffff0000u);
        b -= __uint_as_float(ub & 0xffff0000u);
      }
    }
#pragma unroll
    for (int s = 0; s < 3; ++s) v[s] = __builtin_bit_cast(bf16x8_t, out[s]);
  }
};

// A row already cut into P bf16 planes, padded with zeros to whole blocks.
template <int P>
struct RowPlanes {
  static constexpr int kPlanes = P;
  const uint16_t* p;
  int64_t stride;  // between planes, in elements
  __device__ __forceinline__ void load(int k, bool, bf16x8_t (&v)[P]) const {
#pragma unroll
    for (int s = 0; s < P; ++s) {
      u32x4_t r{0, 0, 0, 0};
      if (p != nullptr) r = *reinterpret_cast<const u32x4_t*>(p + s * stride + k);
      v[s] = __builtin_bit_cast(bf16x8_t, r);
    }
  }
};

// Token (within a tile of 16) that lane l supplies as a matrix row.
__device__ __forceinline__ int lane_token(int lane) { return ((lane & 3) << 2) | ((lane >> 2) & 3); }
// Token of result register i in lane l.
__device__ __forceinline__ int result_token(int i, int lane) { return 4 * i + (lane >> 4); }

// ---------------------------------------------------------------- weights
template <int BITS>
struct Block;
template <>
struct Block<4> {
  static constexpr int kBytes = 1024;
  u32x4_t c;
  __device__ __forceinline__ void load(const uint8_t* p, int lane) {
    c = *reinterpret_cast<const u32x4_t*>(p + lane * 16);
  }
  template <bool EXACT>
  __device__ __forceinline__ bf16x8_t step(int s) const {
    return EXACT ? exact_codes_operand(c[s]) : codes_operand(c[s]);
  }
};
template <>
struct Block<16> {
  static constexpr int kBytes = 4096;
  u32x4_t c[4];
  __device__ __forceinline__ void load(const uint8_t* p, int lane) {
#pragma unroll
    for (int s = 0; s < 4; ++s) c[s] = *reinterpret_cast<const u32x4_t*>(p + (s * 64 + lane) * 16);
  }
  template <bool>
  __device__ __forceinline__ bf16x8_t step(int s) const { return __builtin_bit_cast(bf16x8_t, c[s]); }
};

// A tile of 16 weight rows: its first block and its first block's scales.
struct Tile {
  const uint8_t* codes;
  const uint16_t* scales;
};

// The G scales of lane's row in one block, as loaded; at(i): as fp32.
template <int G>
struct Scales {
  uint32_t v[(G + 1) / 2];
  __device__ __forceinline__ void load(const uint16_t* p, int lane) {
    const uint16_t* q = p + (lane & 15) * G;
    if constexpr (G == 1) {
      v[0] = q[0];
    } else if constexpr (G == 2) {
      v[0] = *reinterpret_cast<const uint32_t*>(q);
    } else {
      const u32x2_t w = *reinterpret_cast<const u32x2_t*>(q);
      v[0] = w[0];
      v[1] = w[1];
    }
  }
  __device__ __forceinline__ float at(int i) const {
    return __uint_as_float(i & 1 ? v[i >> 1] & 0xffff0000u : v[i >> 1] << 16);
  }
};

// acc += tokens x weights over blocks [b0, b1) of NR tiles.  TQ: quads of
// tokens (1: up to 4 tokens, 4 / 8 / 16: up to 16 / 32 / 64); MT = tiles of 16
// tokens.  G: 4-bit scales per block (1, 2, 4), unused for 16 bits.  nfull:
// blocks whose inputs are all below K.
template <int TQ>
constexpr int token_tiles() { return (TQ + 3) / 4; }
// Result registers in use per tile of 16 tokens.
template <int TQ>
constexpr int token_regs() { return TQ < 4 ? TQ : 4; }

template <int BITS, int G, int TQ, int NR, class Row>
struct Product {
  static constexpr int MT = token_tiles<TQ>();
  static constexpr int P = Row::kPlanes;
  static constexpr int kRegs = token_regs<TQ>();
  static constexpr int kAll = NR * MT * kRegs;  // result registers
  static constexpr bool kExact = P == 3;        // fp32 data: codes without the offset
  f32x4_t acc[MT][NR];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int r = 0; r < NR; ++r) acc[m][r] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  }

  struct Loaded {
    bf16x8_t x[MT][4][P];
    Block<BITS> w[NR];
    Scales<G> s[NR];
  };

  static __device__ __forceinline__ void fetch(Loaded& q, const Row (&row)[MT], const Tile (&tile)[NR], int b,
                                               bool whole, int lane) {
    const int k = b * kBlockK + (lane >> 4) * 8;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int s = 0; s < 4; ++s) row[m].load(k + 32 * s, whole, q.x[m][s]);
#pragma unroll
    for (int r = 0; r < NR; ++r) q.w[r].load(tile[r].codes + static_cast<int64_t>(b) * Block<BITS>::kBytes, lane);
    if constexpr (BITS == 4) {
#pragma unroll
      for (int r = 0; r < NR; ++r) q.s[r].load(tile[r].scales + static_cast<int64_t>(b) * (16 * G), lane);
    }
  }

  __device__ __forceinline__ void use(const Loaded& q) {
    if constexpr (BITS == 16) {
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const bf16x8_t b = q.w[r].template step<true>(s);
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int p = P - 1; p >= 0; --p) acc[m][r] = mfma16(q.x[m][s][p], b, acc[m][r]);
        }
    } else {
      constexpr int kSteps = 4 / G;  // steps that share a scale
      const bf16x8_t off = offset_operand();
#pragma unroll
      for (int gr = 0; gr < G; ++gr) {
        f32x4_t base[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          base[m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
          if constexpr (!kExact) {
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
#pragma unroll
              for (int p = P - 1; p >= 0; --p) base[m] = mfma16(q.x[m][gr * kSteps + s][p], off, base[m]);
          }
        }
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          f32x4_t t[MT];
#pragma unroll
          for (int m = 0; m < MT; ++m) t[m] = base[m];
#pragma unroll
          for (int s = 0; s < kSteps; ++s) {
            const bf16x8_t b = q.w[r].template step<kExact>(gr * kSteps + s);
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
              for (int p = P - 1; p >= 0; --p) t[m] = mfma16(q.x[m][gr * kSteps + s][p], b, t[m]);
          }
          const float sc = q.s[r].at(gr);
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < kRegs; ++i) acc[m][r][i] = fmaf(sc, t[m][i], acc[m][r][i]);
        }
      }
    }
  }

  // U blocks are fetched together.
  template <int U>
  __device__ __forceinline__ void run(const Row (&row)[MT], const Tile (&tile)[NR], int b0, int b1, int nfull,
                                      int lane) {
    int b = b0;
    const int whole_end = b1 < nfull ? b1 : nfull;
    if constexpr (U > 1) {
      for (; b + U <= whole_end; b += U) {
        Loaded q[U];
#pragma unroll
        for (int u = 0; u < U; ++u) fetch(q[u], row, tile, b + u, true, lane);
#pragma unroll
        for (int u = 0; u < U; ++u) use(q[u]);
      }
    }
    for (; b < whole_end; ++b) {
      Loaded q;
      fetch(q, row, tile, b, true, lane);
      use(q);
    }
    for (; b < b1; ++b) {
      Loaded q;
      fetch(q, row, tile, b, false, lane);
      use(q);
    }
  }

  // The wave's sums to LDS: register j = (r, m, i) of lane l at
  // red[(wave * kAll + j) * 64 + l].
  __device__ __forceinline__ void put(float* red, int wave, int lane) const {
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < kRegs; ++i) red[(wave * kAll + (r * MT + m) * kRegs + i) * 64 + lane] = acc[m][r][i];
  }
};

// Sum over the waves, in their order, of element o (register * 64 + lane) of
// kAll * 64 put there by Product::put.
template <int kAll>
__device__ __forceinline__ float joined(const float* red, int waves, int o) {
  float v = 0.f;
  for (int w = 0; w < waves; ++w) v += red[w * kAll * 64 + o];
  return v;
}

}  // namespace twell
