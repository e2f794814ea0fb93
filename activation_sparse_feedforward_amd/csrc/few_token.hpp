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
//            inputs, rotated left by three bits: input 2j in bits 4j+3 .. 4j+6
//            and input 2j+1 in bits 4j+19 .. 4j+22 (bit numbers modulo 32).
//            Scales: bf16, [block][16 rows][128 / group].
//
// The matrix instruction takes tokens as its 16 rows and weight rows as its 16
// columns, so a lane's four results belong to one weight row: the group scale
// is one value per lane.  Matrix row m holds token 4 (m % 4) + m / 4, which
// puts tokens 4i .. 4i+3 into result register i of the four lane groups: up to
// four tokens need one register, and one FMA per group of weights.
#pragma once

#include "common.hpp"
#include "launch.hpp"

namespace twell {

constexpr int kTileRows = 16;
constexpr int kBlockK = 128;

__device__ __forceinline__ f32x4_t mfma16(bf16x8_t a, bf16x8_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Where lanes of a wave hand values to each other through LDS: what was written (or
// read) before is done before anything after it, in the compiler's order too, which
// the barrier alone does not ask for.  No workgroup barrier, and no instruction: a
// wave's LDS operations come in order.
__device__ __forceinline__ void lds_handoff() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// fp32 -> bf16 bits, round to nearest even, NaN stays NaN.
__device__ __forceinline__ uint16_t bf16_of(float f) { return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f)); }

// Eight 4-bit codes as bf16 values q / 16, exact; the 16 is made good once, on the
// sums (Product::run).  16 + u with the offset 24 taken off by a product with -24 is
// half the work (7 operations instead of 15; 11008 x 4096 in 6.8 us instead of 7.5 for
// one token, 64 tokens through an expert layer in 62 instead of 66), but a sum then
// holds 24 times every input: beside an input of 1e4 nothing is left of 0.01 times a
// code where the large one's code is 0, and 128 inputs of 2e35 overflow whose products
// do not.
__device__ __forceinline__ bf16x8_t codes_operand(uint32_t w) {
  const uint32_t v = __builtin_rotateright32(w, 3) ^ 0x88888888u;  // u = q + 8 to two's complement
  uint32_t h = v >> 4;
  asm("" : "+v"(h));  // a word of its own: a conversion picks its byte for nothing, but not its nibble
  u32x4_t r;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t n = (j & 1 ? h : v) >> (8 * (j >> 1));
    const float lo = __builtin_amdgcn_cvt_off_f32_i4(n), hi = __builtin_amdgcn_cvt_off_f32_i4(n >> 16);
    r[j] = __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
  }
  return __builtin_bit_cast(bf16x8_t, r);
}

// 16 bytes from an address aligned to the element only (rows of odd width).
typedef uint32_t u32x4_a2_t __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_a4_t __attribute__((ext_vector_type(4), aligned(4)));

// The 16 bytes of a row p of K elements that begin at element k, zeros beyond the
// row's end.  One load, of the row's last 16 bytes at the latest, and a shift:
// eight loads one by one take 5.4 us instead of 4.4 (7 tokens of 5001 x 1999).
__device__ __forceinline__ u32x4_t piece_until(const uint16_t* p, int k, int K) {
  if (K < 8) {
    u32x4_t r{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k + i < K) r[i >> 1] |= static_cast<uint32_t>(p[k + i]) << (16 * (i & 1));
    return r;
  }
  const int at = k < K - 8 ? k : K - 8, n = k - at;  // the first n are not wanted
  const u32x4_t v = *reinterpret_cast<const u32x4_a2_t*>(p + at);
  const uint64_t lo = v[0] | static_cast<uint64_t>(v[1]) << 32, hi = v[2] | static_cast<uint64_t>(v[3]) << 32;
  const uint64_t a = n < 4 ? lo : n < 8 ? hi : 0, b = n < 4 ? hi : 0;
  const int bits = 16 * (n & 3);
  const uint64_t first = a >> bits | (b << 1) << (63 - bits), second = b >> bits;
  return u32x4_t{static_cast<uint32_t>(first), static_cast<uint32_t>(first >> 32), static_cast<uint32_t>(second),
                 static_cast<uint32_t>(second >> 32)};
}
// Four elements are as well loaded one by one (the other way was 3 % slower).
__device__ __forceinline__ u32x4_t piece_until(const float* p, int k, int K) {
  u32x4_t r{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (k + i < K) r[i] = __float_as_uint(p[k + i]);
  return r;
}

// ---------------------------------------------------------------- token operands
// The matrix instruction wants 16 tokens at 16 neighbouring lanes, 16 bytes of
// each: loaded like that, every 16 lanes touch 16 cache lines, which the L1
// serves one at a time (13 bytes a clock measured, of 64), and a single token
// would still take four load instructions of 16 clocks for a block.  Tokens
// therefore come in by rows (16 lanes read 256 consecutive bytes, one load
// takes four rows) and go through a piece of LDS that belongs to the wave
// alone, without a barrier: 16-byte pieces, piece c of row r at place
// c ^ (r % 16), which spreads both the writes and the reads over the banks.
//
// Source: what a row looks like.  A block of 128 inputs is kParts parts of 16
// pieces of 16 bytes; kPlanes bf16 operands whose sum is the value come out.

// Rows of bf16 values.
struct SourceBf16 {
  using Elem = uint16_t;
  static constexpr bool kCuts = false;
  static constexpr int kPlanes = 1, kParts = 1, kReads = 1;
  int K;
  // piece c of a part of block b of row p
  __device__ __forceinline__ u32x4_t piece(const Elem* p, int b, int, int c, bool whole) const {
    const int k = b * kBlockK + c * 8;
    return whole ? *reinterpret_cast<const u32x4_a2_t*>(p + k) : piece_until(p, k, K);
  }
  // the kReads pieces of step s and lane group g (part * 16 + piece), and the
  // operands made of them
  static __device__ __forceinline__ int place(int s, int g, int) { return 4 * s + g; }
  static __device__ __forceinline__ void operands(const u32x4_t (&v)[1], bf16x8_t (&x)[1]) {
    x[0] = __builtin_bit_cast(bf16x8_t, v[0]);
  }
};

// Rows of fp32 values, cut (truncated, so that each rest is exact) into three
// bf16 values: 24 bits of mantissa, so that products with bf16 weights lose
// nothing before the fp32 sum.
struct SourceF32 {
  using Elem = float;
  static constexpr bool kCuts = true;
  static constexpr int kPlanes = 3, kParts = 2, kReads = 2;
  int K;
  __device__ __forceinline__ u32x4_t piece(const Elem* p, int b, int part, int c, bool whole) const {
    const int k = b * kBlockK + part * 64 + c * 4;
    return whole ? *reinterpret_cast<const u32x4_a4_t*>(p + k) : piece_until(p, k, K);
  }
  static __device__ __forceinline__ int place(int s, int g, int i) { return 8 * s + 2 * g + i; }
  // two values as the halves of a word of each plane
  static __device__ __forceinline__ void cut(uint32_t va, uint32_t vb, uint32_t (&out)[3]) {
    float a = __uint_as_float(va), b = __uint_as_float(vb);
#pragma unroll
    for (int s = 0; s < 3; ++s) {
      const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
      out[s] = (ua >> 16) | (ub & 0xffff0000u);
      a -= __uint_as_float(ua & 0xffff0000u);
      b -= __uint_as_float(ub & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void operands(const u32x4_t (&v)[2], bf16x8_t (&x)[3]) {
    u32x4_t out[3];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t w[3];
      cut(v[j >> 1][2 * (j & 1)], v[j >> 1][2 * (j & 1) + 1], w);
#pragma unroll
      for (int s = 0; s < 3; ++s) out[s][j] = w[s];
    }
#pragma unroll
    for (int s = 0; s < 3; ++s) x[s] = __builtin_bit_cast(bf16x8_t, out[s]);
  }
};

// Rows already cut into P bf16 planes, padded with zeros to whole blocks.
template <int P>
struct SourcePlanes {
  using Elem = uint16_t;
  static constexpr bool kCuts = false;
  static constexpr int kPlanes = P, kParts = P, kReads = P;
  int64_t stride;  // between planes, in elements
  __device__ __forceinline__ u32x4_t piece(const Elem* p, int b, int part, int c, bool) const {
    return *reinterpret_cast<const u32x4_t*>(p + (part * stride + b * kBlockK) + c * 8);
  }
  static __device__ __forceinline__ int place(int s, int g, int i) { return 16 * i + 4 * s + g; }
  static __device__ __forceinline__ void operands(const u32x4_t (&v)[P], bf16x8_t (&x)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) x[i] = __builtin_bit_cast(bf16x8_t, v[i]);
  }
};

// Token (within a tile of 16) that lane l supplies as a matrix row.
__device__ __forceinline__ int lane_token(int lane) { return ((lane & 3) << 2) | ((lane >> 2) & 3); }
// Token of result register i in lane l.
__device__ __forceinline__ int result_token(int i, int lane) { return 4 * i + (lane >> 4); }

// Up to 4 TQ tokens, by rows and through LDS.  at(t) is a row for every t; where
// there is no token it is any other one, whose results nobody reads (a matrix
// row's results depend on that row alone).
template <class Src, int TQ>
struct Tokens {
  static constexpr int kRows = 4 * TQ;
  static constexpr int kPartBytes = kRows * 256;
  // fp32 values are cut on their way into LDS where there are fewer rows than
  // the matrix has, since 16 / kRows matrix rows read each (an expert layer of 8
  // tokens, 2 of 16 experts of 1024 x 1024: 20.3 us against 21.5); with all 16
  // rows in use the work is the same and the LDS half as much again.
  static constexpr bool kCutFirst = Src::kCuts && TQ <= 2;
  static constexpr int kLdsBytes = (kCutFirst ? Src::kPlanes : Src::kParts) * kPartBytes;  // of one wave
  Src src;
  const typename Src::Elem* row[TQ];  // row[j]: of token 4 j + lane / 16; a load takes four rows
  char* lds;
  struct Loaded {
    u32x4_t v[TQ][Src::kParts];
  };
  static __device__ __forceinline__ int piece_at(int r, int place) {
    return (place >> 4) * kPartBytes + r * 256 + (((place & 15) ^ (r & 15)) << 4);
  }
  template <class F>
  __device__ __forceinline__ Tokens(Src s, F at, char* lds_, int lane) : src(s), lds(lds_) {
#pragma unroll
    for (int j = 0; j < TQ; ++j) row[j] = at(4 * j + (lane >> 4));
  }
  __device__ __forceinline__ void fetch(Loaded& q, int b, bool whole, int lane) const {
#pragma unroll
    for (int j = 0; j < TQ; ++j)
#pragma unroll
      for (int i = 0; i < Src::kParts; ++i) q.v[j][i] = src.piece(row[j], b, i, lane & 15, whole);
  }
  __device__ __forceinline__ void store(const Loaded& q, int lane) const {
    lds_handoff();  // the block before has been read
#pragma unroll
    for (int j = 0; j < TQ; ++j)
#pragma unroll
      for (int i = 0; i < Src::kParts; ++i) {
        const int r = 4 * j + (lane >> 4), c = lane & 15;
        if constexpr (kCutFirst) {  // four values: half a piece of each plane
          uint32_t lo[3], hi[3];
          Src::cut(q.v[j][i][0], q.v[j][i][1], lo);
          Src::cut(q.v[j][i][2], q.v[j][i][3], hi);
#pragma unroll
          for (int p = 0; p < 3; ++p)
            *reinterpret_cast<u32x2_t*>(lds + piece_at(r, 16 * p + 8 * i + (c >> 1)) + 8 * (c & 1)) = u32x2_t{lo[p], hi[p]};
        } else {
          *reinterpret_cast<u32x4_t*>(lds + piece_at(r, 16 * i + c)) = q.v[j][i];
        }
      }
    lds_handoff();
  }
  __device__ __forceinline__ void step(const Loaded&, int s, int m, int lane, bf16x8_t (&x)[Src::kPlanes]) const {
    const int r = (m * 16 + lane_token(lane)) % kRows, g = lane >> 4;
    if constexpr (kCutFirst) {
#pragma unroll
      for (int p = 0; p < Src::kPlanes; ++p)
        x[p] = *reinterpret_cast<const bf16x8_t*>(lds + piece_at(r, 16 * p + 4 * s + g));
    } else {
      u32x4_t v[Src::kReads];
#pragma unroll
      for (int i = 0; i < Src::kReads; ++i)
        v[i] = *reinterpret_cast<const u32x4_t*>(lds + piece_at(r, Src::place(s, g, i)));
      Src::operands(v, x);
    }
  }
};

// Tiles of 16 tokens for TQ quads.
template <int TQ>
constexpr int token_tiles() { return (TQ + 3) / 4; }
// Result registers in use per tile of 16 tokens.
template <int TQ>
constexpr int token_regs() { return TQ < 4 ? TQ : 4; }

// ---------------------------------------------------------------- weights
// STREAM: past the caches, for weights that are read once and are larger than
// what stays in them.
template <bool STREAM>
__device__ __forceinline__ u32x4_t load_codes(const uint8_t* p) {
  const u32x4_t* q = reinterpret_cast<const u32x4_t*>(p);
  return STREAM ? __builtin_nontemporal_load(q) : *q;
}
template <int BITS>
struct Block;
template <>
struct Block<4> {
  static constexpr int kBytes = 1024;
  u32x4_t c;
  template <bool STREAM>
  __device__ __forceinline__ void load(const uint8_t* p, int lane) {
    c = load_codes<STREAM>(p + lane * 16);
  }
  __device__ __forceinline__ bf16x8_t step(int s) const { return codes_operand(c[s]); }
};
template <>
struct Block<16> {
  static constexpr int kBytes = 4096;
  u32x4_t c[4];
  template <bool STREAM>
  __device__ __forceinline__ void load(const uint8_t* p, int lane) {
#pragma unroll
    for (int s = 0; s < 4; ++s) c[s] = load_codes<STREAM>(p + (s * 64 + lane) * 16);
  }
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

// One block of each of NR tiles.
template <int BITS, int G, int NR, bool STREAM>
struct TileBlocks {
  Block<BITS> w[NR];
  Scales<G> s[NR];
  __device__ __forceinline__ void fetch(const Tile (&tile)[NR], int b, int lane) {
#pragma unroll
    for (int r = 0; r < NR; ++r) w[r].template load<STREAM>(tile[r].codes + static_cast<int64_t>(b) * Block<BITS>::kBytes, lane);
    if constexpr (BITS == 4) {
#pragma unroll
      for (int r = 0; r < NR; ++r) s[r].load(tile[r].scales + static_cast<int64_t>(b) * (16 * G), lane);
    }
  }
};

// acc += tokens x weights over blocks [b0, b1) of NR tiles.  TQ: quads of
// tokens (1, 2 or a multiple of 4); MT = tiles of 16 tokens.  G: 4-bit scales per
// block (1, 2, 4), unused for 16 bits.  nfull: blocks whose inputs are all below K.
template <int BITS, int G, int TQ, int NR, class Src, bool STREAM = false>
struct Product {
  using X = Tokens<Src, TQ>;
  static constexpr int MT = token_tiles<TQ>();
  static constexpr int P = Src::kPlanes;
  static constexpr int kRegs = token_regs<TQ>();
  static constexpr int kAll = NR * MT * kRegs;  // result registers
  f32x4_t acc[MT][NR];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int r = 0; r < NR; ++r) acc[m][r] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  }

  using Weights = TileBlocks<BITS, G, NR, STREAM>;
  using XLoaded = typename X::Loaded;

  __device__ __forceinline__ void use(const XLoaded& xq, const Weights& w, const X& x, int lane) {
    x.store(xq, lane);
    const f32x4_t zero{0.f, 0.f, 0.f, 0.f};
    if constexpr (BITS == 16) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          bf16x8_t v[P];
          x.step(xq, s, m, lane, v);
#pragma unroll
          for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int p = P - 1; p >= 0; --p) acc[m][r] = mfma16(v[p], w.w[r].step(s), acc[m][r]);
        }
      }
    } else {
      constexpr int kSteps = 4 / G;  // steps that share a scale
#pragma unroll
      for (int gr = 0; gr < G; ++gr) {
        f32x4_t t[MT][NR];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int r = 0; r < NR; ++r) t[m][r] = zero;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          bf16x8_t v[MT][P];
#pragma unroll
          for (int m = 0; m < MT; ++m) x.step(xq, gr * kSteps + i, m, lane, v[m]);
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            const bf16x8_t c = w.w[r].step(gr * kSteps + i);
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
              for (int p = P - 1; p >= 0; --p) t[m][r] = mfma16(v[m][p], c, t[m][r]);
          }
        }
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const float sc = w.s[r].at(gr);
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < kRegs; ++i) acc[m][r][i] = fmaf(sc, t[m][r][i], acc[m][r][i]);
        }
      }
    }
  }

  // The weights of U blocks are on their way together.
  template <int U>
  __device__ __forceinline__ void run(const X& x, const Tile (&tile)[NR], int b0, int b1, int nfull, int lane) {
    int b = b0;
    const int whole_end = b1 < nfull ? b1 : nfull;
    if constexpr (U > 1) {
      for (; b + U <= whole_end; b += U) {
        Weights w[U];
        XLoaded xq[2];
        x.fetch(xq[0], b, true, lane);
#pragma unroll
        for (int u = 0; u < U; ++u) w[u].fetch(tile, b + u, lane);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (u + 1 < U) x.fetch(xq[(u + 1) & 1], b + u + 1, true, lane);
          use(xq[u & 1], w[u], x, lane);
        }
      }
    }
    for (; b < whole_end; ++b) one_block(x, tile, b, true, lane);
    for (; b < b1; ++b) one_block(x, tile, b, false, lane);
    if constexpr (BITS == 4) {  // codes_operand
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < NR; ++r) acc[m][r] *= 16.f;
    }
  }
  __device__ __forceinline__ void one_block(const X& x, const Tile (&tile)[NR], int b, bool whole, int lane) {
    XLoaded xq;
    Weights w;
    x.fetch(xq, b, whole, lane);
    w.fetch(tile, b, lane);
    use(xq, w, x, lane);
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
