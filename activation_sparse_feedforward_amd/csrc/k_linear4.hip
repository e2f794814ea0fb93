// y = x W^T for a few tokens with 4-bit weights (layout and arithmetic:
// few_token.hpp).
//
//   y[t,n] = sum_g s[n,g] sum_{k in g} x[t,k] q[n,k]
//
// One workgroup per NR tiles of 16 weight rows and 4 TQ tokens; its waves split
// the inputs and their sums are joined through LDS in wave order, so that one
// launch does it all and a short product still has every CU reading.  Up to 16
// tokens it is bound by reading the codes and unpacking them (0.5 byte and two
// operations a weight): 11008 x 4096 takes 7.5 us for one token (3.1 TB/s) and 8.1
// for 16, 4096 x 1024 2.7 us, of which the launch itself is 1.6.  Beyond that by
// getting the tokens to the matrix core, through the L1 and LDS once per NR tiles:
// 128 tokens of 2048 x 8192 12.7 us (0.34 PFLOP/s), of 16384 x 2048 21.7 us (0.40).
// fp32 data costs three matrix instructions for one: 7 tokens of 5001 x 1999 5.2 us.
#include "few_token.hpp"
#include "internal.hpp"

namespace twell {
namespace {

// Waves of a workgroup, as registers and LDS (the waves' sums) allow.
template <class E, int TQ, int NR>
constexpr int max_waves() {
  return E::kBytes == 2 ? (TQ < 8 && NR * token_tiles<TQ>() <= 4 ? 16 : 8) : TQ <= 2 || (TQ == 4 && NR <= 3) ? 16 : 8;
}

__device__ __forceinline__ bool holds_infinity(const uint16_t* x, int K) {
#pragma unroll 1
  for (int k = 0; k < K; ++k)
    if ((x[k] & 0x7fff) == 0x7f80) return true;
  return false;
}

template <class E, int G, int TQ, int NR>
__global__ __launch_bounds__((max_waves<E, TQ, NR>() * kWave)) void linear4_kernel(LinearArgs a) {
  extern __shared__ __align__(16) char lds[];  // the waves' token pieces, then their sums
  using Src = std::conditional_t<E::kBytes == 2, SourceBf16, SourceF32>;
  using Elem = typename E::storage;
  using Prod = Product<4, G, TQ, NR, Src>;
  constexpr int MT = Prod::MT;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * (4 * TQ);
  const int T = a.T - t0 < 4 * TQ ? static_cast<int>(a.T - t0) : 4 * TQ;

  const typename Prod::X x(
      Src{a.K},
      [&](int t) { return static_cast<const Elem*>(a.x) + (t0 + (t < T ? t : 0)) * a.ldx; },
      lds + wave * Prod::X::kLdsBytes, lane);
  Tile tile[NR];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const int i = blockIdx.x * NR + r;
    const int64_t blk = static_cast<int64_t>(i < a.tiles ? i : a.tiles - 1) * a.blocks;
    tile[r].codes = a.codes + blk * Block<4>::kBytes;
    tile[r].scales = a.scales + blk * (16 * G);
  }
  Prod p;
  p.clear();
  const int b0 = a.blocks * wave / waves, b1 = a.blocks * (wave + 1) / waves;
  p.template run<1>(x, tile, b0, b1, a.K / kBlockK, lane);
  float* red = reinterpret_cast<float*>(lds);
  __syncthreads();  // the pieces have been read
  p.put(red, wave, lane);
  __syncthreads();
  for (int o = threadIdx.x; o < Prod::kAll * 64; o += blockDim.x) {
    float v = joined<Prod::kAll>(red, waves, o);
    const int j = o >> 6, l = o & 63;
    const int i = j % Prod::kRegs, m = (j / Prod::kRegs) % MT, r = j / (Prod::kRegs * MT);
    const int t = m * 16 + result_token(i, l);
    const int n = (blockIdx.x * NR + r) * kTileRows + (l & 15);
    if (t < T && n < a.N) {
      Elem* y = static_cast<Elem*>(a.y) + (t0 + t) * a.ldy + n;
      if constexpr (E::kBytes == 2) {
        // An infinite input makes its token's outputs NaN.  Codes of 0 and the cut of
        // fp32 data do that by themselves; an infinite sum of bf16 data is asked
        // whether it comes from one or from finite inputs.
        if (fabsf(v) == INFINITY && holds_infinity(static_cast<const Elem*>(a.x) + (t0 + t) * a.ldx, a.K)) v = NAN;
        *y = bf16_of(v);
      } else {
        *y = v;
      }
    }
  }
}

template <class E, int G, int TQ, int NR>
hipError_t go(const LinearArgs& a, hipStream_t s) {
  using Prod = Product<4, G, TQ, NR, std::conditional_t<E::kBytes == 2, SourceBf16, SourceF32>>;
  constexpr int kPerWave = Prod::kAll * 256 > Prod::X::kLdsBytes ? Prod::kAll * 256 : Prod::X::kLdsBytes;
  constexpr int kWaves = max_waves<E, TQ, NR>();
  int waves = kWaves;
  while (waves > 1 && waves > a.blocks) waves >>= 1;
  const dim3 grid((a.tiles + NR - 1) / NR, static_cast<unsigned>((a.T + 4 * TQ - 1) / (4 * TQ)));
  return launch_lds<&linear4_kernel<E, G, TQ, NR>, kWaves * kPerWave>(grid, waves * kWave, waves * kPerWave, s, a);
}

// Tiles per workgroup, NR in [kLeast, kMost]: the workgroups go round the CUs
// one after another, and one costs NR tiles and its tokens, about a tile's time.
// (100 tokens of 8192 x 8192: 30.4 us with four tiles in one round against 44.2
// with three in two; one token of 20480 x 2048: 7.1 with three in two rounds
// against 9.1 with four in two.)
template <class E, int G, int TQ, int kLeast, int kMost>
hipError_t by_rows(const LinearArgs& a, int cus, hipStream_t s) {
  const int64_t groups = (a.T + 4 * TQ - 1) / (4 * TQ);
  int best = kMost;
  int64_t least = INT64_MAX;
  for (int nr = kMost; nr >= kLeast; --nr) {
    const int64_t cost = ((a.tiles + nr - 1) / nr * groups + cus - 1) / cus * (nr + 1);
    if (cost < least) {
      least = cost;
      best = nr;
    }
  }
  if constexpr (kLeast <= 1) if (best == 1) return go<E, G, TQ, 1>(a, s);
  if constexpr (kLeast <= 2 && kMost >= 2) if (best == 2) return go<E, G, TQ, 2>(a, s);
  if constexpr (kLeast <= 3 && kMost >= 3) if (best == 3) return go<E, G, TQ, 3>(a, s);
  return go<E, G, TQ, kMost>(a, s);
}

template <class E, int G>
hipError_t by_tokens(const LinearArgs& a, hipStream_t s) {
  const int resident = lockstep_resident(), cus = resident > 0 ? resident : 256;
  // As many tokens as there are at once (their weights are unpacked once), but
  // fewer where that leaves CUs without work: 50 tokens of 700 x 6000 take 5.9 us
  // by sixteens against 8.6 by 32, 16 of 2048 x 8192 5.9 by eights against 6.4.
  auto fills = [&](int tokens) { return static_cast<int64_t>(a.tiles) * ((a.T + tokens - 1) / tokens) <= cus; };
  if (a.T <= 4 || fills(4)) return by_rows<E, G, 1, 1, 4>(a, cus, s);
  if (a.T <= 8 || fills(8)) return by_rows<E, G, 2, 1, 4>(a, cus, s);
  if (a.T <= 16 || fills(16)) return by_rows<E, G, 4, 1, 4>(a, cus, s);
  if constexpr (E::kBytes == 2) {
    // 64 tokens a workgroup save unpacking the codes twice, once that still
    // leaves a workgroup for every CU: 128 tokens of 16384 x 2048 22.0 us against
    // 27.0, but 64 of 8192 x 8192 22.7 against 19.8
    if (a.T > 32 && (a.tiles + 2) / 3 * ((a.T + 63) / 64) >= cus) return by_rows<E, G, 16, 3, 4>(a, cus, s);
    return by_rows<E, G, 8, 1, 4>(a, cus, s);
  }
  return by_rows<E, G, 8, 1, 2>(a, cus, s);
}

template <class E>
hipError_t by_group(const LinearArgs& a, hipStream_t s) {
  if (a.group == 32) return by_tokens<E, 4>(a, s);
  if (a.group == 64) return by_tokens<E, 2>(a, s);
  return by_tokens<E, 1>(a, s);
}

}  // namespace

hipError_t launch_linear4(const LinearArgs& a, int dtype, hipStream_t s) {
  return dtype == 0 ? by_group<EF32>(a, s) : by_group<EBf16>(a, s);
}

}  // namespace twell
