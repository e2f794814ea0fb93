// y = x W^T for a few tokens with 4-bit weights (layout and arithmetic:
// few_token.hpp).
//
// One workgroup per NR tiles of 16 weight rows; its waves split the inputs
// and their sums are joined through LDS in wave order.  Bound by reading the
// codes: 0.5 byte per weight against one shift and one and-or per two weights.
#include "few_token.hpp"
#include "internal.hpp"

namespace twell {
namespace {

// Waves of a workgroup, as registers and LDS (the waves' sums) allow.
template <class E, int TQ, int NR>
constexpr int max_waves() {
  return E::kBytes == 2 ? (NR * token_tiles<TQ>() <= 4 ? 16 : 8) : TQ <= 2 || (TQ == 4 && NR <= 3) ? 16 : 8;
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
    const float v = joined<Prod::kAll>(red, waves, o);
    const int j = o >> 6, l = o & 63;
    const int i = j % Prod::kRegs, m = (j / Prod::kRegs) % MT, r = j / (Prod::kRegs * MT);
    const int t = m * 16 + result_token(i, l);
    const int n = (blockIdx.x * NR + r) * kTileRows + (l & 15);
    if (t < T && n < a.N) {
      Elem* y = static_cast<Elem*>(a.y) + (t0 + t) * a.ldy + n;
      if constexpr (E::kBytes == 2) *y = bf16_of(v);
      else *y = v;
    }
  }
}

template <class E, int G, int TQ, int NR>
hipError_t go(const LinearArgs& a, hipStream_t s) {
  using Prod = Product<4, G, TQ, NR, std::conditional_t<E::kBytes == 2, SourceBf16, SourceF32>>;
  constexpr int kPerWave = Prod::kAll * 256 > Prod::X::kLdsBytes ? Prod::kAll * 256 : Prod::X::kLdsBytes;
  constexpr int kWaves = max_waves<E, TQ, NR>();
  if constexpr (kWaves * kPerWave > 64 * 1024) {
    static const hipError_t attr = hipFuncSetAttribute(reinterpret_cast<const void*>(&linear4_kernel<E, G, TQ, NR>),
                                                       hipFuncAttributeMaxDynamicSharedMemorySize, kWaves * kPerWave);
    if (attr != hipSuccess) return attr;
  }
  int waves = kWaves;
  while (waves > 1 && waves > a.blocks) waves >>= 1;
  const dim3 grid((a.tiles + NR - 1) / NR, static_cast<unsigned>((a.T + 4 * TQ - 1) / (4 * TQ)));
  linear4_kernel<E, G, TQ, NR><<<grid, waves * kWave, waves * kPerWave, s>>>(a);
  return hipGetLastError();
}

// The fewest tiles per workgroup that leave no more than one workgroup for a
// CU, so that all run at once.
template <class E, int G, int TQ, int NR, int kMost>
hipError_t by_rows(const LinearArgs& a, int cus, hipStream_t s) {
  const int64_t groups = (a.T + 4 * TQ - 1) / (4 * TQ);
  if constexpr (NR < kMost) {
    if ((a.tiles + NR - 1) / NR * groups > cus) return by_rows<E, G, TQ, NR + 1, kMost>(a, cus, s);
  }
  return go<E, G, TQ, NR>(a, s);
}

template <class E, int G>
hipError_t by_tokens(const LinearArgs& a, hipStream_t s) {
  const int cus = lockstep_resident() > 0 ? lockstep_resident() : 256;
  if (a.T <= 4) return by_rows<E, G, 1, 1, 4>(a, cus, s);
  if (a.T <= 8) return by_rows<E, G, 2, 1, 4>(a, cus, s);
  if (a.T <= 16) return by_rows<E, G, 4, 1, 4>(a, cus, s);
  if constexpr (E::kBytes == 2) {
    // 64 tokens a workgroup save unpacking the codes twice, once that still
    // leaves a workgroup for every CU
    if (a.T > 32 && (a.tiles + 2) / 3 * ((a.T + 63) / 64) >= cus) return go<E, G, 16, 3>(a, s);
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
