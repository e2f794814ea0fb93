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

// More results per wave need more registers, so fewer waves per workgroup.
template <int TQ, int NR>
constexpr int max_waves() { return NR * token_tiles<TQ>() * token_regs<TQ>() <= 16 ? 16 : 8; }

template <class E, int G, int TQ, int NR>
__global__ __launch_bounds__((max_waves<TQ, NR>() * kWave)) void linear4_kernel(LinearArgs a) {
  extern __shared__ float red[];
  using Row = std::conditional_t<E::kBytes == 2, RowBf16, RowF32>;
  using Elem = typename E::storage;
  using Prod = Product<4, G, TQ, NR, Row>;
  constexpr int MT = Prod::MT;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * (4 * TQ);
  const int T = a.T - t0 < 4 * TQ ? static_cast<int>(a.T - t0) : 4 * TQ;

  Row row[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int t = m * 16 + lane_token(lane);
    row[m].K = a.K;
    row[m].p = t < T ? static_cast<const Elem*>(a.x) + (t0 + t) * a.ldx : nullptr;
  }
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
  p.template run<(Prod::kAll <= 4 && E::kBytes == 2) ? 2 : 1>(row, tile, b0, b1, a.K / kBlockK, lane);
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
void go(const LinearArgs& a, hipStream_t s) {
  constexpr int kAll = NR * token_tiles<TQ>() * token_regs<TQ>();
  int waves = max_waves<TQ, NR>();
  while (waves > 1 && waves > a.blocks) waves >>= 1;
  const dim3 grid((a.tiles + NR - 1) / NR, static_cast<unsigned>((a.T + 4 * TQ - 1) / (4 * TQ)));
  linear4_kernel<E, G, TQ, NR><<<grid, waves * kWave, waves * kAll * 64 * sizeof(float), s>>>(a);
}

// The most tiles per workgroup that still leave a workgroup for every CU.
template <class E, int G, int TQ, int NR>
void by_rows(const LinearArgs& a, int cus, hipStream_t s) {
  const int64_t groups = (a.T + 4 * TQ - 1) / (4 * TQ);
  if constexpr (NR > 1) {
    if ((a.tiles + NR - 1) / NR * groups < cus) {
      by_rows<E, G, TQ, NR / 2>(a, cus, s);
      return;
    }
  }
  go<E, G, TQ, NR>(a, s);
}

template <class E, int G>
void by_tokens(const LinearArgs& a, hipStream_t s) {
  const int cus = 256;
  if (a.T <= 4) by_rows<E, G, 1, (E::kBytes == 2 ? 8 : 4) / (G == 4 ? 4 : 1)>(a, cus, s);
  else if (a.T <= 16) by_rows<E, G, 4, 4>(a, cus, s);
  else by_rows<E, G, 8, E::kBytes == 2 ? 2 : 1>(a, cus, s);
}

template <class E>
void by_group(const LinearArgs& a, hipStream_t s) {
  if (a.group == 32) by_tokens<E, 4>(a, s);
  else if (a.group == 64) by_tokens<E, 2>(a, s);
  else by_tokens<E, 1>(a, s);
}

}  // namespace

hipError_t launch_linear4(const LinearArgs& a, int dtype, hipStream_t s) {
  if (dtype == 0) by_group<EF32>(a, s);
  else by_group<EBf16>(a, s);
  return hipGetLastError();
}

}  // namespace twell
