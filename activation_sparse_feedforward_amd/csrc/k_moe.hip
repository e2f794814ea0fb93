// A mixture-of-experts gated feed-forward layer for a few tokens.
//
//   l[t,e] = x[t] . r[e] + b[e];  the top_k largest per token, softmax weights w
//   y[t]   = sum_i w_i  W_down_e ( act(W_gate_e x) * (W_up_e x) ),   e = ids[t,i]
//
// Three kernels.  (1) moe_route_kernel: one workgroup per token, logits in
// fp32, selection by one wave.  (2) moe_up_kernel: one workgroup per (chosen
// expert, 16 neurons); it gathers the expert's tokens, computes gate and up
// together and writes w * act(g) * u.  (3) moe_down_kernel: one workgroup per 16
// outputs; its waves split the chosen experts' neurons, add each expert's
// products to the rows of its tokens in a private LDS tile and join the tiles
// in wave order, so y is written once and does not depend on timing.
// Only chosen experts' weights are read, each once per call of up to 64
// tokens.  Bound by reading them.
#include "few_token.hpp"
#include "internal.hpp"

namespace twell {
namespace {

// ---------------------------------------------------------------- router
constexpr int kRouteWaves = 16;
constexpr int kRouteAhead = 4;  // experts a wave computes side by side

__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const uint32_t o = __shfl_xor(v, m);
    v = v > o ? v : o;
  }
  return v;
}

// Unsigned key in the order of the logits: NaN above everything, -0 = +0, 0
// below every logit (an expert that does not exist or is taken already).
__device__ __forceinline__ uint32_t order_key(float l) {
  if (l != l) return 0xffffffffu;
  const uint32_t u = __float_as_uint(l + 0.f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}

template <class E>
__device__ __forceinline__ void load8(const typename E::storage* p, int k, int K, float (&f)[8]) {
  if (k + 8 <= K) {
    if constexpr (E::kBytes == 2) {
      const u32x4_t v = *reinterpret_cast<const u32x4_a2_t*>(p + k);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(v[i] << 16);
        f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
      }
    } else {
      const u32x4_t a = *reinterpret_cast<const u32x4_a4_t*>(p + k);
      const u32x4_t b = *reinterpret_cast<const u32x4_a4_t*>(p + k + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[i] = __uint_as_float(a[i]);
        f[4 + i] = __uint_as_float(b[i]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = k + i < K ? load_elem<E>(p, k + i) : 0.f;
  }
}

template <class E>
__global__ __launch_bounds__(kRouteWaves* kWave) void moe_route_kernel(MoeArgs a) {
  __shared__ float logit[kMoeMaxExperts];
  using Elem = typename E::storage;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = blockIdx.x;
  const Elem* x = static_cast<const Elem*>(a.x) + t * a.ldx;
  for (int e0 = wave * kRouteAhead; e0 < a.E; e0 += kRouteWaves * kRouteAhead) {
    float s[kRouteAhead] = {};
    for (int k = lane * 8; k < a.d; k += 512) {
      float xv[8];
      load8<E>(x, k, a.d, xv);
#pragma unroll
      for (int j = 0; j < kRouteAhead; ++j) {
        const int e = e0 + j < a.E ? e0 + j : a.E - 1;
        float rv[8];
        load8<E>(static_cast<const Elem*>(a.router) + static_cast<int64_t>(e) * a.d, k, a.d, rv);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[j] = fmaf(xv[i], rv[i], s[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < kRouteAhead; ++j) {
      const float l = wave_sum(s[j]);
      if (lane == 0 && e0 + j < a.E) logit[e0 + j] = a.bias ? l + a.bias[e0 + j] : l;
    }
  }
  __syncthreads();
  if (wave != 0) return;

  // expert e = 64 r + lane is in key[r]
  constexpr int kRegs = kMoeMaxExperts / 64;
  uint32_t key[kRegs];
#pragma unroll
  for (int r = 0; r < kRegs; ++r) key[r] = r * 64 + lane < a.E ? order_key(logit[r * 64 + lane]) : 0u;
  uint32_t top = 0;
#pragma unroll
  for (int r = 0; r < kRegs; ++r) top = key[r] > top ? key[r] : top;
  const float most = key_value(wave_umax(top));
  const bool none = most == -INFINITY;  // every expert is masked off: all weights 0
  float sum = 0.f;
  for (int r = 0; r * 64 < a.E; ++r)
    if (r * 64 + lane < a.E) sum += expf(logit[r * 64 + lane] - most);
  sum = wave_sum(sum);

  float mine = 0.f, chosen = 0.f;  // lane i keeps choice i
  int mine_id = 0;
  for (int i = 0; i < a.k; ++i) {
    uint32_t m = 0;
#pragma unroll
    for (int r = 0; r < kRegs; ++r) m = key[r] > m ? key[r] : m;
    m = wave_umax(m);
    int id = -1;
#pragma unroll
    for (int r = 0; r < kRegs; ++r) {
      const uint64_t has = __ballot(key[r] == m);
      if (id < 0 && has != 0) {
        const int l = __builtin_ctzll(has);
        id = r * 64 + l;
        if (lane == l) key[r] = 0;
      }
    }
    const float w = none ? 0.f : expf(key_value(m) - most) / sum;
    chosen += w;
    if (lane == i) {
      mine = w;
      mine_id = id;
    }
  }
  if (a.renorm && !none) mine /= chosen;
  if (lane < a.k) {
    a.ids[t * a.k + lane] = mine_id;
    a.weights[t * a.k + lane] = mine;
  }
}

// ---------------------------------------------------------------- shared parts
template <class Prod, int NR>
__device__ __forceinline__ void put_partial(const Prod& p, float* red, int wave, int lane) {
  constexpr int kAll = NR * Prod::MT * Prod::kRegs;
#pragma unroll
  for (int r = 0; r < NR; ++r)
#pragma unroll
    for (int m = 0; m < Prod::MT; ++m)
#pragma unroll
      for (int i = 0; i < Prod::kRegs; ++i)
        red[(wave * kAll + (r * Prod::MT + m) * Prod::kRegs + i) * 64 + lane] = p.acc[m][r][i];
}

// ---------------------------------------------------------------- gate and up
constexpr int kUpWaves = 8;
constexpr int kUpPairs = kMoeBlockTokens * kMoeMaxTopK;

// h = w act(g) u for the tokens list[0 .. n) of one expert and 16 neurons.
template <class E, int BITS, int G, int TQ>
__device__ __forceinline__ void up_tokens(const MoeArgs& a, const Tile (&tile)[2], const int* list, int n, int neuron0,
                                          float* red, int lane, int wave) {
  using Row = std::conditional_t<E::kBytes == 2, RowBf16, RowF32>;
  using Elem = typename E::storage;
  using Prod = Product<BITS, G, TQ, 2, Row>;
  constexpr int MT = Prod::MT;
  Row row[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int i = m * 16 + lane_token(lane);
    row[m].K = a.d;
    row[m].p = i < n ? static_cast<const Elem*>(a.x) + static_cast<int64_t>(list[i] / a.k) * a.ldx : nullptr;
  }
  Prod p;
  p.clear();
  p.template run<(TQ <= 4 && E::kBytes == 2) ? 2 : 1>(row, tile, a.blocks_d * wave / kUpWaves, a.blocks_d * (wave + 1) / kUpWaves, a.d / kBlockK, lane);
  put_partial<Prod, 2>(p, red, wave, lane);
  __syncthreads();
  constexpr int kOne = MT * Prod::kRegs;  // registers of one matrix
  for (int o = threadIdx.x; o < kOne * 64; o += kUpWaves * kWave) {
    float g = 0.f, u = 0.f;
    for (int w = 0; w < kUpWaves; ++w) {
      g += red[w * 2 * kOne * 64 + o];
      u += red[(w * 2 + 1) * kOne * 64 + o];
    }
    const int j = o >> 6, l = o & 63;
    const int i = (j / Prod::kRegs) * 16 + result_token(j % Prod::kRegs, l);
    if (i >= n) continue;
    const int slot = list[i];
    // a NaN gate stays NaN under both activations
    const float act = a.act == 0 ? (g < 0.f ? 0.f : g) : g / (1.f + expf(-g));
    float h = a.weights[slot] * act * u;
    // the down projection reads h as bf16 values whose sum is h: two of them
    // keep 16 bits, so that only the output's own rounding is seen in bf16;
    // three keep all 24 for fp32
    uint16_t* out = a.h + static_cast<int64_t>(slot) * a.h_row + neuron0 + (l & 15);
#pragma unroll
    for (int s = 0; s < (E::kBytes == 2 ? 2 : 3); ++s) {
      const uint16_t b = bf16_of(h);
      out[s * a.h_plane] = b;
      h -= bf16_bits_to_f32(b);
    }
  }
  __syncthreads();
}

template <class E, int BITS, int G, int TQ>
__global__ __launch_bounds__(kUpWaves* kWave) void moe_up_kernel(MoeArgs a) {
  __shared__ int ids[kUpPairs];
  __shared__ int list[kMoeBlockTokens];
  __shared__ uint8_t taken[kMoeMaxExperts];
  __shared__ float red[kUpWaves * 2 * token_tiles<TQ>() * (TQ < 4 ? TQ : 4) * 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int which = blockIdx.y;  // of the chosen experts, in ascending order
  const int pairs = a.T * a.k;
  for (int e = threadIdx.x; e < a.E; e += kUpWaves * kWave) taken[e] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < pairs; i += kUpWaves * kWave) {
    // a choice of weight 0 is no choice; a NaN weight is one
    const int id = a.weights[i] == 0.f ? -1 : a.ids[i];
    ids[i] = id;
    if (id >= 0) taken[id] = 1;
  }
  __syncthreads();
  int expert = -1, chosen = 0;
  for (int e0 = 0; e0 < a.E; e0 += 64) {
    uint64_t has = __ballot(e0 + lane < a.E && taken[e0 + lane] != 0);
    const int c = __popcll(has);
    if (expert < 0 && which < chosen + c) {
      for (int i = chosen; i < which; ++i) has &= has - 1;
      expert = e0 + __builtin_ctzll(has);
    }
    chosen += c;
  }
  const bool first = blockIdx.x == 0 && wave == 0;
  if (first && which == 0 && lane == 0) *a.n_chosen = chosen;
  if (expert < 0) return;  // the whole workgroup
  if (wave == 0) {
    int n = 0, before = 0;
    for (int i0 = 0; i0 < pairs; i0 += 64) {
      const int id = i0 + lane < pairs ? ids[i0 + lane] : -1;
      const uint64_t has = __ballot(id == expert);
      if (id == expert) list[n + __popcll(has & ((1ull << lane) - 1))] = i0 + lane;
      n += __popcll(has);
      before += __popcll(__ballot(id >= 0 && id < expert));
    }
    if (lane == 0) ids[0] = n;  // every id has been read
    if (first) {
      for (int i = lane; i < n; i += 64) a.pairs[before + i] = list[i];
      if (lane == 0) a.chosen[which] = MoeChosen{expert, before, n, 0};
    }
  }
  __syncthreads();
  const int n = ids[0];
  const int ti = blockIdx.x;
  const int neuron0 = ti * kTileRows;
  if (ti >= a.tiles_f) {  // the neurons that fill the last block of 128
    for (int o = threadIdx.x; o < n * kTileRows; o += kUpWaves * kWave) {
      uint16_t* out = a.h + static_cast<int64_t>(list[o / kTileRows]) * a.h_row + neuron0 + o % kTileRows;
#pragma unroll
      for (int s = 0; s < (E::kBytes == 2 ? 2 : 3); ++s) out[s * a.h_plane] = 0;
    }
    return;
  }
  const int64_t blk = (static_cast<int64_t>(expert) * a.tiles_f + ti) * a.blocks_d;
  const Tile tile[2] = {{a.gate_codes + blk * Block<BITS>::kBytes, a.gate_scales + blk * (16 * G)},
                        {a.up_codes + blk * Block<BITS>::kBytes, a.up_scales + blk * (16 * G)}};
  if constexpr (TQ <= 4) {
    up_tokens<E, BITS, G, TQ>(a, tile, list, n, neuron0, red, lane, wave);
  } else {
    if (n <= 16) {
      up_tokens<E, BITS, G, 4>(a, tile, list, n, neuron0, red, lane, wave);
    } else {
      for (int i = 0; i < n; i += 4 * TQ)
        up_tokens<E, BITS, G, TQ>(a, tile, list + i, n - i < 4 * TQ ? n - i : 4 * TQ, neuron0, red, lane, wave);
    }
  }
}

// ---------------------------------------------------------------- down
// Waves of the down kernel: more than 16 tokens need more registers.
template <int TQ>
constexpr int down_waves() { return TQ <= 4 ? 16 : 8; }
// row sums, pair list and chosen experts of the largest call
constexpr int kDownLds =
    (8 * kMoeBlockTokens * kTileRows + kUpPairs) * 4 + kMoeMaxExperts * static_cast<int>(sizeof(MoeChosen));

// Adds blocks [b0, b1) of one expert's down products to its tokens' rows.
template <int BITS, int G, int TQ, int P>
__device__ __forceinline__ void down_tokens(const MoeArgs& a, const Tile (&tile)[1], const int* list, int n, int b0,
                                            int b1, float* mine, int lane) {
  using Row = RowPlanes<P>;
  using Prod = Product<BITS, G, TQ, 1, Row>;
  constexpr int MT = Prod::MT;
  Row row[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int i = m * 16 + lane_token(lane);
    row[m].stride = a.h_plane;
    row[m].p = i < n ? a.h + static_cast<int64_t>(list[i]) * a.h_row : nullptr;
  }
  Prod p;
  p.clear();
  p.template run<(TQ <= 4 && P == 2 && BITS == 4) ? 2 : 1>(row, tile, b0, b1, b1, lane);
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < Prod::kRegs; ++i) {
      const int s = m * 16 + result_token(i, lane);
      if (s < n) mine[(list[s] / a.k) * kTileRows + (lane & 15)] += p.acc[m][0][i];
    }
}

template <class E, int BITS, int G, int TQ>
__global__ __launch_bounds__(down_waves<TQ>() * kWave) void moe_down_kernel(MoeArgs a) {
  constexpr int P = E::kBytes == 2 ? 2 : 3;
  constexpr int kDownWaves = down_waves<TQ>();
  extern __shared__ float lds[];
  float* sums = lds;  // [waves][T][16]
  MoeChosen* chosen = reinterpret_cast<MoeChosen*>(sums + kDownWaves * a.T * kTileRows);
  int* pairs = reinterpret_cast<int*>(chosen + a.most_chosen);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n_chosen = *a.n_chosen;
  for (int i = threadIdx.x; i < kDownWaves * a.T * kTileRows; i += kDownWaves * kWave) sums[i] = 0.f;
  for (int i = threadIdx.x; i < n_chosen; i += kDownWaves * kWave) chosen[i] = a.chosen[i];
  // entries beyond the list's end are not used
  for (int i = threadIdx.x; i < a.T * a.k; i += kDownWaves * kWave) pairs[i] = a.pairs[i];
  __syncthreads();

  float* mine = sums + wave * a.T * kTileRows;
  const int ti = blockIdx.x;
  const int total = n_chosen * a.blocks_f;
  int b = static_cast<int>(static_cast<int64_t>(total) * wave / kDownWaves);
  const int end = static_cast<int>(static_cast<int64_t>(total) * (wave + 1) / kDownWaves);
  while (b < end) {
    const int c = b / a.blocks_f, b0 = b % a.blocks_f;
    const int b1 = b0 + (end - b) < a.blocks_f ? b0 + (end - b) : a.blocks_f;
    const MoeChosen q = chosen[c];
    const int64_t blk = (static_cast<int64_t>(q.expert) * a.tiles_d + ti) * a.blocks_f;
    const Tile tile[1] = {{a.down_codes + blk * Block<BITS>::kBytes, a.down_scales + blk * (16 * G)}};
    const int* list = pairs + q.first;
    if constexpr (TQ <= 4) {
      down_tokens<BITS, G, TQ, P>(a, tile, list, q.n, b0, b1, mine, lane);
    } else {
      if (q.n <= 16) {
        down_tokens<BITS, G, 4, P>(a, tile, list, q.n, b0, b1, mine, lane);
      } else {
        for (int i = 0; i < q.n; i += 4 * TQ)
          down_tokens<BITS, G, TQ, P>(a, tile, list + i, q.n - i < 4 * TQ ? q.n - i : 4 * TQ, b0, b1, mine, lane);
      }
    }
    b += b1 - b0;
  }
  __syncthreads();
  for (int o = threadIdx.x; o < a.T * kTileRows; o += kDownWaves * kWave) {
    float v = 0.f;
    for (int w = 0; w < kDownWaves; ++w) v += sums[w * a.T * kTileRows + o];
    const int n = ti * kTileRows + o % kTileRows;
    if (n < a.d) {
      const int64_t at = static_cast<int64_t>(o / kTileRows) * a.ldy + n;
      if constexpr (E::kBytes == 2) static_cast<uint16_t*>(a.y)[at] = bf16_of(v);
      else static_cast<float*>(a.y)[at] = v;
    }
  }
}

template <class E, int BITS, int G, int TQ>
hipError_t go(const MoeArgs& a, hipStream_t s) {
  const dim3 up(static_cast<unsigned>(a.blocks_f * (kBlockK / kTileRows)), static_cast<unsigned>(a.most_chosen));
  moe_up_kernel<E, BITS, G, TQ><<<up, kUpWaves * kWave, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  constexpr int kDownWaves = down_waves<TQ>();
  const size_t lds = (static_cast<size_t>(kDownWaves) * a.T * kTileRows + a.T * a.k) * 4 + a.most_chosen * sizeof(MoeChosen);
  // the row sums of 64 tokens with the longest lists pass the default limit
  static const hipError_t attr =
      hipFuncSetAttribute(reinterpret_cast<const void*>(&moe_down_kernel<E, BITS, G, TQ>),
                          hipFuncAttributeMaxDynamicSharedMemorySize, kDownLds);
  if (attr != hipSuccess) return attr;
  moe_down_kernel<E, BITS, G, TQ><<<a.tiles_d, kDownWaves * kWave, lds, s>>>(a);
  return hipGetLastError();
}

template <class E, int BITS, int G>
hipError_t by_tokens(const MoeArgs& a, hipStream_t s) {
  if (a.T <= 4) return go<E, BITS, G, 1>(a, s);
  if (a.T <= 16) return go<E, BITS, G, 4>(a, s);
  return go<E, BITS, G, 8>(a, s);
}

template <class E>
hipError_t by_weights(const MoeArgs& a, hipStream_t s) {
  if (a.bits == 16) return by_tokens<E, 16, 1>(a, s);
  if (a.group == 32) return by_tokens<E, 4, 4>(a, s);
  if (a.group == 64) return by_tokens<E, 4, 2>(a, s);
  return by_tokens<E, 4, 1>(a, s);
}

}  // namespace

hipError_t launch_moe_route(const MoeArgs& a, int64_t T, int dtype, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(T));
  if (dtype == 0) moe_route_kernel<EF32><<<grid, kRouteWaves * kWave, 0, s>>>(a);
  else moe_route_kernel<EBf16><<<grid, kRouteWaves * kWave, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_moe_experts(const MoeArgs& a, int dtype, hipStream_t s) {
  return dtype == 0 ? by_weights<EF32>(a, s) : by_weights<EBf16>(a, s);
}

}  // namespace twell
