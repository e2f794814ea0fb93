// A mixture-of-experts gated feed-forward layer for a few tokens.
//
//   l[t,e] = x[t] . r[e] + b[e];  the top_k largest per token, softmax weights w
//   y[t]   = sum_i w_i  W_down_e ( act(W_gate_e x) * (W_up_e x) ),   e = ids[t,i]
//
// (1) moe_route_kernel: one workgroup per token, logits in fp32, selection by
// one wave (up to four tokens: moe_logits_kernel, or nothing).  (2)
// moe_up_kernel: one workgroup per (chosen expert, NT tiles of 16 neurons); it
// gathers the expert's tokens, computes gate and up together and writes h =
// w * act(g) * u.  (3) moe_down_kernel: one workgroup per
// (chosen expert, NT tiles of 16 outputs), writes every pair's part, and
// (4) moe_join_kernel adds them up in the order of the choices; few tokens with
// little to read take moe_down_few_kernel instead of both.
// Nothing depends on timing.  Only chosen experts' weights are read, each once
// per 16 of its tokens (by moe_down_few_kernel once per token).
//
// Bound by reading them.  16 tokens, 4 of 32 bf16 experts of 2048 x 1024: 68 us for
// 355 MB, of which up 40 (6.1 TB/s), down 22 (5.3), route 4.6, join 4.6.  64
// tokens, 8 of 64 in 4 bits: 66 us for 215 MB, of which up 32 (4.5 TB/s), down 24
// (2.9), route 6.0, join 4.7; unpacking keeps the vector units busy for half of up
// and a third of down, and down moves as many bytes of h, in two planes, as of
// codes.  One token, 2 of 8 bf16 experts of 1024 x 4096: 15.4 us for 50 MB, up 9.9
// and down 6.3, bound by starting and draining two launches of one round each, the
// second on 64 CUs.
#include "few_token.hpp"
#include "internal.hpp"

namespace twell {
namespace {

// Most waves of a workgroup of the up and down kernels (chosen at launch).
constexpr int kMostWaves = 8;

// ---------------------------------------------------------------- router
constexpr int kRouteWaves = 16;
constexpr int kRouteAhead = 4;  // experts a wave computes side by side

// Largest value over the 64 lanes (the steps of wave_sum).
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
  auto most = [](uint32_t a, int b) { return a > static_cast<uint32_t>(b) ? a : static_cast<uint32_t>(b); };
  v = most(v, dpp_take<0xB1>(static_cast<int>(v)));
  v = most(v, dpp_take<0x4E>(static_cast<int>(v)));
  v = most(v, dpp_take<0x141>(static_cast<int>(v)));
  v = most(v, dpp_take<0x140>(static_cast<int>(v)));
  v = most(v, dpp_take<0x142, 0xa>(static_cast<int>(v)));
  v = most(v, dpp_take<0x143, 0xc>(static_cast<int>(v)));
  return static_cast<uint32_t>(wave_last(static_cast<int>(v)));
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

// Eight inputs of a row.
template <class E>
struct Eight {
  u32x4_t v[E::kBytes / 2];
  __device__ __forceinline__ void load(const typename E::storage* p) {
    if constexpr (E::kBytes == 2) {
      v[0] = *reinterpret_cast<const u32x4_a2_t*>(p);
    } else {
      v[0] = *reinterpret_cast<const u32x4_a4_t*>(p);
      v[1] = *reinterpret_cast<const u32x4_a4_t*>(p + 4);
    }
  }
  // s += this . o; bf16 by pairs: products of bf16 values are exact in fp32
  __device__ __forceinline__ float dot(const Eight& o, float s) const {
    if constexpr (E::kBytes == 2) {
      const bf16x8_t a = __builtin_bit_cast(bf16x8_t, v[0]), b = __builtin_bit_cast(bf16x8_t, o.v[0]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        s = __builtin_amdgcn_fdot2_f32_bf16(bf16x2_t{a[2 * i], a[2 * i + 1]}, bf16x2_t{b[2 * i], b[2 * i + 1]}, s, false);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) s = fmaf(__uint_as_float(v[i >> 2][i & 3]), __uint_as_float(o.v[i >> 2][i & 3]), s);
    }
    return s;
  }
};

// s[j] += x . r[j] over inputs [k0, k0 + 512 U), eight per lane and 512; all
// loads ahead of all sums, since what bounds a wave is how much it has in flight.
template <class E, int U, int J>
__device__ __forceinline__ void route_dots(const typename E::storage* x, const typename E::storage* const (&r)[J], int k,
                                           float (&s)[J]) {
  Eight<E> xv[U], rv[U][J];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    xv[u].load(x + k + 512 * u);
#pragma unroll
    for (int j = 0; j < J; ++j) rv[u][j].load(r[j] + k + 512 * u);
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int j = 0; j < J; ++j) s[j] = xv[u].dot(rv[u][j], s[j]);
}

// Logits of token t and experts [e0, e0 + J), in every lane; of experts that do
// not exist: the last one's.
template <class E, int J>
__device__ __forceinline__ void route_logits(const MoeArgs& a, int64_t t, int e0, int lane, float (&s)[J]) {
  using Elem = typename E::storage;
  constexpr int U = E::kBytes == 2 ? 4 : 2;
  const Elem* x = static_cast<const Elem*>(a.x) + t * a.ldx;
  const Elem* r[J];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    r[j] = static_cast<const Elem*>(a.router) + static_cast<int64_t>(e0 + j < a.E ? e0 + j : a.E - 1) * a.d;
    s[j] = 0.f;
  }
  int k0 = 0;
  for (; k0 + 512 * U <= a.d; k0 += 512 * U) route_dots<E, U>(x, r, k0 + lane * 8, s);
  for (; k0 + 512 <= a.d; k0 += 512) route_dots<E, 1>(x, r, k0 + lane * 8, s);
  const int k = k0 + lane * 8;
  if (k + 8 <= a.d) {
    route_dots<E, 1>(x, r, k, s);
  } else {
    for (int i = k; i < a.d; ++i) {
      const float xv = load_elem<E>(x, i);
#pragma unroll
      for (int j = 0; j < J; ++j) s[j] = fmaf(xv, load_elem<E>(r[j], i), s[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < J; ++j) {
    s[j] = wave_sum(s[j]);
    if (a.bias) s[j] += a.bias[e0 + j < a.E ? e0 + j : a.E - 1];
  }
}

// A token's choices from its logits, by one wave: lane i < top_k has choice i.
struct Choice {
  int id;
  float weight;
  // a choice of weight 0 is no choice; a NaN weight is one
  __device__ __forceinline__ int live() const { return weight == 0.f ? -1 : id; }
};
template <int kRegs>  // kRegs * 64 >= E
__device__ __forceinline__ Choice choose(const MoeArgs& a, const float* logit, int lane) {
  float l[kRegs];  // expert e = 64 r + lane is in l[r] and key[r]
  uint32_t key[kRegs];
  uint32_t top = 0;
#pragma unroll
  for (int r = 0; r < kRegs; ++r) l[r] = r * 64 + lane < a.E ? logit[r * 64 + lane] : 0.f;
#pragma unroll
  for (int r = 0; r < kRegs; ++r) {
    key[r] = r * 64 + lane < a.E ? order_key(l[r]) : 0u;
    top = key[r] > top ? key[r] : top;
  }
  const float most = key_value(wave_umax(top));
  const bool none = most == -INFINITY;  // every expert is masked off: all weights 0
  float sum = 0.f;
#pragma unroll
  for (int r = 0; r < kRegs; ++r)
    if (r * 64 + lane < a.E) sum += expf(l[r] - most);
  sum = wave_sum(sum);

  uint32_t mine_key = 0;
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
        const int at = __builtin_ctzll(has);
        id = r * 64 + at;
        if (lane == at) key[r] = 0;
      }
    }
    if (lane == i) {
      mine_key = m;
      mine_id = id;
    }
  }
  float mine = lane < a.k && !none ? expf(key_value(mine_key) - most) / sum : 0.f;
  if (a.renorm && !none) mine /= wave_sum(mine);
  return {mine_id, mine};
}
__device__ __forceinline__ Choice choose(const MoeArgs& a, const float* logit, int lane) {
  if (a.E <= 64) return choose<1>(a, logit, lane);
  if (a.E <= 256) return choose<4>(a, logit, lane);
  return choose<kMoeMaxExperts / 64>(a, logit, lane);
}

__device__ __forceinline__ void tell_choice(const MoeArgs& a, int64_t t, const Choice& c, int lane) {
  if (lane >= a.k) return;
  a.ids[t * a.k + lane] = c.id;
  a.weights[t * a.k + lane] = c.weight;
  a.live[t * a.k + lane] = c.live();
}

// More than four tokens: a workgroup per token.  Bound by one CU's share of the
// L2's bandwidth: 6.0 us for 64 experts of d 2048, 4.6 for 32.
template <class E>
__global__ __launch_bounds__(kRouteWaves* kWave) void moe_route_kernel(MoeArgs a) {
  __shared__ float logit[kMoeMaxExperts];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = blockIdx.x;
  for (int e0 = wave * kRouteAhead; e0 < a.E; e0 += kRouteWaves * kRouteAhead) {
    float s[kRouteAhead];
    route_logits<E, kRouteAhead>(a, t, e0, lane, s);
#pragma unroll
    for (int j = 0; j < kRouteAhead; ++j)
      if (lane == 0 && e0 + j < a.E) logit[e0 + j] = s[j];
  }
  __syncthreads();
  if (wave == 0) tell_choice(a, t, choose(a, logit, lane), lane);
}

// Up to four tokens: a wave per logit spreads the router over the chip, 2.8 us
// for 256 KB of it where one workgroup takes 5.8, nearly all of it launch and one
// trip to memory; the up kernel's workgroups choose for themselves.
constexpr int kLogitWaves = 4;
template <class E>
__global__ __launch_bounds__(kLogitWaves* kWave) void moe_logits_kernel(MoeArgs a) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int e = blockIdx.x * kLogitWaves + wave, t = blockIdx.y;
  if (e >= a.E) return;
  float s[1];
  route_logits<E, 1>(a, t, e, lane, s);
  if (lane == 0) a.logits[t * a.E + e] = s[0];
}

// What a workgroup of the up kernel works out for itself for up to four tokens:
// the choices, and where that is a matter of one or two logits a wave the logits
// too (1 token, 2 of 8 experts, d 1024: 15.4 us for a call against 16.7; 4 of 16,
// d 2048: 12.4 against 12.9; 4 of 32: 13.5 against 12.9; 8 of 64: 22.7 against
// 16.6).  64 KB of router: 8 experts of d 4096 take 15.0 against 16.2; with 128 KB
// it is 18.4 against 19.4 for 8 of d 8192, and 15.3 either way for 16 of d 4096.
constexpr int kOwnPerWave = 2;
constexpr int64_t kOwnBytes = 64 << 10;
constexpr int kOwnLogits = kOwnPerWave * kMostWaves;
struct FewChoices {
  int live[4 * kMoeMaxTopK];
  float weight[4 * kMoeMaxTopK];
  float logit[kOwnLogits];
};
template <class E>
__device__ __forceinline__ void few_choose(const MoeArgs& a, FewChoices& c, int lane, int wave, int waves) {
  if (a.own_logits) {
    for (int i = wave; i < a.T * a.E; i += waves) {
      float s[1];
      route_logits<E, 1>(a, i / a.E, i % a.E, lane, s);
      if (lane == 0) c.logit[i] = s[0];
    }
    __syncthreads();
  }
  for (int t = wave; t < a.T; t += waves) {
    const Choice mine = a.own_logits ? choose(a, c.logit + t * a.E, lane) : choose(a, a.logits + t * a.E, lane);
    if (lane < a.k) {
      c.live[t * a.k + lane] = mine.live();
      c.weight[t * a.k + lane] = mine.weight;
    }
    if (blockIdx.x == 0 && blockIdx.y == 0) tell_choice(a, t, mine, lane);
  }
  __syncthreads();
}

// ---------------------------------------------------------------- expert lists
// Where one wave works out its expert and the expert's pairs.  Every wave does
// so for itself, without a barrier: the pairs come from the L2 once, and
// what follows are LDS and lane operations of a few hundred cycles.
struct alignas(16) WaveList {
  uint8_t taken[kMoeMaxExperts];  // more than 64 experts
  int pair[kMoeBlockTokens];
};

__device__ __forceinline__ uint32_t wave_or(uint32_t v) {
  v |= dpp_take<0xB1>(static_cast<int>(v));
  v |= dpp_take<0x4E>(static_cast<int>(v));
  v |= dpp_take<0x141>(static_cast<int>(v));
  v |= dpp_take<0x140>(static_cast<int>(v));
  v |= dpp_take<0x142, 0xa>(static_cast<int>(v));
  v |= dpp_take<0x143, 0xc>(static_cast<int>(v));
  return static_cast<uint32_t>(wave_last(static_cast<int>(v)));
}

// Pairs of a list of choices, kPairsAhead for each lane at once.
template <int kPairsAhead>
struct LivePairs {
  int id[kPairsAhead];
  __device__ __forceinline__ void fetch(const int* live, int pairs, int i0, int lane) {
#pragma unroll
    for (int u = 0; u < kPairsAhead; ++u) {
      const int i = i0 + u * 64 + lane;
      id[u] = live[i < pairs ? i : pairs - 1];  // all loads at once: no branch
    }
#pragma unroll
    for (int u = 0; u < kPairsAhead; ++u)
      if (i0 + u * 64 + lane >= pairs) id[u] = -1;
  }
  __device__ __forceinline__ void fetch(const MoeArgs& a, int i0, int lane) { fetch(a.live, a.T * a.k, i0, lane); }
};

// The `which`-th chosen expert (ascending), or -1 if there are not that many.
template <int kPairsAhead>
__device__ __forceinline__ int find_expert(const MoeArgs& a, LivePairs<kPairsAhead>& live, int which, WaveList& l,
                                           int lane) {
  const int pairs = a.T * a.k;
  int expert = -1, before = 0;  // chosen experts below the 64 looked at
  auto look = [&](int e0, uint64_t has) {
    const int c = __popcll(has);
    if (expert < 0 && which < before + c) {
      for (int i = before; i < which; ++i) has &= has - 1;
      expert = e0 + __builtin_ctzll(has);
    }
    before += c;
  };
  if (a.E <= 64) {
    uint32_t lo = 0, hi = 0;
    for (int i0 = 0; i0 < pairs; i0 += kPairsAhead * 64) {
      if (i0 > 0) live.fetch(a, i0, lane);
#pragma unroll
      for (int u = 0; u < kPairsAhead; ++u) {
        const uint32_t bit = live.id[u] < 0 ? 0u : 1u << (live.id[u] & 31);
        lo |= live.id[u] < 32 ? bit : 0u;
        hi |= live.id[u] < 32 ? 0u : bit;
      }
    }
    look(0, static_cast<uint64_t>(wave_or(hi)) << 32 | wave_or(lo));
  } else {
    reinterpret_cast<u32x4_t*>(l.taken)[lane] = u32x4_t{0, 0, 0, 0};
    lds_handoff();
    for (int i0 = 0; i0 < pairs; i0 += kPairsAhead * 64) {
      if (i0 > 0) live.fetch(a, i0, lane);
#pragma unroll
      for (int u = 0; u < kPairsAhead; ++u)
        if (live.id[u] >= 0) l.taken[live.id[u]] = 1;
    }
    lds_handoff();
    for (int e0 = 0; e0 < a.E; e0 += 64) look(e0, __ballot(l.taken[e0 + lane] != 0));
  }
  if (pairs > kPairsAhead * 64) live.fetch(a, 0, lane);
  return expert;
}

// The expert's (token, choice) pairs, ascending, into l.pair; returns how many.
// live: the first pairs.
template <int kPairsAhead>
__device__ __forceinline__ int find_pairs(const MoeArgs& a, LivePairs<kPairsAhead>& live, int expert, WaveList& l,
                                          int lane) {
  const int pairs = a.T * a.k;
  int n = 0;
  for (int i0 = 0; i0 < pairs; i0 += kPairsAhead * 64) {
    if (i0 > 0) live.fetch(a, i0, lane);
#pragma unroll
    for (int u = 0; u < kPairsAhead; ++u) {
      const uint64_t has = __ballot(live.id[u] == expert);
      if (live.id[u] == expert) l.pair[n + __popcll(has & ((1ull << lane) - 1))] = i0 + u * 64 + lane;
      n += __popcll(has);
    }
  }
  lds_handoff();
  return n;
}

// Token of a pair: pair / k, exact since (pair + 1/2) / k is at least 1/64 from
// every whole number and pair < 2^11.
__device__ __forceinline__ int64_t token_of(int pair, const MoeArgs& a) {
  return static_cast<int>((static_cast<float>(pair) + 0.5f) * a.inv_k);
}

// Waves a SIMD that the registers are to leave room for: four, but three where
// four spill and that shows, which is with fp32 data and 16-bit weights (64 tokens,
// 4 of 16 experts of 1500 x 700: 62 us against 77) and in the down kernel with
// fp32 data (the same in 4 bits: 55 us against 60; the up kernel gains and loses
// by it).  With four, the down kernel for bf16 data and 4 bits keeps 10 to 19
// registers in memory, and still that is the better on most sizes: 64 tokens, 8 of
// 64 experts of 2048 x 1024 66 us against 69 with three, 4 tokens 34 against 38, 48
// tokens, 2 of 8 of 1024 x 4096 35 against 33.  Up with fp32 data and 4 bits keeps 2
// to 6 in memory, down 5.
template <class E, int BITS, bool DOWN>
constexpr int least_waves() { return E::kBytes == 4 && (BITS == 16 || DOWN) ? 3 : 4; }

// LDS of one wave: its list, and its token pieces or, after them, its sums.
template <class Prod>
constexpr int wave_lds() { return Prod::kAll * 256 > Prod::X::kLdsBytes ? Prod::kAll * 256 : Prod::X::kLdsBytes; }

// ---------------------------------------------------------------- gate and up
template <class E, int BITS, int G, int TQ, int NT, bool STREAM>
using UpProduct = Product<BITS, G, TQ, 2 * NT, std::conditional_t<E::kBytes == 2, SourceBf16, SourceF32>, STREAM>;

template <int NT>
using Tiles = Tile[NT];

template <int BITS, int G, int NT>
__device__ __forceinline__ void up_tiles(const MoeArgs& a, int expert, int ti, Tiles<2 * NT>& tile) {
#pragma unroll
  for (int r = 0; r < NT; ++r) {
    const int i = ti + r < a.tiles_f ? ti + r : a.tiles_f - 1;
    const int64_t blk = (static_cast<int64_t>(expert) * a.tiles_f + i) * a.blocks_d;
    tile[2 * r] = {a.gate_codes + blk * Block<BITS>::kBytes, a.gate_scales + blk * (16 * G)};
    tile[2 * r + 1] = {a.up_codes + blk * Block<BITS>::kBytes, a.up_scales + blk * (16 * G)};
  }
}

// h = w act(g) u for n <= 4 TQ pairs of one expert and the neurons of NT tiles
// from tile ti on.  lds: wave_lds per wave.
template <class E, int BITS, int G, int TQ, int NT, bool kFew = false>
__device__ __forceinline__ void up_pairs(const MoeArgs& a, const Tiles<2 * NT>& tile, int ti, const int* pair, int n,
                                         const float* weights, char* lds, int lane, int wave, int waves) {
  using Elem = typename E::storage;
  using Prod = UpProduct<E, BITS, G, TQ, NT, !kFew>;
  constexpr int kOne = Prod::kRegs;  // registers of one tile
  const typename Prod::X x(
      {a.d},
      [&](int i) { return static_cast<const Elem*>(a.x) + token_of(pair[i < n ? i : 0], a) * a.ldx; },
      lds + wave * Prod::X::kLdsBytes, lane);
  float* red = reinterpret_cast<float*>(lds);
  Prod p;
  p.clear();
  p.template run<(E::kBytes == 2 && kFew ? 2 : 1)>(x, tile, a.blocks_d * wave / waves,
                                                      a.blocks_d * (wave + 1) / waves, a.d / kBlockK, lane);
  __syncthreads();  // the token pieces have been read
  p.put(red, wave, lane);
  __syncthreads();
  for (int o = threadIdx.x; o < NT * kOne * 64; o += waves * kWave) {
    const int r = o / (kOne * 64), l = o & 63;
    const int i = result_token(o / 64 % kOne, l);
    if (i >= n) continue;
    const float g = joined<Prod::kAll>(red, waves, o + r * kOne * 64);
    const float u = joined<Prod::kAll>(red, waves, o + (r + 1) * kOne * 64);
    // a NaN gate stays NaN under both activations
    const float act = a.act == 0 ? (g < 0.f ? 0.f : g) : g / (1.f + expf(-g));
    float h = weights[pair[i]] * act * u;
    if (ti + r >= a.tiles_f) h = 0.f;  // neurons that fill the last block of 128
    // the down projection reads h as bf16 values whose sum is h: three keep all 24
    // bits for fp32; two keep 16, which moves a bf16 y by 1e-4 of its norm where its
    // own rounding moves it by 1.7e-3 (with 24 bits for it 64 tokens in 4 bits take
    // 72.6 us instead of 66.9, one token 16.6 instead of 15.4)
    uint16_t* out = a.h + static_cast<int64_t>(pair[i]) * a.h_row + (ti + r) * kTileRows + (l & 15);
#pragma unroll
    for (int s = 0; s < (E::kBytes == 2 ? 2 : 3); ++s) {
      const uint16_t b = bf16_of(h);
      out[s * a.h_plane] = b;
      h -= bf16_bits_to_f32(b);
    }
  }
}

// The row's expert and pairs for the down kernel.
__device__ __forceinline__ void hand_on(const MoeArgs& a, int expert, int n, const WaveList& list, int lane, int wave) {
  if (blockIdx.x != 0 || wave != 0) return;
  if (lane == 0) a.chosen[blockIdx.y] = MoeChosen{expert, n};
  if (lane < n) a.chosen_pairs[blockIdx.y * kMoeBlockTokens + lane] = list.pair[lane];
}

// One workgroup per expert and NT tiles of gate and up alike, so that act(g) * u
// needs no pass of its own; its waves split the inputs.  kFew: up to four tokens.
// Where there are at least as many pairs as experts, nearly every expert has a
// token: row y of the grid is then expert y, which needs no search.
template <class E, int BITS, int G, bool kFew, int NT>
__global__ __launch_bounds__(kMostWaves* kWave, (least_waves<E, BITS, false>())) void moe_up_kernel(MoeArgs a) {
  __shared__ WaveList lists[kMostWaves];
  extern __shared__ __align__(16) char lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const int ti = blockIdx.x * NT;
  WaveList& list = lists[wave];
  LivePairs<(kFew ? 2 : 8)> live;
  Tiles<2 * NT> tile;
  if constexpr (kFew) {
    __shared__ FewChoices choices;
    few_choose<E>(a, choices, lane, wave, waves);
    live.fetch(choices.live, a.T * a.k, 0, lane);
    const int expert = find_expert(a, live, blockIdx.y, list, lane);
    const int n = expert < 0 ? 0 : find_pairs(a, live, expert, list, lane);
    hand_on(a, expert, n, list, lane, wave);
    if (n == 0) return;  // the whole workgroup
    up_tiles<BITS, G, NT>(a, expert, ti, tile);
    up_pairs<E, BITS, G, 1, NT, true>(a, tile, ti, list.pair, n, choices.weight, lds, lane, wave, waves);
  } else {
    live.fetch(a, 0, lane);
    const int expert = a.by_expert ? static_cast<int>(blockIdx.y) : find_expert(a, live, blockIdx.y, list, lane);
    const int n = expert < 0 ? 0 : find_pairs(a, live, expert, list, lane);
    hand_on(a, expert, n, list, lane, wave);
    if (n == 0) return;
    up_tiles<BITS, G, NT>(a, expert, ti, tile);
    if (n <= 4) {
      up_pairs<E, BITS, G, 1, NT>(a, tile, ti, list.pair, n, a.weights, lds, lane, wave, waves);
    } else if (n <= 8) {
      up_pairs<E, BITS, G, 2, NT>(a, tile, ti, list.pair, n, a.weights, lds, lane, wave, waves);
    } else {
      for (int i = 0; i < n; i += 16) {
        if (i > 0) __syncthreads();
        up_pairs<E, BITS, G, 4, NT>(a, tile, ti, list.pair + i, n - i < 16 ? n - i : 16, a.weights, lds, lane, wave,
                                    waves);
      }
    }
  }
}

// ---------------------------------------------------------------- down
// The planes that hold h.
template <class E>
constexpr int h_planes() { return E::kBytes == 2 ? 2 : 3; }
template <class E, int BITS, int G, int TQ, int NT>
using DownProduct = Product<BITS, G, TQ, NT, SourcePlanes<h_planes<E>()>, true>;

// z[pair] = W_down_e h[pair] (the weight is in h already) for n <= 4 TQ pairs of one expert and the outputs
// of NT tiles from tile ti on.
template <class E, int BITS, int G, int TQ, int NT>
__device__ __forceinline__ void down_pairs(const MoeArgs& a, const Tiles<NT>& tile, int ti, const int* pair, int n,
                                           char* lds, int lane, int wave, int waves) {
  using Prod = DownProduct<E, BITS, G, TQ, NT>;
  constexpr int kOne = Prod::kRegs;
  const typename Prod::X x(
      {a.h_plane}, [&](int i) { return a.h + static_cast<int64_t>(pair[i < n ? i : 0]) * a.h_row; },
      lds + wave * Prod::X::kLdsBytes, lane);
  float* red = reinterpret_cast<float*>(lds);
  Prod p;
  p.clear();
  p.template run<1>(x, tile, a.blocks_f * wave / waves, a.blocks_f * (wave + 1) / waves, a.blocks_f, lane);
  __syncthreads();  // the token pieces have been read
  p.put(red, wave, lane);
  __syncthreads();
  for (int o = threadIdx.x; o < NT * kOne * 64; o += waves * kWave) {
    const int r = o / (kOne * 64), l = o & 63;
    const int i = result_token(o / 64 % kOne, l);
    const int out = (ti + r) * kTileRows + (l & 15);
    if (i < n && out < a.d) a.z[static_cast<int64_t>(pair[i]) * a.d + out] = joined<Prod::kAll>(red, waves, o);
  }
}

template <class E, int BITS, int G, int NT>
__global__ __launch_bounds__(kMostWaves* kWave, (least_waves<E, BITS, true>())) void moe_down_kernel(MoeArgs a) {
  extern __shared__ __align__(16) char lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const int ti = blockIdx.x * NT;
  const MoeChosen c = a.chosen[blockIdx.y];
  const int expert = __builtin_amdgcn_readfirstlane(c.expert), n = __builtin_amdgcn_readfirstlane(c.n);
  if (n == 0) return;
  Tiles<NT> tile;
#pragma unroll
  for (int r = 0; r < NT; ++r) {
    const int i = ti + r < a.tiles_d ? ti + r : a.tiles_d - 1;
    const int64_t blk = (static_cast<int64_t>(expert) * a.tiles_d + i) * a.blocks_f;
    tile[r] = {a.down_codes + blk * Block<BITS>::kBytes, a.down_scales + blk * (16 * G)};
  }
  const int* pair = a.chosen_pairs + blockIdx.y * kMoeBlockTokens;
  if (n <= 4) {
    down_pairs<E, BITS, G, 1, NT>(a, tile, ti, pair, n, lds, lane, wave, waves);
  } else if (n <= 8) {
    down_pairs<E, BITS, G, 2, NT>(a, tile, ti, pair, n, lds, lane, wave, waves);
  } else {
    for (int i = 0; i < n; i += 16) {
      if (i > 0) __syncthreads();
      down_pairs<E, BITS, G, 4, NT>(a, tile, ti, pair + i, n - i < 16 ? n - i : 16, lds, lane, wave, waves);
    }
  }
}

// y[t] = sum over the choices of z, in the order of the choices; z in fp32, since
// it is rounded once as y.  Bound by launch and latency: 4.7 us for 4 MB of z.
template <class E>
__global__ __launch_bounds__(256) void moe_join_kernel(MoeArgs a) {
  constexpr int U = 8;
  const int n = blockIdx.x * 256 + threadIdx.x;
  const int64_t t = blockIdx.y;
  if (n >= a.d) return;
  const int* live = a.live + t * a.k;
  const float* z = a.z + t * a.k * a.d + n;
  float v = 0.f;
  for (int i0 = 0; i0 < a.k; i0 += U) {
    float part[U];
    bool on[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u < a.k ? i0 + u : a.k - 1;
      part[u] = z[static_cast<int64_t>(i) * a.d];  // of a choice that does not count: anything
      on[u] = (i0 + u < a.k) & (live[i] >= 0);  // no branch: all loads at once
    }
#pragma unroll
    for (int u = 0; u < U; ++u) v += on[u] ? part[u] : 0.f;
  }
  const int64_t at = t * a.ldy + n;
  if constexpr (E::kBytes == 2) static_cast<uint16_t*>(a.y)[at] = bf16_of(v);
  else static_cast<float*>(a.y)[at] = v;
}

// Few tokens and little to read: one workgroup per 16 outputs takes all pairs,
// its waves splitting (pair, block) among them, and writes y at once.  A pair's
// h is every row of the matrix operand, so that all lane groups hold its result;
// group t % 4 adds it to the sum of token t, so a token's choices come together
// in one register.  TQ: quads of tokens.
constexpr int kFewWaves = 16;
// (pair, block)s that it takes at the most (one_down), of which each wave has its
// share on the way at once.
template <class E>
constexpr int few_blocks() { return E::kBytes == 2 ? 64 : 32; }

template <class E, int BITS, int G, int TQ>
__global__ __launch_bounds__(kFewWaves* kWave) void moe_down_few_kernel(MoeArgs a) {
  constexpr int P = E::kBytes == 2 ? 2 : 3;
  using Prod = Product<BITS, G, 1, 1, SourcePlanes<P>>;
  static_assert(Prod::kAll == 1);
  __shared__ __align__(16) char lds[kFewWaves * Prod::X::kLdsBytes];
  __shared__ float red[kFewWaves * TQ * 64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ti = blockIdx.x;
  const int total = a.T * a.k * a.blocks_f;
  int b = total * wave / kFewWaves;
  const int end = total * (wave + 1) / kFewWaves;
  float sum[TQ] = {};
  while (b < end) {
    const int pair = b / a.blocks_f, b0 = b % a.blocks_f;
    const int b1 = b0 + (end - b) < a.blocks_f ? b0 + (end - b) : a.blocks_f;
    b += b1 - b0;
    const int expert = a.live[pair];
    if (expert < 0) continue;
    const typename Prod::X x(
        {a.h_plane}, [&](int) { return a.h + static_cast<int64_t>(pair) * a.h_row; },
        lds + wave * Prod::X::kLdsBytes, lane);
    const int64_t blk = (static_cast<int64_t>(expert) * a.tiles_d + ti) * a.blocks_f;
    const Tile tile[1] = {{a.down_codes + blk * Block<BITS>::kBytes, a.down_scales + blk * (16 * G)}};
    Prod p;
    p.clear();
    p.template run<few_blocks<E>() / kFewWaves>(x, tile, b0, b1, b1, lane);
    const int t = pair / a.k;
#pragma unroll
    for (int q = 0; q < TQ; ++q)
      if (result_token(q, lane) == t) sum[q] += p.acc[0][0][0];
  }
#pragma unroll
  for (int q = 0; q < TQ; ++q) red[(wave * TQ + q) * 64 + lane] = sum[q];
  __syncthreads();
  if (wave >= TQ) return;
  const int t = result_token(wave, lane), n = ti * kTileRows + (lane & 15);
  if (t < a.T && n < a.d) {
    const float v = joined<TQ>(red, kFewWaves, threadIdx.x);
    const int64_t at = static_cast<int64_t>(t) * a.ldy + n;
    if constexpr (E::kBytes == 2) static_cast<uint16_t*>(a.y)[at] = bf16_of(v);
    else static_cast<float*>(a.y)[at] = v;
  }
}

template <class E>
hipError_t go_route(const MoeArgs& a, hipStream_t s) {
  if (a.T > 4) return launch(moe_route_kernel<E>, dim3(static_cast<unsigned>(a.T)), kRouteWaves * kWave, 0, s, a);
  if (a.own_logits) return hipSuccess;
  const dim3 grid(static_cast<unsigned>((a.E + kLogitWaves - 1) / kLogitWaves), static_cast<unsigned>(a.T));
  return launch(moe_logits_kernel<E>, grid, kLogitWaves * kWave, 0, s, a);
}

// Waves per workgroup: as few as still make kFillWaves waves.  A workgroup's
// waves wait for each other twice, so what fills the chip with single waves
// streams best.  Half as many and twice as many waves are slower: 64 tokens, 8 of
// 64 experts of 2048 x 1024 in 4 bits 65.4 us against 68.0 and 68.4, 512 tokens 541
// against 581 and 556, 1 token, 2 of 8 of 1024 x 4096 12.8 against 13.7 and 12.8;
// but not with fp32 data, whose waves hold more: 64 tokens, 4 of 16 bf16 experts of
// 1500 x 700 62.2 against 55.6 with half as many.
constexpr int64_t kFillWaves = 4096;
int waves_for(int64_t groups, int blocks) {
  int w = 1;
  while (w < kMostWaves && w < blocks && groups * w < kFillWaves) w <<= 1;
  return w;
}

template <class E, int BITS, int G, bool kFew, int NT>
hipError_t go_choices_up(MoeArgs a, hipStream_t s) {
  // the tiles that fill the last block of neurons are written too
  const dim3 grid(static_cast<unsigned>(a.blocks_f * (kBlockK / kTileRows) / NT), static_cast<unsigned>(a.most_chosen));
  constexpr int kLds = wave_lds<UpProduct<E, BITS, G, kFew ? 1 : 4, NT, !kFew>>();
  const int w = waves_for(static_cast<int64_t>(grid.x) * grid.y, a.blocks_d);
  a.own_logits = kFew && a.T * a.E <= kOwnPerWave * w && static_cast<int64_t>(a.T) * a.E * a.d * E::kBytes <= kOwnBytes;
  const hipError_t e = go_route<E>(a, s);
  if (e != hipSuccess) return e;
  return launch_lds<&moe_up_kernel<E, BITS, G, kFew, NT>, kMostWaves * kLds>(grid, w * kWave, w * kLds, s, a);
}

template <class E, int BITS, int G, int NT>
hipError_t go_down(const MoeArgs& a, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>((a.tiles_d + NT - 1) / NT), static_cast<unsigned>(a.most_chosen));
  constexpr int kLds = wave_lds<DownProduct<E, BITS, G, 4, NT>>();
  const int w = waves_for(static_cast<int64_t>(grid.x) * grid.y, a.blocks_f);
  const hipError_t e = launch_lds<&moe_down_kernel<E, BITS, G, NT>, kMostWaves * kLds>(grid, w * kWave, w * kLds, s, a);
  if (e != hipSuccess) return e;
  const dim3 join(static_cast<unsigned>((a.d + 255) / 256), static_cast<unsigned>(a.T));
  return launch(moe_join_kernel<E>, join, 256, 0, s, a);
}

// Up to so many (pair, block)s for a workgroup, and bytes in all, few tokens take the
// one kernel: it reads an expert's weights once per pair, on as many CUs as there
// are tiles of outputs, but saves a launch and the way of the parts through memory.
// Whole calls, this one against the other: 1 token, 2 of 8 experts of 1024 x 4096
// (64 blocks) 15.4 against 18.1 us in bf16, 12.8 against 14.9 in 4 bits; 8 tokens, 1
// of 4 in 4 bits, 512 x 512 (32) 10.8 against 11.6; 16 tokens, 1 of 8, 1024 x 512
// (64) 13.2 against 13.2, in fp32 14.7 against 13.6; 5 tokens, 3 of 7, 1001 x 707
// (90) 16.1 against 14.6.  Beyond 24 MB it depends on what is in the caches: 1 token,
// 2 of 8 bf16 experts of 2048 x 4096 (32 MB) 25.5 against 24.6 with the weights of
// three calls before still there, 25.9 against 27.2 with those of twelve.
template <class E>
bool one_down(const MoeArgs& a, int block_bytes) {
  const int64_t blocks = static_cast<int64_t>(a.T) * a.k * a.blocks_f;
  return a.T <= 16 && blocks <= few_blocks<E>() && blocks * a.tiles_d * block_bytes <= int64_t(24) << 20;
}

// Whether NT of `tiles` tiles a workgroup leave work for most CUs, three quarters:
// more tiles share the tokens' way through LDS, fewer give more CUs something to
// read.  With half of the CUs 4 tokens, 2 of 8 experts of 1024 x 4096 in 4 bits take
// 26.8 us against 24.1 and 16, 1 of 8 of 1024 x 512, 14.0 against 13.2 (but 40, 2 of
// 8 of 1024 x 700, 18.5 against 19.3); with all of them 5 tokens, 3 of 7 of 1001 x
// 707, 15.0 against 14.6.
bool fills(const MoeArgs& a, int cus, int tiles, int NT) {
  return static_cast<int64_t>((tiles + NT - 1) / NT) * a.most_chosen * 4 >= int64_t(3) * cus;
}

template <class E, int BITS, int G>
hipError_t by_tokens(const MoeArgs& a, hipStream_t s) {
  constexpr bool kSlim = BITS == 4 && E::kBytes == 2;  // room for twice the tiles in registers
  const int resident = lockstep_resident(), cus = resident > 0 ? resident : 256;
  hipError_t e;
  if (a.T <= 4) {
    e = go_choices_up<E, BITS, G, true, 1>(a, s);
  } else if (kSlim && fills(a, cus, a.blocks_f * (kBlockK / kTileRows), 2)) {
    e = go_choices_up<E, BITS, G, false, kSlim ? 2 : 1>(a, s);
  } else {
    e = go_choices_up<E, BITS, G, false, 1>(a, s);
  }
  if (e != hipSuccess) return e;
  if (one_down<E>(a, Block<BITS>::kBytes)) {
    return launch(a.T <= 4 ? moe_down_few_kernel<E, BITS, G, 1> : moe_down_few_kernel<E, BITS, G, 4>, dim3(a.tiles_d),
                  kFewWaves * kWave, 0, s, a);
  }
  if (kSlim && fills(a, cus, a.tiles_d, 4)) return go_down<E, BITS, G, kSlim ? 4 : 2>(a, s);
  if (fills(a, cus, a.tiles_d, 2)) return go_down<E, BITS, G, 2>(a, s);
  return go_down<E, BITS, G, 1>(a, s);
}

template <class E>
hipError_t by_weights(const MoeArgs& a, hipStream_t s) {
  if (a.bits == 16) return by_tokens<E, 16, 1>(a, s);
  if (a.group == 32) return by_tokens<E, 4, 4>(a, s);
  if (a.group == 64) return by_tokens<E, 4, 2>(a, s);
  return by_tokens<E, 4, 1>(a, s);
}

}  // namespace

hipError_t launch_moe(const MoeArgs& a, int dtype, hipStream_t s) {
  return dtype == 0 ? by_weights<EF32>(a, s) : by_weights<EBf16>(a, s);
}

}  // namespace twell
