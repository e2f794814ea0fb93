// Tokens to their experts and back: the order of (token, choice) pairs by
// expert, the rows moved there, and the weighted sums back, with gradients.
//
// A pair p = t * k + i is choice i of token t.  Pairs are sorted by expert,
// stably, and row pair_row[p] of the sorted rows belongs to pair p (-1: the
// pair's expert is not one of 0 .. E-1, so it has no row).
#include "internal.hpp"
#include "launch.hpp"
#include "rows.hpp"

namespace twell {
namespace {

// ------------------------------------------------------------------ sorting
// A counting sort.  Each workgroup has a run of pairs and each of its waves a
// run of those.  Counting needs no order (whole numbers added in LDS come out
// the same whatever the order); a pair's place then is: rows of lower experts
// + this expert's pairs in earlier workgroups + in earlier waves + in earlier
// rounds of the wave + in lower lanes of the round.
constexpr int kSortWaves = 16;
constexpr int kSortMostBlocks = 256;
constexpr int kSortAlone = 4096;  // pairs that one workgroup sorts alone, in one launch (6.0 us replayed; 16000: 15.4)
constexpr int kSortRun = 2048;    // else pairs of a workgroup, at the least (131072 of 64 experts in us: 11.3 with 1024,
                                  // 9.8, 10.4 with 4096; 16000: 7.0, 7.6, 7.8)
// With many experts adding up the counts of all workgroups, in each of them, shows: 131072 pairs of 64, 256 and 1024
// experts take 9.9, 11.4 and 15.0 us, 2^25 pairs of 64 and 1024 experts 193 and 225.

__device__ __forceinline__ void wave_handoff() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

struct SortRun {
  int64_t begin, end;  // pairs of this wave
};
__device__ __forceinline__ SortRun sort_run(const TokensSortArgs& a, int wave, int waves) {
  const int64_t first = static_cast<int64_t>(blockIdx.x) * a.run;
  const int64_t last = min(first + a.run, a.pairs);
  const int64_t each = ((a.run + waves - 1) / waves + 63) / 64 * 64;
  const int64_t b = min(first + wave * each, last);
  return {b, min(b + each, last)};
}

__device__ __forceinline__ int expert_of(const TokensSortArgs& a, int64_t p, int64_t end) {
  const int e = p < end ? a.ids[p] : -1;
  return static_cast<uint32_t>(e) < static_cast<uint32_t>(a.E) ? e : a.E;
}

// counts[wave][e]: pairs of each wave, then of the waves before it (in place);
// total(e, n) gets the workgroup's own number.
template <class Total>
__device__ __forceinline__ void count_waves(const TokensSortArgs& a, int* counts, Total total) {
  const int waves = blockDim.x >> 6, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int i = threadIdx.x; i < waves * a.E; i += blockDim.x) counts[i] = 0;
  __syncthreads();
  const SortRun r = sort_run(a, wave, waves);
  for (int64_t p = r.begin; p < r.end; p += 64) {
    const int e = expert_of(a, p + lane, r.end);
    if (e < a.E) atomicAdd(&counts[wave * a.E + e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
    int n = 0;
    for (int w = 0; w < waves; ++w) {
      const int c = counts[w * a.E + e];
      counts[w * a.E + e] = n;
      n += c;
    }
    total(e, n);
  }
}

__global__ __launch_bounds__(kSortWaves* kWave) void tokens_count_kernel(TokensSortArgs a) {
  extern __shared__ __align__(16) int lds_counts[];
  int* mine = a.hist + static_cast<int64_t>(blockIdx.x) * a.E;
  count_waves(a, lds_counts, [&](int e, int n) { mine[e] = n; });
}

// Every workgroup counts its waves' pairs again and adds up what is before it.
// lds: counts [waves][E], base [E], starts [E].
__global__ __launch_bounds__(kSortWaves* kWave) void tokens_place_kernel(TokensSortArgs a) {
  extern __shared__ __align__(16) int lds_counts[];
  const int waves = blockDim.x >> 6, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  int* base = lds_counts + waves * a.E;
  int* starts = base + a.E;
  const int blocks = gridDim.x;
  count_waves(a, lds_counts, [&](int e, int n) {
    int before = 0, all = n;
    if (blocks > 1) {
      all = 0;
#pragma unroll 8
      for (int b = 0; b < blocks; ++b) {
        const int c = a.hist[static_cast<int64_t>(b) * a.E + e];
        before += b < static_cast<int>(blockIdx.x) ? c : 0;
        all += c;
      }
    }
    base[e] = before;
    starts[e] = all;
  });
  __syncthreads();
  if (wave == 0) {  // exclusive sums over the experts
    int carry = 0;
    for (int e0 = 0; e0 < a.E; e0 += 64) {
      const int e = e0 + lane;
      const int n = e < a.E ? starts[e] : 0;
      const int in = wave_incl_scan(n);
      if (e < a.E) {
        base[e] += carry + in - n;
        if (blockIdx.x == 0) a.offsets[e] = carry + in - n;
      }
      carry += wave_last(in);
    }
    if (blockIdx.x == 0 && lane == 0) a.offsets[a.E] = carry;
  }
  __syncthreads();
  const SortRun r = sort_run(a, wave, waves);
  int* mine = lds_counts + wave * a.E;
  const uint64_t below = (uint64_t(1) << lane) - 1;
  for (int64_t p0 = r.begin; p0 < r.end; p0 += 64) {
    const int64_t p = p0 + lane;
    const int e = expert_of(a, p, r.end);
    uint64_t same = ~uint64_t(0);  // lanes with this lane's expert
    for (int bit = 0; bit < a.bits; ++bit) {
      const bool on = (e >> bit) & 1;
      const uint64_t m = __ballot(on);
      same &= on ? m : ~m;
    }
    const bool live = e < a.E;
    const int first = live ? mine[e] : 0;
    wave_handoff();
    if (live && (same & below) == 0) mine[e] = first + __popcll(same);
    wave_handoff();
    if (p < r.end) a.pair_row[p] = live ? base[e] + first + __popcll(same & below) : -1;
  }
}

// ------------------------------------------------------------------ rows
// All three kernels are bound by the rows they read and write; nothing is
// computed that takes as long.  A wave has a piece of one token: what a token
// reads or writes once (x, y, dy) is then touched once, and its k rows are read
// or written whole lines at a time, all their loads in flight together.  16384
// tokens of 2048 in bf16, 8 choices each: gather 114 us, combine 118, its gradient
// 231, which is 5.3, 5.1 and 4.9 TB/s, where a copy of 2 GiB reaches 4.9.

// Row of a pair, or -1.  The bound keeps a list that was not made by the sort
// from leading outside the rows.
__device__ __forceinline__ int row_of(const TokensArgs& a, int64_t pair) {
  const int r = a.pair_row[pair];
  return static_cast<uint32_t>(r) < static_cast<uint32_t>(a.pairs) ? r : -1;
}

constexpr int kRowWaves = 4;

struct WavePiece {
  int64_t t;
  int c;  // first element of this lane's first 16 bytes
};
template <class E, int U>
__device__ __forceinline__ bool wave_piece(const TokensArgs& a, WavePiece& w) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kRowWaves + wave;
  w.t = id / a.pieces;
  w.c = (static_cast<int>(id % a.pieces) * U * kWave + (threadIdx.x & 63)) * Piece<E>::kN;
  return w.t < a.T;
}

template <class E, int U>
__global__ __launch_bounds__(kRowWaves* kWave) void tokens_gather_kernel(TokensArgs a) {
  using S = typename E::storage;
  WavePiece w;
  if (!wave_piece<E, U>(a, w)) return;
  const S* x = static_cast<const S*>(a.x) + w.t * a.ld_tokens;
  constexpr int kStep = kWave * Piece<E>::kN;
  u32x4_t v[U];
#pragma unroll
  for (int u = 0; u < U; ++u) v[u] = load_piece<E>(x, w.c + u * kStep, a.d);
  for (int i = 0; i < a.k; ++i) {
    const int r = row_of(a, w.t * a.k + i);
    if (r < 0) continue;
    S* to = static_cast<S*>(a.rows_out) + static_cast<int64_t>(r) * a.ld_out;
#pragma unroll
    for (int u = 0; u < U; ++u) store_piece<E>(to, w.c + u * kStep, a.d, v[u]);
  }
}

// Sums in fp32, choices in their order; one rounding.
template <class E, int U>
__global__ __launch_bounds__(kRowWaves* kWave) void tokens_combine_kernel(TokensArgs a) {
  using S = typename E::storage;
  using P = Piece<E>;
  WavePiece w;
  if (!wave_piece<E, U>(a, w)) return;
  constexpr int kStep = kWave * P::kN;
  constexpr int kAhead = 8 / U;  // choices whose loads are in flight together
  float sum[U][P::kN];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int j = 0; j < P::kN; ++j) sum[u][j] = 0.f;
  for (int i0 = 0; i0 < a.k; i0 += kAhead) {
    u32x4_t v[kAhead][U];
    float wt[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t p = w.t * a.k + i0 + i;
      const int r = i0 + i < a.k ? row_of(a, p) : -1;
      wt[i] = r < 0 ? 0.f : a.weights ? a.weights[p] : 1.f;
#pragma unroll
      for (int u = 0; u < U; ++u) v[i][u] = u32x4_t{0, 0, 0, 0};
      if (wt[i] != 0.f) {  // a weight of 0 adds nothing, whatever its row holds
        const S* from = static_cast<const S*>(a.rows) + static_cast<int64_t>(r) * a.ld_rows;
#pragma unroll
        for (int u = 0; u < U; ++u) v[i][u] = load_piece<E>(from, w.c + u * kStep, a.d);
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float f[P::kN];
        P::unpack(v[i][u], f);
#pragma unroll
        for (int j = 0; j < P::kN; ++j) sum[u][j] = fmaf(wt[i], f[j], sum[u][j]);
      }
  }
  S* y = static_cast<S*>(a.y) + w.t * a.ld_tokens;
#pragma unroll
  for (int u = 0; u < U; ++u) store_piece<E>(y, w.c + u * kStep, a.d, P::pack(sum[u]));
}

// drows[r] = w dy[t], dweights[p] = rows[r] . dy[t].  A wave has a whole token, or,
// of few tokens, one of its choices (a.pieces waves a token); dy stays in registers
// where U x 1 KB hold it (KEEP), else it is read again for each choice, from the caches.
template <class E, int U, bool KEEP>
__global__ __launch_bounds__(kRowWaves* kWave) void tokens_combine_bwd_kernel(TokensArgs a) {
  using S = typename E::storage;
  using P = Piece<E>;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kRowWaves + wave;
  const int64_t t = id / a.pieces;
  if (t >= a.T) return;
  const int lane = threadIdx.x & 63;
  constexpr int kStep = kWave * P::kN;
  const S* dy = static_cast<const S*>(a.dy) + t * a.ld_tokens;
  u32x4_t g[U];
  if constexpr (KEEP) {
#pragma unroll
    for (int u = 0; u < U; ++u) g[u] = load_piece<E>(dy, lane * P::kN + u * kStep, a.d);
  }
  for (int i = static_cast<int>(id % a.pieces); i < a.k; i += a.pieces) {
    const int64_t p = t * a.k + i;
    const int r = row_of(a, p);
    float dot = 0.f;
    if (r >= 0) {
      const float wt = a.weights[p];
      const S* row = static_cast<const S*>(a.rows) + static_cast<int64_t>(r) * a.ld_rows;
      S* to = a.rows_out ? static_cast<S*>(a.rows_out) + static_cast<int64_t>(r) * a.ld_out : nullptr;
      for (int c0 = lane * P::kN; c0 < (KEEP ? lane * P::kN + 1 : a.d); c0 += U * kStep) {
        u32x4_t v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if constexpr (!KEEP) g[u] = load_piece<E>(dy, c0 + u * kStep, a.d);
          v[u] = a.dweights ? load_piece<E>(row, c0 + u * kStep, a.d) : u32x4_t{0, 0, 0, 0};
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float f[P::kN], h[P::kN];
          P::unpack(v[u], f);
          P::unpack(g[u], h);
#pragma unroll
          for (int j = 0; j < P::kN; ++j) {
            dot = fmaf(f[j], h[j], dot);
            h[j] *= wt;
          }
          if (to) store_piece<E>(to, c0 + u * kStep, a.d, P::pack(h));
        }
      }
    }
    if (a.dweights) {
      dot = wave_sum(dot);
      if (lane == 0) a.dweights[p] = dot;
    }
  }
}

template <class E, int U>
unsigned piece_grid(TokensArgs& a) {
  const int per = U * kWave * Piece<E>::kN;
  a.pieces = (a.d + per - 1) / per;
  return static_cast<unsigned>((a.T * a.pieces + kRowWaves - 1) / kRowWaves);
}

template <class E>
hipError_t go_gather(TokensArgs a, hipStream_t s) {
  const unsigned n = piece_grid<E, 2>(a);
  return launch(tokens_gather_kernel<E, 2>, dim3(n), kRowWaves * kWave, 0, s, a);
}
template <class E>
hipError_t go_combine(TokensArgs a, hipStream_t s) {
  const unsigned n = piece_grid<E, 1>(a);
  return launch(tokens_combine_kernel<E, 1>, dim3(n), kRowWaves * kWave, 0, s, a);
}
// Choices one after the other leave each wave a trip to memory for each: 8 choices of 2048 wide bf16 rows take, split
// and not, 3.4 and 10.4 us for one token, 7.2 and 14.3 for 512, 24.7 and 23.5 for 2047.
constexpr int64_t kSplitTokens = 2048;
template <class E>
hipError_t go_combine_bwd(TokensArgs a, hipStream_t s) {
  a.pieces = a.T < kSplitTokens ? a.k : 1;
  const dim3 grid(static_cast<unsigned>((a.T * a.pieces + kRowWaves - 1) / kRowWaves));
  constexpr int kOne = kWave * Piece<E>::kN;
  if (a.d <= 4 * kOne) return launch(tokens_combine_bwd_kernel<E, 4, true>, grid, kRowWaves * kWave, 0, s, a);
  return launch(tokens_combine_bwd_kernel<E, 4, false>, grid, kRowWaves * kWave, 0, s, a);
}

}  // namespace

int tokens_sort_blocks(int64_t pairs) {
  if (pairs <= kSortAlone) return 1;
  const int64_t n = (pairs + kSortRun - 1) / kSortRun;
  return static_cast<int>(n < kSortMostBlocks ? n : kSortMostBlocks);
}

hipError_t launch_tokens_sort(TokensSortArgs a, hipStream_t s) {
  const int blocks = tokens_sort_blocks(a.pairs);
  a.run = (a.pairs + blocks - 1) / blocks;
  a.bits = 32 - __builtin_clz(static_cast<unsigned>(a.E));  // of E itself too, which stands for no expert
  const int64_t waves64 = (a.run + kWave - 1) / kWave;
  const int waves = static_cast<int>(waves64 < 1 ? 1 : waves64 < kSortWaves ? waves64 : kSortWaves);
  const size_t lds = static_cast<size_t>(waves + 2) * a.E * 4;
  constexpr size_t kMost = (kSortWaves + 2) * kMoeMaxExperts * 4;
  if (blocks > 1) {
    const hipError_t e = launch_lds<&tokens_count_kernel, kMost>(dim3(blocks), waves * kWave, lds, s, a);
    if (e != hipSuccess) return e;
  }
  return launch_lds<&tokens_place_kernel, kMost>(dim3(blocks), waves * kWave, lds, s, a);
}

hipError_t launch_tokens_gather(const TokensArgs& a, int dtype, hipStream_t s) {
  return dtype == 1 ? go_gather<EBf16>(a, s) : go_gather<EF32>(a, s);
}
hipError_t launch_tokens_combine(const TokensArgs& a, int dtype, hipStream_t s) {
  return dtype == 1 ? go_combine<EBf16>(a, s) : go_combine<EF32>(a, s);
}
hipError_t launch_tokens_combine_bwd(const TokensArgs& a, int dtype, hipStream_t s) {
  return dtype == 1 ? go_combine_bwd<EBf16>(a, s) : go_combine_bwd<EF32>(a, s);
}

}  // namespace twell
