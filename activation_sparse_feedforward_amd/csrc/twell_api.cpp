// C ABI of libtwell: host-side validation and kernel dispatch.  Every check
// happens before any HIP call, so a bad descriptor or pointer costs nothing on
// the device and can be tested without a GPU.
#include <hip/hip_runtime_api.h>

#include <atomic>
#include <cstdint>

#include "../../include/twell.h"
#include "api_internal.hpp"
#include "internal.hpp"

namespace {

constexpr int64_t kIndexLimit = int64_t(1) << 31;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
int elem_bytes(const twell_desc* d) { return d->dtype == TWELL_BF16 ? 2 : 4; }

// Shape checks shared by every entry point.
twell_status check_desc(const twell_desc* d) {
  if (!d) return TWELL_EINVAL;
  if (d->T < 0 || d->d_model <= 0 || d->d_ff <= 0 || d->tile_n <= 0 || d->slots <= 0) return TWELL_EINVAL;
  if (d->dtype != TWELL_FP32 && d->dtype != TWELL_BF16) return TWELL_EINVAL;
  if (d->d_ff % d->tile_n != 0) return TWELL_EINVAL;
  if (d->slots > d->tile_n) return TWELL_EINVAL;
  if (d->tile_n != 64 && d->tile_n != 128) return TWELL_EUNSUPPORTED;
  if (d->dtype == TWELL_BF16) {
    if (d->d_model % 512 != 0 || d->d_model > 4096) return TWELL_EUNSUPPORTED;
  } else {
    if (d->d_model % 256 != 0 || d->d_model > 2048) return TWELL_EUNSUPPORTED;
  }
  const int64_t widest = d->d_ff > d->d_model ? d->d_ff : d->d_model;
  if (d->T > 0 && d->T > (kIndexLimit - 1) / widest) return TWELL_EUNSUPPORTED;
  return TWELL_OK;
}

twell_status check_act(const twell_act& a) {
  if (!a.count || !a.idx || !a.val) return TWELL_EINVAL;
  if (!aligned16(a.count) || !aligned16(a.idx) || !aligned16(a.val)) return TWELL_EINVAL;
  return TWELL_OK;
}

twell_status check_dense_ptr(const void* p) {
  if (!p || !aligned16(p)) return TWELL_EINVAL;
  return TWELL_OK;
}

size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

// Workspace layout of the hybrid forward: router block counts, then the dense
// rows' hidden activations h [max_dense_rows x d_ff].
// Split-K factor of the dense rows' GEMMs that reduce over d_ff.
int dense_splits(const twell_desc* d) { return twell::split_k_for(d->d_ff, 128 / elem_bytes(d)); }

// Heavy ELL rows of the hybrid forward (row total > max(2 C, 2 x mean)): at
// most kHeavyCap of them are cut into heavy_groups() tile ranges each.
constexpr int64_t kHeavyCap = 1024;
int64_t heavy_cap(const twell_desc* d) { return d->T < kHeavyCap ? d->T : kHeavyCap; }
int heavy_groups(const twell_desc* d) {
  const int n_t = d->d_ff / d->tile_n;
  return n_t < 8 ? n_t : 8;
}

// Workspace layout of the hybrid forward: router block counts, the dense rows'
// hidden activations h [max_dense_rows x d_ff], the split-K partials of their
// down GEMM [splits x max_dense_rows x d_model] fp32 (splits > 1 only), then
// the light / heavy split of the ELL rows (row totals, block totals, the two
// lists, their counters) and the heavy rows' partial outputs
// [groups x heavy_cap x d_model] fp32.
struct HybridWs {
  size_t block_dense, h, part, row_total, block_total, block_heavy, light, heavy, split_n, heavy_part, total;
};
HybridWs hybrid_ws(const twell_desc* d, int64_t max_dense_rows) {
  HybridWs w{};
  const size_t T = static_cast<size_t>(d->T);
  const size_t nblk = (T + 255) / 256;
  const size_t cap = static_cast<size_t>(max_dense_rows);
  const int sp = dense_splits(d);
  w.block_dense = 0;
  w.h = align256(nblk * 4);
  w.part = w.h + align256(cap * d->d_ff * elem_bytes(d));
  size_t o = w.part + (sp > 1 ? align256(static_cast<size_t>(sp) * cap * d->d_model * 4) : 0);
  w.row_total = o;   o += align256(T * 4);
  w.block_total = o; o += align256(nblk * 4);
  w.block_heavy = o; o += align256(nblk * 4);
  w.light = o;       o += align256(T * 4);
  w.heavy = o;       o += align256(static_cast<size_t>(heavy_cap(d)) * 4);
  w.split_n = o;     o += 256;
  w.heavy_part = o;  o += align256(static_cast<size_t>(heavy_groups(d)) * heavy_cap(d) * d->d_model * 4);
  w.total = o;
  return w;
}

// Workspace layout of the backward.
struct BwdWs {
  size_t blk_hist, blk_mask, neuron_off, pairs, coef, g_d, u_d, e_d, dg_d, du_d, h_d, dx_part, row_total, block_total, block_heavy,
      light, heavy, split_n, dx_hpart, total;
};
BwdWs bwd_ws(const twell_desc* d, int64_t max_dense_rows) {
  BwdWs w{};
  const size_t T = static_cast<size_t>(d->T), F = static_cast<size_t>(d->d_ff);
  const size_t slots = T * static_cast<size_t>(d->d_ff / d->tile_n) * static_cast<size_t>(d->slots);
  const size_t cap = static_cast<size_t>(max_dense_rows), eb = static_cast<size_t>(elem_bytes(d));
  size_t o = 0;
  w.blk_hist = o;   o += align256(((T + 63) / 64) * F * 4);
  w.blk_mask = o;   o += align256(((T + 63) / 64) * F * 8);
  w.neuron_off = o; o += align256((F + 1) * 4);
  w.pairs = o;      o += align256(slots * 8);
  w.coef = o;       o += align256(slots * 8);
  w.g_d = o;        o += align256(cap * F * 4);
  w.u_d = o;        o += align256(cap * F * 4);
  w.e_d = o;        o += align256(cap * F * 4);
  w.dg_d = o;       o += align256(cap * F * eb);
  w.du_d = o;       o += align256(cap * F * eb);
  w.h_d = o;        o += align256(cap * F * eb);
  const int sp = dense_splits(d);
  w.dx_part = o;    o += sp > 1 ? align256(static_cast<size_t>(sp) * cap * static_cast<size_t>(d->d_model) * 4) : 0;
  w.row_total = o;  o += align256(T * 4);
  w.block_total = o; o += align256(((T + 255) / 256) * 4);
  w.block_heavy = o; o += align256(((T + 255) / 256) * 4);
  w.light = o;      o += align256(T * 4);
  w.heavy = o;      o += align256(static_cast<size_t>(heavy_cap(d)) * 4);
  w.split_n = o;    o += 256;
  w.dx_hpart = o;   o += align256(static_cast<size_t>(heavy_groups(d)) * heavy_cap(d) * d->d_model * 4);
  w.total = o;
  return w;
}

#define TWELL_TRY(expr)                      \
  do {                                       \
    twell_status st_ = (expr);               \
    if (st_ != TWELL_OK) return st_;         \
  } while (0)

twell_status from_hip(hipError_t e) { return e == hipSuccess ? TWELL_OK : TWELL_EHIP; }

// ---------------------------------------------------------------- few-token products
constexpr int32_t kMaxSide = 1 << 20;           // rows, inputs and tokens of the few-token products
constexpr int64_t kMaxMatrix = int64_t(1) << 34;  // rows x inputs of one matrix
constexpr int64_t kMaxStride = int64_t(1) << 40;

bool known_dtype(int32_t t) { return t == TWELL_FP32 || t == TWELL_BF16; }
bool elem_aligned(const void* p, int32_t dtype) {
  return (reinterpret_cast<uintptr_t>(p) & (dtype == TWELL_BF16 ? 1u : 3u)) == 0;
}
int32_t tiles_of(int32_t rows) { return (rows + 15) / 16; }
int32_t blocks_of(int32_t cols) { return (cols + 127) / 128; }

twell_status check_wdesc(const twell_wdesc* d) {
  if (!d || d->experts <= 0 || d->rows <= 0 || d->cols <= 0) return TWELL_EINVAL;
  if (d->bits != 4 && d->bits != 16) return TWELL_EINVAL;
  if (d->bits == 16 ? d->group != 0 : (d->group != 32 && d->group != 64 && d->group != 128)) return TWELL_EINVAL;
  if (d->experts > twell::kMoeMaxExperts || d->rows > kMaxSide || d->cols > kMaxSide) return TWELL_EUNSUPPORTED;
  if (static_cast<int64_t>(d->rows) * d->cols > kMaxMatrix) return TWELL_EUNSUPPORTED;
  return TWELL_OK;
}

twell_status check_planes(const twell_wdesc* d, const twell_wplanes& p) {
  if (!p.codes || !aligned16(p.codes)) return TWELL_EINVAL;
  if (d->bits == 4 && (!p.scales || !aligned16(p.scales))) return TWELL_EINVAL;
  return TWELL_OK;
}

twell::WeightsArgs weights_args(const twell_wdesc* d, const twell_wplanes& p) {
  twell::WeightsArgs a{};
  a.codes = static_cast<uint8_t*>(p.codes);
  a.scales = static_cast<uint16_t*>(p.scales);
  a.experts = d->experts;
  a.N = d->rows;
  a.K = d->cols;
  a.bits = d->bits;
  a.group = d->group;
  a.tiles = tiles_of(d->rows);
  a.blocks = blocks_of(d->cols);
  return a;
}

twell_wdesc moe_in_desc(const twell_moe_desc* d) { return {d->experts, d->d_ff, d->d_model, d->bits, d->group}; }
twell_wdesc moe_out_desc(const twell_moe_desc* d) { return {d->experts, d->d_model, d->d_ff, d->bits, d->group}; }

twell_status check_moe(const twell_moe_desc* d) {
  if (!d || d->T < 0 || d->top_k <= 0 || d->top_k > d->experts) return TWELL_EINVAL;
  if (!known_dtype(d->dtype)) return TWELL_EINVAL;
  if (d->act != TWELL_RELU && d->act != TWELL_SILU) return TWELL_EINVAL;
  if (d->renorm != 0 && d->renorm != 1) return TWELL_EINVAL;
  const twell_wdesc in = moe_in_desc(d);
  TWELL_TRY(check_wdesc(&in));
  if (d->ldx < d->d_model || d->ldy < d->d_model) return TWELL_EINVAL;
  if (d->top_k > twell::kMoeMaxTopK || d->T > kMaxSide || d->ldx > kMaxStride || d->ldy > kMaxStride)
    return TWELL_EUNSUPPORTED;
  return TWELL_OK;
}

// Workspace of the mixture of experts: the hidden values of one block of
// tokens' (token, choice) pairs, the pairs' outputs, the choices that count, and
// the chosen experts with their pairs.
struct MoeWs {
  size_t h, z, logits, live, chosen, chosen_pairs, total;
  int64_t h_plane, h_row;
  int32_t block_tokens;
};
MoeWs moe_ws(const twell_moe_desc* d) {
  MoeWs w{};
  w.block_tokens = static_cast<int32_t>(d->T < twell::kMoeBlockTokens ? d->T : twell::kMoeBlockTokens);
  const int64_t pairs = static_cast<int64_t>(w.block_tokens) * d->top_k;
  w.h_row = static_cast<int64_t>(blocks_of(d->d_ff)) * 128;
  w.h_plane = pairs * w.h_row;
  size_t o = 0;
  w.h = o;        o += align256(static_cast<size_t>(w.h_plane) * 2 * (d->dtype == TWELL_BF16 ? 2 : 3));
  w.z = o;        o += align256(static_cast<size_t>(pairs) * static_cast<size_t>(d->d_model) * 4);
  const size_t few = static_cast<size_t>(w.block_tokens < 4 ? w.block_tokens : 4);
  w.logits = o;   o += align256(few * static_cast<size_t>(d->experts) * 4);
  w.live = o;     o += align256(static_cast<size_t>(pairs) * 4);
  const size_t chosen = static_cast<size_t>(pairs < d->experts ? pairs : d->experts);
  w.chosen = o;       o += align256(chosen * sizeof(twell::MoeChosen));
  w.chosen_pairs = o; o += align256(chosen * twell::kMoeBlockTokens * 4);
  w.total = o;
  return w;
}

// ---------------------------------------------------------------- a layer over many tokens
twell_status check_elems(const void* p, int32_t dtype) { return p && elem_aligned(p, dtype) ? TWELL_OK : TWELL_EINVAL; }

constexpr int64_t kMaxElems = int64_t(1) << 33;  // tokens x width: what the grids of one launch reach

twell_status check_tokens(const twell_tokens_desc* d) {
  if (!d || d->T < 0 || d->d_model <= 0 || d->experts <= 0 || d->top_k <= 0) return TWELL_EINVAL;
  if (!known_dtype(d->dtype) || d->ld_tokens < d->d_model || d->ld_rows < d->d_model) return TWELL_EINVAL;
  if (d->T > kMaxSide || d->d_model > kMaxSide || d->T * d->d_model > kMaxElems) return TWELL_EUNSUPPORTED;
  if (d->experts > twell::kMoeMaxExperts || d->top_k > twell::kMoeMaxTopK) return TWELL_EUNSUPPORTED;
  if (d->ld_tokens > kMaxStride || d->ld_rows > kMaxStride) return TWELL_EUNSUPPORTED;
  return TWELL_OK;
}
// Counts of each workgroup of the sort.
size_t tokens_ws(const twell_tokens_desc* d) {
  return align256(static_cast<size_t>(twell::tokens_sort_blocks(d->T * d->top_k)) * d->experts * 4);
}
twell::TokensArgs tokens_args(const twell_tokens_desc* d, const int32_t* pair_row) {
  twell::TokensArgs a{};
  a.pair_row = pair_row;
  a.T = d->T;
  a.pairs = d->T * d->top_k;
  a.ld_tokens = d->ld_tokens;
  a.ld_rows = d->ld_rows;
  a.d = d->d_model;
  a.k = d->top_k;
  return a;
}

twell_status check_norm(const twell_norm_desc* d) {
  if (!d || d->T < 0 || d->d_model <= 0 || !known_dtype(d->dtype) || !known_dtype(d->w_dtype)) return TWELL_EINVAL;
  if (!(d->eps >= 0.f) || d->eps > 3.4e38f) return TWELL_EINVAL;
  if (d->ldx < d->d_model || d->ldy < d->d_model || d->lddx < d->d_model) return TWELL_EINVAL;
  if (d->T > kMaxSide || d->d_model > twell::kNormMostWidth) return TWELL_EUNSUPPORTED;
  if (d->ldx > kMaxStride || d->ldy > kMaxStride || d->lddx > kMaxStride) return TWELL_EUNSUPPORTED;
  return TWELL_OK;
}
// Each workgroup's sums of dw and db.
size_t norm_ws(const twell_norm_desc* d) {
  return align256(static_cast<size_t>(twell::norm_blocks(d->T, d->d_model, d->dtype)) * 2 * d->d_model * 4);
}
twell::NormArgs norm_args(const twell_norm_desc* d) {
  twell::NormArgs a{};
  a.T = d->T;
  a.ldx = d->ldx;
  a.ldy = d->ldy;
  a.lddx = d->lddx;
  a.d = d->d_model;
  a.blocks = twell::norm_blocks(d->T, d->d_model, d->dtype);
  a.eps = d->eps;
  return a;
}

twell_status check_fp8(const twell_fp8_desc* d) {
  if (!d || d->experts <= 0 || d->rows <= 0 || d->cols <= 0) return TWELL_EINVAL;
  if (d->experts > twell::kMoeMaxExperts || d->rows > kMaxSide || d->cols > kMaxSide) return TWELL_EUNSUPPORTED;
  if (static_cast<int64_t>(d->rows) * d->cols > kMaxMatrix) return TWELL_EUNSUPPORTED;
  return TWELL_OK;
}
twell_status check_fp8_planes(const twell_wplanes& p) {
  return p.codes && p.scales && aligned16(p.codes) && aligned16(p.scales) ? TWELL_OK : TWELL_EINVAL;
}
int32_t quads_of(int32_t blocks) { return (blocks + 3) / 4; }
twell_fp8_desc transposed(const twell_fp8_desc* d) { return {d->experts, d->cols, d->rows}; }

twell::F8PackArgs fp8_pack_args(const twell_fp8_desc* d, const twell_wplanes& p) {
  twell::F8PackArgs a{};
  a.codes = static_cast<uint8_t*>(p.codes);
  a.scales = static_cast<uint8_t*>(p.scales);
  a.experts = d->experts;
  a.N = d->rows;
  a.K = d->cols;
  a.tiles = tiles_of(d->rows);
  a.blocks = blocks_of(d->cols);
  a.quads = quads_of(a.blocks);
  a.tiles_t = tiles_of(d->cols);
  a.blocks_t = blocks_of(d->rows);
  a.quads_t = quads_of(a.blocks_t);
  return a;
}

// What a call with T rows asks of T, offsets and the rows' tensors.
constexpr int64_t kMaxProduct = int64_t(1) << 37;  // rows x width of a result: what the grid of one launch reaches
twell_status check_fp8_rows(const twell_fp8_desc* d, int64_t T, const int32_t* offsets, int32_t dtype) {
  TWELL_TRY(check_fp8(d));
  if (T < 0 || !known_dtype(dtype) || !aligned4(offsets) || (!offsets && d->experts != 1)) return TWELL_EINVAL;
  if (T > kMaxSide || T * d->rows > kMaxProduct || T * d->cols > kMaxProduct) return TWELL_EUNSUPPORTED;
  return TWELL_OK;
}
twell_status check_stride(int64_t ld, int64_t width) {
  return ld < width ? TWELL_EINVAL : ld > kMaxStride ? TWELL_EUNSUPPORTED : TWELL_OK;
}

// Workspace of a product: the codes and scales of T rows of `cols` inputs, whose
// tiles of 16 begin anew for each expert.
struct Fp8Ws {
  int64_t most_tiles;
  size_t codes, scales, total;
};
Fp8Ws fp8_ws(const twell_fp8_desc* d, int64_t T) {
  Fp8Ws w{};
  const size_t blocks = static_cast<size_t>(blocks_of(d->cols));
  w.most_tiles = T / 16 + d->experts;
  w.codes = 0;
  w.scales = static_cast<size_t>(w.most_tiles) * blocks * 2048;
  w.total = align256(w.scales + static_cast<size_t>(w.most_tiles) * ((blocks + 3) / 4) * 64);
  return w;
}

// Of the gradients: dx's product, and before it dw's parts in the same place.
size_t fp8_bwd_ws(const twell_fp8_desc* d, int64_t T) {
  const twell_fp8_desc t = transposed(d);
  const int parts = twell::wgrad_parts(T, d->rows, d->cols, d->experts);
  const size_t dx = fp8_ws(&t, T).total;
  const size_t dw = parts == 1 ? 0
                               : static_cast<size_t>(parts) * static_cast<size_t>(d->experts) *
                                     static_cast<size_t>(d->rows) * static_cast<size_t>(d->cols) * 4;
  return dx > dw ? dx : align256(dw);
}

// y = Q(x) W^T, arguments checked.
twell_status fp8_product(const twell_fp8_desc* d, const twell_wplanes& p, int64_t T, const int32_t* offsets,
                         int32_t dtype, const void* x, int64_t ldx, void* y, int64_t ldy, void* ws, hipStream_t s) {
  const Fp8Ws w = fp8_ws(d, T);
  const int32_t blocks = blocks_of(d->cols);
  uint8_t* wsb = static_cast<uint8_t*>(ws);
  twell::F8RowsArgs r{};
  r.x = x;
  r.codes = wsb + w.codes;
  r.scales = wsb + w.scales;
  r.offsets = offsets;
  r.T = T;
  r.ldx = ldx;
  r.most_tiles = w.most_tiles;
  r.K = d->cols;
  r.blocks = blocks;
  r.quads = quads_of(blocks);
  r.experts = d->experts;
  twell::F8GemmArgs g{};
  g.w_codes = static_cast<const uint8_t*>(p.codes);
  g.w_scales = static_cast<const uint8_t*>(p.scales);
  g.x_codes = r.codes;
  g.x_scales = r.scales;
  g.x = x;
  g.ldx = ldx;
  g.K = d->cols;
  g.y = y;
  g.offsets = offsets;
  g.T = T;
  g.ldy = ldy;
  g.most_tiles = w.most_tiles;
  g.N = d->rows;
  g.tiles = tiles_of(d->rows);
  g.blocks = blocks;
  g.quads = r.quads;
  g.experts = d->experts;
  return from_hip(twell::launch_f8_product(g, r, dtype, s));
}

}  // namespace

namespace twell {

// Workgroups of the lockstep kernels the device runs at once: one per CU
// (their LDS or VGPR footprint).  0 when the device cannot be queried: the
// launchers then issue the whole grid in one dispatch.
int lockstep_resident() {
  static std::atomic<int> cached[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return 0;
  if (dev < 64) {
    const int v = cached[dev].load(std::memory_order_relaxed);
    if (v > 0) return v;
  }
  int n = 0;
  if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0) return 0;
  if (dev < 64) cached[dev].store(n, std::memory_order_relaxed);
  return n;
}

}  // namespace twell

namespace twell {

twell_status hybrid_check(const twell_desc* d, const void* x, const void* w_gate_t, twell_act act,
                          const void* w_up_t, const void* w_down, void* y, const twell_route* route,
                          size_t* ws_need) {
  TWELL_TRY(check_desc(d));
  if (!route || route->max_dense_rows < 0 || !ws_need) return TWELL_EINVAL;
  *ws_need = 0;
  if (d->T == 0) return TWELL_OK;
  TWELL_TRY(check_dense_ptr(x));
  TWELL_TRY(check_dense_ptr(w_gate_t));
  TWELL_TRY(check_act(act));
  TWELL_TRY(check_dense_ptr(w_up_t));
  TWELL_TRY(check_dense_ptr(w_down));
  TWELL_TRY(check_dense_ptr(y));
  if (!route->ell_rows || !route->n_rows || !route->row_kind) return TWELL_EINVAL;
  if (route->max_dense_rows > 0 && !route->dense_rows) return TWELL_EINVAL;
  if (!aligned4(route->ell_rows) || !aligned4(route->n_rows) ||
      (route->dense_rows && !aligned4(route->dense_rows)))
    return TWELL_EINVAL;
  *ws_need = hybrid_ws(d, route->max_dense_rows).total;
  return TWELL_OK;
}

twell_status hybrid_launch(const twell_desc* d, const void* x, const void* w_gate_t, twell_act act,
                           const void* w_up_t, const void* w_down, void* y, const twell_route* route,
                           void* ws, void* stream) {
  const HybridWs hw = hybrid_ws(d, route->max_dense_rows);
  hipStream_t s = static_cast<hipStream_t>(stream);
  char* wsb = static_cast<char*>(ws);

  twell::RouteArgs r{};
  r.count = act.count;
  r.T = d->T;
  r.n_t = d->d_ff / d->tile_n;
  r.C = d->slots;
  r.cap = route->max_dense_rows;
  r.flags = route->row_kind;
  r.block_dense = reinterpret_cast<int32_t*>(wsb + hw.block_dense);
  r.ell_rows = route->ell_rows;
  r.dense_rows = route->dense_rows;
  r.n_rows = route->n_rows;
  r.row_total = reinterpret_cast<int32_t*>(wsb + hw.row_total);
  r.block_total = reinterpret_cast<int32_t*>(wsb + hw.block_total);
  r.light_rows = reinterpret_cast<int32_t*>(wsb + hw.light);
  r.heavy_rows = reinterpret_cast<int32_t*>(wsb + hw.heavy);
  r.split_n = reinterpret_cast<int32_t*>(wsb + hw.split_n);
  r.block_heavy = reinterpret_cast<int32_t*>(wsb + hw.block_heavy);
  r.heavy_cap = heavy_cap(d);
  TWELL_TRY(from_hip(twell::launch_route(r, s)));
  TWELL_TRY(from_hip(twell::launch_route_split(r, s)));

  twell::FusedArgs f{};
  f.x = x;
  f.count = act.count;
  f.idx = act.idx;
  f.val = act.val;
  f.w_up_t = w_up_t;
  f.w_down = w_down;
  f.y = y;
  f.rows = r.light_rows;
  f.n_rows_dev = r.split_n + 0;
  f.row_total = r.row_total;  // written by the route pass above
  f.T = d->T;
  f.d = d->d_model;
  f.F = d->d_ff;
  f.tile_n = d->tile_n;
  f.C = d->slots;
  TWELL_TRY(from_hip(twell::launch_fused_updown(f, d->dtype, s)));
  twell::FusedArgs fh = f;  // heavy ELL rows, cut into tile ranges
  fh.rows = r.heavy_rows;
  fh.n_rows_dev = r.split_n + 1;
  fh.groups = heavy_groups(d);
  fh.part = reinterpret_cast<float*>(wsb + hw.heavy_part);
  fh.part_rows = r.heavy_cap;
  TWELL_TRY(from_hip(twell::launch_fused_split(fh, d->dtype, s)));

  if (route->max_dense_rows == 0) return TWELL_OK;
  twell::GateUpArgs g{};
  g.x = x;
  g.w_gate_t = w_gate_t;
  g.w_up_t = w_up_t;
  g.h = wsb + hw.h;
  g.rows = route->dense_rows;
  g.n_rows_dev = route->n_rows + 1;
  g.M = route->max_dense_rows;
  g.d = d->d_model;
  g.F = d->d_ff;
  TWELL_TRY(from_hip(twell::launch_gateup(g, d->dtype, s)));
  twell::DownArgs dn{};
  dn.h = wsb + hw.h;
  dn.w_down = w_down;
  dn.y = y;
  dn.rows = route->dense_rows;
  dn.n_rows_dev = route->n_rows + 1;
  dn.M = route->max_dense_rows;
  dn.d = d->d_model;
  dn.F = d->d_ff;
  dn.splits = dense_splits(d);
  dn.part = reinterpret_cast<float*>(wsb + hw.part);
  return from_hip(twell::launch_down(dn, d->dtype, s));
}


}  // namespace twell

extern "C" {

twell_status twell_sizes(const twell_desc* d, int64_t max_dense_rows, twell_sizes_t* out) {
  TWELL_TRY(check_desc(d));
  if (!out || max_dense_rows < 0) return TWELL_EINVAL;
  const size_t T = static_cast<size_t>(d->T);
  const size_t n_t = static_cast<size_t>(d->d_ff / d->tile_n);
  const size_t C = static_cast<size_t>(d->slots);
  const size_t eb = static_cast<size_t>(elem_bytes(d));
  out->count = T * n_t * 4;
  out->idx = T * n_t * C;
  out->val = T * n_t * C * eb;
  out->ws_dense_fwd = align256(T * static_cast<size_t>(d->d_ff) * eb) +
                      static_cast<size_t>(d->d_model) * static_cast<size_t>(d->d_ff) * eb;
  const HybridWs hw = hybrid_ws(d, max_dense_rows);
  out->ws_hybrid = hw.total;
  out->ws_bwd = bwd_ws(d, max_dense_rows).total;
  out->ws_pack_classic = T * static_cast<size_t>(d->d_ff) * eb;
  return TWELL_OK;
}

twell_status twell_pack(const twell_desc* d, const void* x, const void* w_gate_t, twell_act act,
                        int64_t* stats, void* gate_dbg, void* stream) {
  TWELL_TRY(check_desc(d));
  if (d->T == 0) return TWELL_OK;
  TWELL_TRY(check_dense_ptr(x));
  TWELL_TRY(check_dense_ptr(w_gate_t));
  TWELL_TRY(check_act(act));
  if (stats && (reinterpret_cast<uintptr_t>(stats) & 7u)) return TWELL_EINVAL;
  if (gate_dbg && !aligned4(gate_dbg)) return TWELL_EINVAL;
  twell::PackArgs a{};
  a.x = x;
  a.w_gate_t = w_gate_t;
  a.T = d->T;
  a.d = d->d_model;
  a.F = d->d_ff;
  a.tile_n = d->tile_n;
  a.C = d->slots;
  a.count = act.count;
  a.idx = act.idx;
  a.val = act.val;
  a.stats = reinterpret_cast<unsigned long long*>(stats);
  a.gate_dbg = gate_dbg;
  return from_hip(twell::launch_gate_pack(a, d->dtype, static_cast<hipStream_t>(stream)));
}

twell_status twell_ffn_fwd(const twell_desc* d, const void* x, twell_act act, const void* w_up_t,
                           const void* w_down, void* y, void* stream) {
  TWELL_TRY(check_desc(d));
  if (d->T == 0) return TWELL_OK;
  TWELL_TRY(check_dense_ptr(x));
  TWELL_TRY(check_act(act));
  TWELL_TRY(check_dense_ptr(w_up_t));
  TWELL_TRY(check_dense_ptr(w_down));
  TWELL_TRY(check_dense_ptr(y));
  twell::FusedArgs a{};
  a.rows = nullptr;
  a.n_rows_dev = nullptr;
  a.x = x;
  a.count = act.count;
  a.idx = act.idx;
  a.val = act.val;
  a.w_up_t = w_up_t;
  a.w_down = w_down;
  a.y = y;
  a.T = d->T;
  a.d = d->d_model;
  a.F = d->d_ff;
  a.tile_n = d->tile_n;
  a.C = d->slots;
  return from_hip(twell::launch_fused_updown(a, d->dtype, static_cast<hipStream_t>(stream)));
}

twell_status twell_ffn_fwd_hybrid(const twell_desc* d, const void* x, const void* w_gate_t, twell_act act,
                                  const void* w_up_t, const void* w_down, void* y, const twell_route* route,
                                  void* ws, size_t ws_bytes, void* stream) {
  size_t need = 0;
  TWELL_TRY(twell::hybrid_check(d, x, w_gate_t, act, w_up_t, w_down, y, route, &need));
  if (d->T == 0) return TWELL_OK;
  if (!ws || !aligned16(ws) || ws_bytes < need) return TWELL_EINVAL;
  return twell::hybrid_launch(d, x, w_gate_t, act, w_up_t, w_down, y, route, ws, stream);
}

twell_status twell_ffn_bwd(const twell_desc* d, const void* x, twell_act act, const twell_route* route,
                           const void* w_gate_t, const void* w_up_t, const void* w_down, const void* dy,
                           float l1_coef, void* dx, float* dw_gate_t, float* dw_up_t, float* dw_down,
                           void* ws, size_t ws_bytes, void* stream) {
  TWELL_TRY(check_desc(d));
  if (!route || route->max_dense_rows < 0) return TWELL_EINVAL;
  TWELL_TRY(check_dense_ptr(w_gate_t));
  TWELL_TRY(check_dense_ptr(w_up_t));
  TWELL_TRY(check_dense_ptr(w_down));
  TWELL_TRY(check_dense_ptr(dw_gate_t));
  TWELL_TRY(check_dense_ptr(dw_up_t));
  TWELL_TRY(check_dense_ptr(dw_down));
  const BwdWs bw = bwd_ws(d, route->max_dense_rows);
  if (!ws || !aligned16(ws) || ws_bytes < bw.total) return TWELL_EINVAL;
  if (d->T > 0) {
    TWELL_TRY(check_dense_ptr(x));
    TWELL_TRY(check_dense_ptr(dy));
    TWELL_TRY(check_dense_ptr(dx));
    TWELL_TRY(check_act(act));
    if (!route->ell_rows || !route->n_rows) return TWELL_EINVAL;
    if (route->max_dense_rows > 0 && !route->dense_rows) return TWELL_EINVAL;
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  char* wsb = static_cast<char*>(ws);
  twell::BwdArgs a{};
  a.x = x;
  a.dy = dy;
  a.count = act.count;
  a.idx = act.idx;
  a.val = act.val;
  a.w_gate_t = w_gate_t;
  a.w_up_t = w_up_t;
  a.w_down = w_down;
  a.ell_rows = route->ell_rows;
  a.dense_rows = route->dense_rows;
  a.n_rows = route->n_rows;
  a.T = d->T;
  a.cap = d->T > 0 ? route->max_dense_rows : 0;
  a.d = d->d_model;
  a.F = d->d_ff;
  a.tile_n = d->tile_n;
  a.C = d->slots;
  a.l1 = l1_coef;
  a.dx = dx;
  a.dw_gate_t = dw_gate_t;
  a.dw_up_t = dw_up_t;
  a.dw_down = dw_down;
  a.blk_hist = reinterpret_cast<int32_t*>(wsb + bw.blk_hist);
  a.blk_mask = reinterpret_cast<unsigned long long*>(wsb + bw.blk_mask);
  a.neuron_off = reinterpret_cast<int32_t*>(wsb + bw.neuron_off);
  a.pairs = reinterpret_cast<int2*>(wsb + bw.pairs);
  a.coef = reinterpret_cast<float2*>(wsb + bw.coef);
  a.g_d = reinterpret_cast<float*>(wsb + bw.g_d);
  a.u_d = reinterpret_cast<float*>(wsb + bw.u_d);
  a.e_d = reinterpret_cast<float*>(wsb + bw.e_d);
  a.dg_d = wsb + bw.dg_d;
  a.du_d = wsb + bw.du_d;
  a.h_d = wsb + bw.h_d;
  a.dx_splits = dense_splits(d);
  a.dx_part = reinterpret_cast<float*>(wsb + bw.dx_part);
  a.row_total = reinterpret_cast<int32_t*>(wsb + bw.row_total);
  a.block_total = reinterpret_cast<int32_t*>(wsb + bw.block_total);
  a.light_rows = reinterpret_cast<int32_t*>(wsb + bw.light);
  a.heavy_rows = reinterpret_cast<int32_t*>(wsb + bw.heavy);
  a.split_n = reinterpret_cast<int32_t*>(wsb + bw.split_n);
  a.block_heavy = reinterpret_cast<int32_t*>(wsb + bw.block_heavy);
  a.heavy_cap = heavy_cap(d);
  a.groups = heavy_groups(d);
  a.dx_hpart = reinterpret_cast<float*>(wsb + bw.dx_hpart);
  // dense rows first: their weight-gradient GEMM stores its part of dW, which
  // the ELL rows' per-neuron pass reads and adds to its own sums before its one
  // write of each row (instead of a separate read-modify-write pass over dW)
  TWELL_TRY(from_hip(twell::launch_bwd_dense(a, d->dtype, s)));
  return from_hip(twell::launch_bwd_sparse(a, d->dtype, s));
}

twell_status twell_pack_classic(const twell_desc* d, const void* x, const void* w_gate_t, twell_act act,
                                void* ws, size_t ws_bytes, void* stream) {
  TWELL_TRY(check_desc(d));
  if (d->T == 0) return TWELL_OK;
  TWELL_TRY(check_dense_ptr(x));
  TWELL_TRY(check_dense_ptr(w_gate_t));
  TWELL_TRY(check_act(act));
  TWELL_TRY(check_dense_ptr(ws));
  twell_sizes_t sz;
  TWELL_TRY(twell_sizes(d, 0, &sz));
  if (ws_bytes < sz.ws_pack_classic) return TWELL_EINVAL;
  twell::ClassicArgs a{};
  a.x = x;
  a.w_gate_t = w_gate_t;
  a.dense = ws;
  a.T = d->T;
  a.d = d->d_model;
  a.F = d->d_ff;
  a.tile_n = d->tile_n;
  a.C = d->slots;
  a.count = act.count;
  a.idx = act.idx;
  a.val = act.val;
  return from_hip(twell::launch_classic_pack(a, d->dtype, static_cast<hipStream_t>(stream)));
}

twell_status twell_dense_ffn_fwd(const twell_desc* d, const void* x, const void* w_gate_t,
                                 const void* w_up_t, const void* w_down, void* y, void* ws,
                                 size_t ws_bytes, void* stream) {
  TWELL_TRY(check_desc(d));
  if (d->T == 0) return TWELL_OK;
  TWELL_TRY(check_dense_ptr(x));
  TWELL_TRY(check_dense_ptr(w_gate_t));
  TWELL_TRY(check_dense_ptr(w_up_t));
  TWELL_TRY(check_dense_ptr(w_down));
  TWELL_TRY(check_dense_ptr(y));
  TWELL_TRY(check_dense_ptr(ws));
  twell_sizes_t sz;
  TWELL_TRY(twell_sizes(d, 0, &sz));
  if (ws_bytes < sz.ws_dense_fwd) return TWELL_EINVAL;
  hipStream_t s = static_cast<hipStream_t>(stream);
  twell::GateUpArgs g{};
  g.x = x;
  g.w_gate_t = w_gate_t;
  g.w_up_t = w_up_t;
  g.h = ws;
  g.rows = nullptr;
  g.n_rows_dev = nullptr;
  g.M = d->T;
  g.d = d->d_model;
  g.F = d->d_ff;
  twell::DownArgs dn{};
  dn.h = ws;
  dn.w_down = w_down;
  dn.w_down_t = static_cast<char*>(ws) + align256(static_cast<size_t>(d->T) * d->d_ff * elem_bytes(d));
  dn.y = y;
  dn.rows = nullptr;
  dn.n_rows_dev = nullptr;
  dn.M = d->T;
  dn.d = d->d_model;
  dn.F = d->d_ff;
  return from_hip(twell::launch_dense256(g, dn, d->dtype, s));
}

twell_status twell_weights_sizes(const twell_wdesc* d, twell_wsizes_t* out) {
  TWELL_TRY(check_wdesc(d));
  if (!out) return TWELL_EINVAL;
  const size_t blocks = static_cast<size_t>(d->experts) * static_cast<size_t>(tiles_of(d->rows)) *
                        static_cast<size_t>(blocks_of(d->cols));
  out->codes = blocks * (d->bits == 4 ? 1024 : 4096);
  out->scales = d->bits == 4 ? blocks * 16 * static_cast<size_t>(128 / d->group) * 2 : 0;
  return TWELL_OK;
}

twell_status twell_weights_pack(const twell_wdesc* d, const void* w, int32_t w_dtype, int32_t transposed,
                                twell_wplanes out, void* stream) {
  TWELL_TRY(check_wdesc(d));
  if (!known_dtype(w_dtype) || (transposed != 0 && transposed != 1)) return TWELL_EINVAL;
  if (d->bits == 16 && w_dtype != TWELL_BF16) return TWELL_EUNSUPPORTED;  // would round
  if (!w || !elem_aligned(w, w_dtype)) return TWELL_EINVAL;
  TWELL_TRY(check_planes(d, out));
  twell::WeightsArgs a = weights_args(d, out);
  a.w = w;
  return from_hip(twell::launch_weights_pack(a, w_dtype, transposed != 0, static_cast<hipStream_t>(stream)));
}

twell_status twell_weights_unpack(const twell_wdesc* d, twell_wplanes in, void* w, int32_t w_dtype, void* stream) {
  TWELL_TRY(check_wdesc(d));
  if (!known_dtype(w_dtype)) return TWELL_EINVAL;
  if (d->bits == 16 && w_dtype != TWELL_BF16) return TWELL_EUNSUPPORTED;
  if (!w || !elem_aligned(w, w_dtype)) return TWELL_EINVAL;
  TWELL_TRY(check_planes(d, in));
  twell::WeightsArgs a = weights_args(d, in);
  a.out = w;
  return from_hip(twell::launch_weights_unpack(a, w_dtype, static_cast<hipStream_t>(stream)));
}

twell_status twell_linear_fwd(const twell_wdesc* d, twell_wplanes w, int64_t T, int32_t dtype, const void* x,
                              int64_t ldx, void* y, int64_t ldy, void* stream) {
  TWELL_TRY(check_wdesc(d));
  if (T < 0 || !known_dtype(dtype) || ldx < d->cols || ldy < d->rows) return TWELL_EINVAL;
  if (d->experts != 1 || d->bits != 4 || T > kMaxSide || ldx > kMaxStride || ldy > kMaxStride)
    return TWELL_EUNSUPPORTED;
  if (T == 0) return TWELL_OK;
  if (!x || !y || !elem_aligned(x, dtype) || !elem_aligned(y, dtype)) return TWELL_EINVAL;
  TWELL_TRY(check_planes(d, w));
  twell::LinearArgs a{};
  a.x = x;
  a.y = y;
  a.codes = static_cast<const uint8_t*>(w.codes);
  a.scales = static_cast<const uint16_t*>(w.scales);
  a.T = T;
  a.ldx = ldx;
  a.ldy = ldy;
  a.N = d->rows;
  a.K = d->cols;
  a.group = d->group;
  a.tiles = tiles_of(d->rows);
  a.blocks = blocks_of(d->cols);
  return from_hip(twell::launch_linear4(a, dtype, static_cast<hipStream_t>(stream)));
}

twell_status twell_moe_sizes(const twell_moe_desc* d, size_t* ws) {
  TWELL_TRY(check_moe(d));
  if (!ws) return TWELL_EINVAL;
  *ws = moe_ws(d).total;
  return TWELL_OK;
}

twell_status twell_moe_fwd(const twell_moe_desc* d, const void* x, const void* w_router, const float* router_bias,
                           twell_wplanes gate, twell_wplanes up, twell_wplanes down, void* y, int32_t* ids,
                           float* weights, void* ws, size_t ws_bytes, void* stream) {
  TWELL_TRY(check_moe(d));
  if (d->T == 0) return TWELL_OK;
  if (!x || !w_router || !y || !ids || !weights) return TWELL_EINVAL;
  if (!elem_aligned(x, d->dtype) || !elem_aligned(w_router, d->dtype) || !elem_aligned(y, d->dtype))
    return TWELL_EINVAL;
  if (!aligned4(ids) || !aligned4(weights) || (router_bias && !aligned4(router_bias))) return TWELL_EINVAL;
  const twell_wdesc in = moe_in_desc(d);
  TWELL_TRY(check_planes(&in, gate));
  TWELL_TRY(check_planes(&in, up));
  TWELL_TRY(check_planes(&in, down));
  const MoeWs w = moe_ws(d);
  if (!ws || !aligned16(ws) || ws_bytes < w.total) return TWELL_EINVAL;

  hipStream_t s = static_cast<hipStream_t>(stream);
  char* wsb = static_cast<char*>(ws);
  twell::MoeArgs a{};
  a.x = x;
  a.y = y;
  a.router = w_router;
  a.bias = router_bias;
  a.ids = ids;
  a.weights = weights;
  a.gate_codes = static_cast<const uint8_t*>(gate.codes);
  a.up_codes = static_cast<const uint8_t*>(up.codes);
  a.down_codes = static_cast<const uint8_t*>(down.codes);
  a.gate_scales = static_cast<const uint16_t*>(gate.scales);
  a.up_scales = static_cast<const uint16_t*>(up.scales);
  a.down_scales = static_cast<const uint16_t*>(down.scales);
  a.ldx = d->ldx;
  a.ldy = d->ldy;
  a.E = d->experts;
  a.k = d->top_k;
  a.inv_k = 1.0f / static_cast<float>(d->top_k);
  a.d = d->d_model;
  a.f = d->d_ff;
  a.bits = d->bits;
  a.group = d->group;
  a.act = d->act;
  a.renorm = d->renorm;
  a.tiles_f = tiles_of(d->d_ff);
  a.blocks_d = blocks_of(d->d_model);
  a.tiles_d = tiles_of(d->d_model);
  a.blocks_f = blocks_of(d->d_ff);
  a.h = reinterpret_cast<uint16_t*>(wsb + w.h);
  a.h_plane = w.h_plane;
  a.h_row = w.h_row;
  a.z = reinterpret_cast<float*>(wsb + w.z);
  a.logits = reinterpret_cast<float*>(wsb + w.logits);
  a.live = reinterpret_cast<int32_t*>(wsb + w.live);
  a.chosen = reinterpret_cast<twell::MoeChosen*>(wsb + w.chosen);
  a.chosen_pairs = reinterpret_cast<int32_t*>(wsb + w.chosen_pairs);
  const int64_t eb = d->dtype == TWELL_BF16 ? 2 : 4;
  for (int64_t t0 = 0; t0 < d->T; t0 += w.block_tokens) {
    a.T = static_cast<int32_t>(d->T - t0 < w.block_tokens ? d->T - t0 : w.block_tokens);
    a.x = static_cast<const char*>(x) + t0 * d->ldx * eb;
    a.y = static_cast<char*>(y) + t0 * d->ldy * eb;
    a.ids = ids + t0 * d->top_k;
    a.weights = weights + t0 * d->top_k;
    const int64_t pairs = static_cast<int64_t>(a.T) * d->top_k;
    a.most_chosen = static_cast<int32_t>(pairs < d->experts ? pairs : d->experts);
    a.by_expert = pairs >= d->experts;
    TWELL_TRY(from_hip(twell::launch_moe(a, d->dtype, s)));
  }
  return TWELL_OK;
}

twell_status twell_tokens_sizes(const twell_tokens_desc* d, size_t* ws) {
  TWELL_TRY(check_tokens(d));
  if (!ws) return TWELL_EINVAL;
  *ws = tokens_ws(d);
  return TWELL_OK;
}

twell_status twell_tokens_sort(const twell_tokens_desc* d, const int32_t* ids, int32_t* offsets, int32_t* pair_row,
                               void* ws, size_t ws_bytes, void* stream) {
  TWELL_TRY(check_tokens(d));
  if (!offsets || !aligned4(offsets)) return TWELL_EINVAL;
  if (d->T > 0 && (!ids || !pair_row || !aligned4(ids) || !aligned4(pair_row))) return TWELL_EINVAL;
  if (!ws || !aligned16(ws) || ws_bytes < tokens_ws(d)) return TWELL_EINVAL;
  twell::TokensSortArgs a{};
  a.ids = ids;
  a.offsets = offsets;
  a.pair_row = pair_row;
  a.hist = static_cast<int32_t*>(ws);
  a.pairs = d->T * d->top_k;
  a.E = d->experts;
  return from_hip(twell::launch_tokens_sort(a, static_cast<hipStream_t>(stream)));
}

twell_status twell_tokens_gather(const twell_tokens_desc* d, const void* x, const int32_t* pair_row, void* rows,
                                 void* stream) {
  TWELL_TRY(check_tokens(d));
  if (d->T == 0) return TWELL_OK;
  TWELL_TRY(check_elems(x, d->dtype));
  TWELL_TRY(check_elems(rows, d->dtype));
  if (!pair_row || !aligned4(pair_row)) return TWELL_EINVAL;
  twell::TokensArgs a = tokens_args(d, pair_row);
  a.x = x;
  a.rows_out = rows;
  a.ld_out = d->ld_rows;
  return from_hip(twell::launch_tokens_gather(a, d->dtype, static_cast<hipStream_t>(stream)));
}

twell_status twell_tokens_combine(const twell_tokens_desc* d, const void* rows, const int32_t* pair_row,
                                  const float* weights, void* y, void* stream) {
  TWELL_TRY(check_tokens(d));
  if (d->T == 0) return TWELL_OK;
  TWELL_TRY(check_elems(rows, d->dtype));
  TWELL_TRY(check_elems(y, d->dtype));
  if (!pair_row || !aligned4(pair_row) || (weights && !aligned4(weights))) return TWELL_EINVAL;
  twell::TokensArgs a = tokens_args(d, pair_row);
  a.rows = rows;
  a.weights = weights;
  a.y = y;
  return from_hip(twell::launch_tokens_combine(a, d->dtype, static_cast<hipStream_t>(stream)));
}

twell_status twell_tokens_combine_bwd(const twell_tokens_desc* d, const void* rows, const int32_t* pair_row,
                                      const float* weights, const void* dy, void* drows, int64_t ld_drows,
                                      float* dweights, void* stream) {
  TWELL_TRY(check_tokens(d));
  if (drows && ld_drows < d->d_model) return TWELL_EINVAL;
  if (drows && ld_drows > kMaxStride) return TWELL_EUNSUPPORTED;
  if (d->T == 0 || (!drows && !dweights)) return TWELL_OK;
  TWELL_TRY(check_elems(dy, d->dtype));
  if (dweights) TWELL_TRY(check_elems(rows, d->dtype));
  if (drows) TWELL_TRY(check_elems(drows, d->dtype));
  if (!pair_row || !aligned4(pair_row) || !weights || !aligned4(weights) || (dweights && !aligned4(dweights)))
    return TWELL_EINVAL;
  twell::TokensArgs a = tokens_args(d, pair_row);
  a.rows = rows;
  a.weights = weights;
  a.dy = dy;
  a.rows_out = drows;
  a.ld_out = ld_drows;
  a.dweights = dweights;
  return from_hip(twell::launch_tokens_combine_bwd(a, d->dtype, static_cast<hipStream_t>(stream)));
}

twell_status twell_layernorm_sizes(const twell_norm_desc* d, size_t* ws) {
  TWELL_TRY(check_norm(d));
  if (!ws) return TWELL_EINVAL;
  *ws = norm_ws(d);
  return TWELL_OK;
}

twell_status twell_layernorm_fwd(const twell_norm_desc* d, const void* x, const void* w, const void* b, void* y,
                                 float* stats, void* stream) {
  TWELL_TRY(check_norm(d));
  if (d->T == 0) return TWELL_OK;
  TWELL_TRY(check_elems(x, d->dtype));
  TWELL_TRY(check_elems(y, d->dtype));
  if ((w && !elem_aligned(w, d->w_dtype)) || (b && !elem_aligned(b, d->w_dtype)) || (stats && !aligned4(stats)))
    return TWELL_EINVAL;
  twell::NormArgs a = norm_args(d);
  a.x = x;
  a.w = w;
  a.b = b;
  a.y = y;
  a.stats = stats;
  return from_hip(twell::launch_norm_fwd(a, d->dtype, d->w_dtype, static_cast<hipStream_t>(stream)));
}

twell_status twell_layernorm_bwd(const twell_norm_desc* d, const void* x, const void* w, const float* stats,
                                 const void* dy, void* dx, float* dw, float* db, void* ws, size_t ws_bytes,
                                 void* stream) {
  TWELL_TRY(check_norm(d));
  if (d->T > 0) {
    TWELL_TRY(check_elems(x, d->dtype));
    TWELL_TRY(check_elems(dy, d->dtype));
    TWELL_TRY(check_elems(dx, d->dtype));
    if (!stats || !aligned4(stats) || (w && !elem_aligned(w, d->w_dtype))) return TWELL_EINVAL;
    if (!ws || !aligned16(ws) || ws_bytes < norm_ws(d)) return TWELL_EINVAL;
  }
  if ((dw && !aligned4(dw)) || (db && !aligned4(db))) return TWELL_EINVAL;
  twell::NormArgs a = norm_args(d);
  a.x = x;
  a.w = w;
  a.stats_in = stats;
  a.dy = dy;
  a.dx = dx;
  a.dw = dw;
  a.db = db;
  a.part = static_cast<float*>(ws);
  return from_hip(twell::launch_norm_bwd(a, d->dtype, d->w_dtype, static_cast<hipStream_t>(stream)));
}

twell_status twell_fp8_weights_sizes(const twell_fp8_desc* d, twell_wsizes_t* out) {
  TWELL_TRY(check_fp8(d));
  if (!out) return TWELL_EINVAL;
  const size_t tiles = static_cast<size_t>(d->experts) * static_cast<size_t>(tiles_of(d->rows));
  const int32_t blocks = blocks_of(d->cols);
  out->codes = tiles * static_cast<size_t>(blocks) * 2048;
  out->scales = tiles * static_cast<size_t>(quads_of(blocks)) * 64;
  return TWELL_OK;
}

twell_status twell_fp8_weights_pack(const twell_fp8_desc* d, const void* w, int32_t w_dtype, twell_wplanes out,
                                    const twell_wplanes* out_t, void* stream) {
  TWELL_TRY(check_fp8(d));
  if (!known_dtype(w_dtype)) return TWELL_EINVAL;
  TWELL_TRY(check_elems(w, w_dtype));
  TWELL_TRY(check_fp8_planes(out));
  twell::F8PackArgs a = fp8_pack_args(d, out);
  a.w = w;
  if (out_t) {
    TWELL_TRY(check_fp8_planes(*out_t));
    a.codes_t = static_cast<uint8_t*>(out_t->codes);
    a.scales_t = static_cast<uint8_t*>(out_t->scales);
  }
  return from_hip(twell::launch_f8_pack(a, w_dtype, static_cast<hipStream_t>(stream)));
}

twell_status twell_fp8_weights_unpack(const twell_fp8_desc* d, twell_wplanes in, void* w, int32_t w_dtype,
                                      void* stream) {
  TWELL_TRY(check_fp8(d));
  if (!known_dtype(w_dtype)) return TWELL_EINVAL;
  TWELL_TRY(check_elems(w, w_dtype));
  TWELL_TRY(check_fp8_planes(in));
  twell::F8PackArgs a = fp8_pack_args(d, in);
  a.out = w;
  return from_hip(twell::launch_f8_unpack(a, w_dtype, static_cast<hipStream_t>(stream)));
}

twell_status twell_fp8_linear_sizes(const twell_fp8_desc* d, int64_t T, size_t* ws_fwd, size_t* ws_bwd) {
  TWELL_TRY(check_fp8(d));
  if (T < 0 || !ws_fwd || !ws_bwd) return TWELL_EINVAL;
  if (T > kMaxSide) return TWELL_EUNSUPPORTED;
  *ws_fwd = fp8_ws(d, T).total;
  *ws_bwd = fp8_bwd_ws(d, T);
  return TWELL_OK;
}

twell_status twell_fp8_linear_fwd(const twell_fp8_desc* d, twell_wplanes w, int64_t T, const int32_t* offsets,
                                  int32_t dtype, const void* x, int64_t ldx, void* y, int64_t ldy, void* ws,
                                  size_t ws_bytes, void* stream) {
  TWELL_TRY(check_fp8_rows(d, T, offsets, dtype));
  TWELL_TRY(check_stride(ldx, d->cols));
  TWELL_TRY(check_stride(ldy, d->rows));
  if (T == 0) return TWELL_OK;
  TWELL_TRY(check_elems(x, dtype));
  TWELL_TRY(check_elems(y, dtype));
  TWELL_TRY(check_fp8_planes(w));
  if (!ws || !aligned16(ws) || ws_bytes < fp8_ws(d, T).total) return TWELL_EINVAL;
  return fp8_product(d, w, T, offsets, dtype, x, ldx, y, ldy, ws, static_cast<hipStream_t>(stream));
}

twell_status twell_fp8_linear_bwd(const twell_fp8_desc* d, twell_wplanes w_t, int64_t T, const int32_t* offsets,
                                  int32_t dtype, const void* x, int64_t ldx, const void* dy, int64_t lddy, void* dx,
                                  int64_t lddx, float* dw, void* ws, size_t ws_bytes, void* stream) {
  TWELL_TRY(check_fp8_rows(d, T, offsets, dtype));
  TWELL_TRY(check_stride(lddy, d->rows));
  if (dw) TWELL_TRY(check_stride(ldx, d->cols));
  if (dx) TWELL_TRY(check_stride(lddx, d->cols));
  if (dw && !aligned4(dw)) return TWELL_EINVAL;
  const twell_fp8_desc t = transposed(d);
  if (T > 0 && (dx || dw)) {
    TWELL_TRY(check_elems(dy, dtype));
    if (dw) TWELL_TRY(check_elems(x, dtype));
    if (dx) {
      TWELL_TRY(check_elems(dx, dtype));
      TWELL_TRY(check_fp8_planes(w_t));
    }
    if (!ws || !aligned16(ws) || ws_bytes < fp8_bwd_ws(d, T)) return TWELL_EINVAL;
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dw) {
    twell::WgradArgs a{};
    a.x = x;
    a.dy = dy;
    a.dw = dw;
    a.offsets = T > 0 ? offsets : nullptr;
    a.T = T;
    a.ldx = ldx;
    a.ldy = lddy;
    a.N = d->rows;
    a.K = d->cols;
    a.experts = d->experts;
    a.parts = twell::wgrad_parts(T, d->rows, d->cols, d->experts);
    a.part = static_cast<float*>(ws);
    TWELL_TRY(from_hip(twell::launch_wgrad(a, dtype, s)));
  }
  if (!dx || T == 0) return TWELL_OK;
  return fp8_product(&t, w_t, T, offsets, dtype, dy, lddy, dx, lddx, ws, s);
}

const char* twell_status_str(twell_status s) {
  switch (s) {
    case TWELL_OK: return "ok";
    case TWELL_EINVAL: return "invalid argument (descriptor, pointer, alignment or workspace size)";
    case TWELL_EUNSUPPORTED: return "shape or dtype not supported by the library";
    case TWELL_EHIP: return "HIP launch error";
    case TWELL_ESCRATCH: return "the problem needs more scratch than the allocation-free entry point holds";
  }
  return "unknown status";
}

}  // extern "C"
