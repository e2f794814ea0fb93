/*
 * twell.h -- C ABI of libtwell: the TwELL activation-sparse gated FFN on MI355X (gfx950).
 *
 * The layer is  y = (ReLU(x W_gate) * (x W_up)) W_down  with a ReLU gate, whose
 * output is mostly exact zeros.  Sources: the page "Sakana AI and NVIDIA
 * introduce TwELL with CUDA kernels for 20.5% inference and 21.9% training"
 * (noticias.mechatronicstore.cl), called P2 below, sections
 *   "¿Qué hace distinto a TwELL frente a ELL clásico?"  (P2 §TwELL-vs-ELL):
 *       tile-local packing built in the gate matmul's epilogue, the fused
 *       up/down inference kernel, the hybrid ELL / dense-fallback format;
 *   "Receta de entrenamiento: dos cambios y nada más"  (P2 §Receta):
 *       ReLU gate, L1 penalty on the hidden activations;
 *   "¿Cuál es el problema que TwELL resuelve?"  (P2 §Problema):
 *       the dense Tensor-Core FFN that the sparse path is measured against.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Layouts (all row-major, contiguous):
 *      x, y, dy, dx     [T x d_model]          dtype
 *      w_gate_t         [d_ff x d_model]        dtype   row j = neuron j's gate weights
 *      w_up_t           [d_ff x d_model]        dtype   row j = neuron j's up weights
 *      w_down           [d_ff x d_model]        dtype   row j = neuron j's output row
 *    so g = x . w_gate_t^T, u = x . w_up_t^T, y = h . w_down.
 *  - TwELL (twell_act), with n_t = d_ff / tile_n and C = slots:
 *      count  int32  [T][n_t]        number of non-zeros of ReLU(g) in the (row, tile),
 *                                    the TRUE number even when it exceeds C;
 *      idx    uint8  [T][n_t][C]     tile-local column (0..tile_n-1) of each stored non-zero;
 *      val    dtype  [T][n_t][C]     its value ReLU(g) rounded to dtype.
 *    Slots s < min(count, C) hold the non-zeros in ascending column order; the
 *    others hold idx 0 and value +0.  A value is a non-zero iff its rounded
 *    (stored) value is not zero.
 *  - Pointers: every array argument is a DEVICE pointer, 16-byte aligned,
 *    owned by the caller.  The library never allocates or frees memory;
 *    scratch memory is passed in as `ws`, except by the allocation-free
 *    twell_ffn_fwd_hybrid_noalloc, whose scratch is a static device array.
 *  - Streams: `stream` is a hipStream_t passed as void* (NULL = default
 *    stream).  All calls are asynchronous: they return after host-side
 *    validation and the kernel launches, with no host synchronisation.
 *  - Errors: TWELL_EINVAL for a bad descriptor, NULL / misaligned pointer or
 *    too-small workspace (nothing is launched); TWELL_EUNSUPPORTED for a valid
 *    shape the library has no kernel for; TWELL_EHIP when a launch fails;
 *    TWELL_ESCRATCH when a problem exceeds the allocation-free entry point's
 *    static scratch (nothing is launched).
 *    Data-dependent conditions (overflowing tiles, dense-row cap exceeded) are
 *    reported in device counters, never as host errors.
 *  - Supported shapes: dtype BF16 with d_model % 512 == 0 and d_model <= 4096,
 *    or FP32 with d_model % 256 == 0 and d_model <= 2048; tile_n in {64, 128};
 *    d_ff % tile_n == 0; 1 <= slots <= tile_n; T >= 0 (T == 0 is a no-op);
 *    T * max(d_model, d_ff) < 2^31.
 *  - Threading: calls are thread-safe (the shared state is a per-device cache
 *    of the CU count and of the scratch address, held in atomics), except that
 *    calls of twell_ffn_fwd_hybrid_noalloc must not overlap on one device.
 */
#ifndef TWELL_H
#define TWELL_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  TWELL_OK = 0,
  TWELL_EINVAL = 1,
  TWELL_EUNSUPPORTED = 2,
  TWELL_EHIP = 3,
  TWELL_ESCRATCH = 4 /* the problem needs more scratch than the allocation-free entry point holds */
} twell_status;

typedef enum { TWELL_FP32 = 0, TWELL_BF16 = 1 } twell_dtype;

/* Problem descriptor.  T = tokens, d_model / d_ff = FFN widths, tile_n = TwELL
 * tile width T_n (the gate matmul's N tile), slots = C. */
typedef struct {
  int64_t T;
  int32_t d_model;
  int32_t d_ff;
  int32_t tile_n;
  int32_t slots;
  int32_t dtype; /* twell_dtype */
} twell_desc;

/* The three TwELL planes (device pointers, layouts above). */
typedef struct {
  int32_t* count;
  uint8_t* idx;
  void* val;
} twell_act;

/* Row routing of the hybrid format (device arrays owned by the caller).
 * Written by twell_ffn_fwd_hybrid; read by the backward. */
typedef struct {
  int32_t* ell_rows;      /* [T]               rows served from TwELL, ascending           */
  int32_t* dense_rows;    /* [max_dense_rows]  rows served by the dense fallback, ascending */
  int32_t* n_rows;        /* [3]  {n_ell, n_dense, dense rows beyond max_dense_rows}        */
  uint8_t* row_kind;      /* [T]  1 = row went to the dense fallback, 0 = TwELL             */
  int64_t max_dense_rows; /* capacity of dense_rows and of the fallback workspace           */
} twell_route;

/* Byte sizes of the TwELL planes and of the workspaces, for a descriptor. */
typedef struct {
  size_t count;        /* T * n_t * 4                                        */
  size_t idx;          /* T * n_t * C                                        */
  size_t val;          /* T * n_t * C * sizeof(dtype)                        */
  size_t ws_dense_fwd; /* twell_dense_ffn_fwd: h [T x d_ff] + W_down^T         */
  size_t ws_hybrid;    /* workspace of twell_ffn_fwd_hybrid (max_dense_rows)  */
  size_t ws_bwd;       /* workspace of twell_ffn_bwd (max_dense_rows)         */
  size_t ws_pack_classic; /* twell_pack_classic: dense ReLU(g) [T x d_ff]      */
} twell_sizes_t;

/* Fill *out for descriptor *d and a dense-row capacity (>= 0).  Host only.
 * Returns TWELL_EINVAL / TWELL_EUNSUPPORTED like the compute calls would. */
twell_status twell_sizes(const twell_desc* d, int64_t max_dense_rows, twell_sizes_t* out);

/* Gate GEMM + ReLU + TwELL pack, in ONE kernel dispatch.
 * [P2 §TwELL-vs-ELL: the sparse format is produced inside the epilogue of the
 * gate matmul, with no extra launch and no dense write of the activations.]
 *   x [T x d_model], w_gate_t [d_ff x d_model] (dtype)  ->  act (all three planes written).
 * g accumulates in fp32; ReLU(g) is rounded to dtype before the non-zero test.
 * stats  (device int64[2], nullable): ACCUMULATED (atomic add) with
 *        [0] += number of (row, tile) pairs whose count exceeds slots,
 *        [1] += sum of all counts (= non-zeros of ReLU(g));  zero it first.
 * gate_dbg (device, nullable): if given, the same kernel also writes the dense
 *        ReLU(g) [T x d_ff] in dtype (parity / debugging only; it is the dense
 *        write-back the method exists to avoid, so leave it NULL when timing). */
twell_status twell_pack(const twell_desc* d, const void* x, const void* w_gate_t, twell_act act,
                        int64_t* stats, void* gate_dbg, void* stream);

/* The same TwELL planes built the classic way, as a baseline for twell_pack:
 * [P2 §Problema and §TwELL-vs-ELL: converting a dense activation tensor to a
 * sparse format in a separate kernel costs an extra launch and a full write
 * and read of that tensor, which eats the saving.]
 * Kernel 1: the gate GEMM (same accumulation order as twell_pack) writes
 *           ReLU(g) rounded to dtype densely into ws, [T x d_ff];
 * Kernel 2: one wave per (row, tile) converts it to TwELL.
 * act is written exactly as twell_pack writes it (byte-identical planes).
 * ws: twell_sizes().ws_pack_classic bytes. */
twell_status twell_pack_classic(const twell_desc* d, const void* x, const void* w_gate_t, twell_act act,
                                void* ws, size_t ws_bytes, void* stream);

/* Fused up + down projection on TwELL input: one fused kernel, the
 * intermediate never written to memory.
 * [P2 §TwELL-vs-ELL: one fused kernel reads TwELL and runs the up and down
 * projections together; the intermediate never reaches global memory.]
 * Dispatches, by batch size T and row width d_model: below 2048 rows a
 * one-workgroup-per-row kernel (16 waves; 8 for bf16 rows wider than 2048), in
 * ONE dispatch; a one-wave-per-row kernel, in ONE dispatch, for fp32 rows
 * wider than 1024 and for bf16 rows wider than 2048 from 2048 to 4095 rows.
 * All other batches take the lockstep kernel (workgroups of W waves --
 * 16, or 8 for bf16 rows wider than 2048 -- that sweep the neuron tiles
 * together, each wave holding R rows: as many as its registers, the
 * workgroup's LDS and the per-wave list allow -- 2 at d_model = 2048 and at
 * 2560 .. 4096, 4 at d_model <= 1024 when C <= 32 -- but fewer while that
 * would leave CUs without a workgroup), dispatched once per generation of
 * workgroups the device runs at once (one per CU), on disjoint row blocks:
 * ceil(ceil(T / (W R)) / CUs) dispatches of the same kernel, e.g. 2 at
 * T = 16384, d_model = 2048 (W = 16, R = 2), 1 at T = 8192, d_model = 1024
 * (R = 2) and 4 at T = 16384, d_model = 4096 (W = 8, R = 2) on a 256-CU
 * MI355X.  Every row is computed start to finish by one workgroup of one
 * dispatch; a workgroup deals its rows to its waves by their entry counts (a
 * row's result does not depend on the wave).
 * Bits: each row's tiles are summed starting at a chunk that depends on its
 * workgroup's index and generation, hence on the device's CU count; y is
 * bitwise reproducible on one device (and on devices with the same CU count),
 * and within the stated tolerance elsewhere.
 * For every row t and stored slot (neuron j = b*tile_n + idx, value a):
 *   u = x[t] . w_up_t[j];  h = a * u;  y[t] += h * w_down[j]   (fp32 accumulate)
 * y [T x d_model] is overwritten (stored in dtype).  A tile with count > slots
 * contributes only its stored slots (the plain format is lossy there; the
 * hybrid entry point is the remedy). */
twell_status twell_ffn_fwd(const twell_desc* d, const void* x, twell_act act, const void* w_up_t,
                           const void* w_down, void* y, void* stream);

/* Hybrid forward: row router + fused TwELL path on ELL rows + dense MFMA
 * fallback on dense rows.  [P2 §TwELL-vs-ELL: for training, whose sparsity is
 * far from uniform, each row goes at run time either to a compact ELL store
 * or to a dense fallback when it has too many non-zeros.]
 * act must come from twell_pack on the same x and w_gate_t.
 * Kernels (same stream, no host synchronisation):
 *   1-2. router: a row is dense iff some tile has count > slots; ascending
 *        ell_rows / dense_rows, n_rows, row_kind.  At most max_dense_rows
 *        rows are kept dense; further dense rows are served (lossily) from
 *        TwELL and counted in n_rows[2].
 *   3.   fused up/down (as twell_ffn_fwd) over ell_rows; ELL rows with far
 *        more non-zeros than the batch's mean row (> max(2 slots, 2 x mean),
 *        at most 1024 of them) are cut into tile ranges processed in parallel
 *        and summed in a fixed order; the other ELL rows are dealt over
 *        windows of 8 lockstep workgroups by their entry counts.  Which
 *        workgroup computes a row therefore differs from twell_ffn_fwd, so its
 *        y can differ in the last bits (deterministic either way);
 *   4-5. dense gate|up GEMM over the gathered dense rows (h = ReLU(g) * u,
 *        recomputed, kept in ws), then the down GEMM scattered into y.
 * y [T x d_model] is overwritten.  ws: twell_sizes(d, max_dense_rows).ws_hybrid bytes. */
twell_status twell_ffn_fwd_hybrid(const twell_desc* d, const void* x, const void* w_gate_t, twell_act act,
                                  const void* w_up_t, const void* w_down, void* y, const twell_route* route,
                                  void* ws, size_t ws_bytes, void* stream);

/* Backward of the hybrid-format FFN, reusing the forward's TwELL and route.
 * [P2 §Receta: ReLU gate and an L1 term on the hidden activations;
 *  P2 §TwELL-vs-ELL: the training format is the hybrid one.]
 * Loss whose gradients are returned:  L = sum(y * dy) + l1_coef * sum|h|,
 * with h = ReLU(g) * u the hidden activation feeding w_down (sign(0) = 0,
 * ReLU'(0) = 0).  Given dy [T x d_model] (dtype):
 *   dx        [T x d_model]  dtype, overwritten (every row);
 *   dw_gate_t, dw_up_t, dw_down  [d_ff x d_model] fp32, overwritten.
 * act and route must be those of the twell_pack / twell_ffn_fwd_hybrid call on
 * the same x.  Rows in route->ell_rows use only their stored TwELL slots (a
 * row the forward served lossily from TwELL is differentiated the same way);
 * rows in route->dense_rows are recomputed densely on MFMA.
 * Deterministic: each neuron's weight gradient is the sum of its ELL rows'
 * terms in ascending token order, plus the dense rows' GEMM result (bitwise
 * the same on any device).  dx of the ELL rows comes from
 * a lockstep kernel dispatched once per generation of resident workgroups like
 * twell_ffn_fwd's (16 waves per workgroup, 8 for bf16 rows wider than 2048,
 * which take it from 4096 rows on and one wave per row below; fp32 rows wider
 * than 1024 always one wave per row), with the same dependence of its bits on
 * the CU count.
 * ws: twell_sizes(d, route->max_dense_rows).ws_bwd bytes. */
twell_status twell_ffn_bwd(const twell_desc* d, const void* x, twell_act act, const twell_route* route,
                           const void* w_gate_t, const void* w_up_t, const void* w_down, const void* dy,
                           float l1_coef, void* dx, float* dw_gate_t, float* dw_up_t, float* dw_down,
                           void* ws, size_t ws_bytes, void* stream);

/* Bytes of the static device scratch array of twell_ffn_fwd_hybrid_noalloc
 * (one copy per device the library runs on, held until the process ends). */
#define TWELL_NOALLOC_SCRATCH_BYTES ((size_t)128 << 20)

/* twell_ffn_fwd_hybrid without a workspace argument, for callers that cannot
 * allocate device memory: code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc.  Same arguments, kernels, results (bit for
 * bit) and route outputs as twell_ffn_fwd_hybrid; its workspace is instead a
 * static device array of TWELL_NOALLOC_SCRATCH_BYTES per device, whose device
 * address is looked up (hipGetSymbolAddress) on the first call on each
 * device.  It calls no hipMalloc / hipFree and allocates nothing.
 *   Limit: twell_sizes(d, route->max_dense_rows).ws_hybrid must not exceed
 *   TWELL_NOALLOC_SCRATCH_BYTES, else TWELL_ESCRATCH is returned and nothing
 *   is launched (e.g. the 2B-class shape, T = 16384, d_model = 2048,
 *   d_ff = 8192, fits with max_dense_rows up to 454).
 *   Every call on a device shares that device's array: calls that overlap on
 *   one device (other streams, other threads) race and must not be issued.
 *   The array keeps the last call's contents; no part of it needs to start
 *   at zero (every workspace entry is written before it is read). */
twell_status twell_ffn_fwd_hybrid_noalloc(const twell_desc* d, const void* x, const void* w_gate_t,
                                          twell_act act, const void* w_up_t, const void* w_down, void* y,
                                          const twell_route* route, void* stream);

/* The library's own dense MFMA FFN, the baseline the sparse path is compared with.
 * [P2 §Problema: GPUs are built for dense matrix products; the sparse path must
 * beat the dense one.]
 * Kernel 1: W_down^T [d_model x d_ff] written into ws (after h, 256-byte aligned);
 * Kernel 2: g = x w_gate, u = x w_up in one GEMM, epilogue h = ReLU(g) * u
 *           stored to ws as dtype [T x d_ff];
 * Kernel 3: y = h w_down (y overwritten, dtype).
 * ws must hold twell_sizes().ws_dense_fwd bytes. */
twell_status twell_dense_ffn_fwd(const twell_desc* d, const void* x, const void* w_gate_t,
                                 const void* w_up_t, const void* w_down, void* y, void* ws,
                                 size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * Serving a few tokens: weights laid out once (in 4 bits or bf16), a product
 * with 4-bit weights, and a mixture-of-experts gated feed-forward layer.
 *
 * These entry points take odd widths and strided rows.  x, y, w and w_router
 * need only the alignment of their elements; planes and workspaces are 16-byte
 * aligned.  Rows of x and y are ldx / ldy elements apart (>= their width), and
 * x and y must not overlap.  Limits: rows, inputs and tokens up to 2^20, rows x
 * inputs of one matrix up to 2^34, 1024 experts, top_k up to 32, strides up to
 * 2^40 elements (TWELL_EUNSUPPORTED beyond). */

/* `experts` matrices of `rows` outputs x `cols` inputs held in `bits` (4 or 16)
 * per weight.  bits = 4: `group` (32, 64 or 128) consecutive inputs of a row
 * share one scale (the last group of a row may be short); bits = 16: group = 0. */
typedef struct {
  int32_t experts;
  int32_t rows;
  int32_t cols;
  int32_t bits;
  int32_t group;
} twell_wdesc;

/* Laid-out weights (device pointers; scales is not used for 16 bits).  Blocks
 * of 16 rows x 128 inputs, [experts][ceil(rows/16)][ceil(cols/128)], padded with
 * zeros.  In a block, lane l (0..63) holds row l % 16 and inputs 32 s + 8 (l / 16)
 * + 0..7 for s = 0..3:
 *   bits = 16: bf16 [s][l][8]                                        4096 bytes
 *   bits = 4:  32-bit words [l][s], codes as q + 8: input 2j of the eight in bits
 *              4j+3 .. 4j+6 and input 2j+1 in bits 4j+19 .. 4j+22, bit numbers
 *              modulo 32 (the word is rotated left by three)           1024 bytes
 *              and scales bf16 [16 rows][128 / group]. */
typedef struct {
  void* codes;
  void* scales;
} twell_wplanes;

typedef struct {
  size_t codes;
  size_t scales;
} twell_wsizes_t;

/* Byte sizes of the planes.  Host only. */
twell_status twell_weights_sizes(const twell_wdesc* d, twell_wsizes_t* out);

/* Lay weights out.  w: [experts][rows][cols], or with transposed = 1
 * [experts][cols][rows] (w_down as the layer above keeps it, one row per
 * neuron, is the transposed form of its d_model x d_ff matrix); contiguous,
 * bf16, or fp32 when bits = 4.
 * bits = 4: scale s = bf16(max|w| * r) of the group, r = 1/7 in fp32; code q =
 * w / s in fp32, rounded to nearest even and clamped to -7 .. 7 (0 where s = 0).
 * A group that holds an infinity or a NaN gets a NaN scale: all its values
 * become NaN. */
twell_status twell_weights_pack(const twell_wdesc* d, const void* w, int32_t w_dtype, int32_t transposed,
                                twell_wplanes out, void* stream);

/* The values the planes stand for, q * s (exact in fp32) or the bf16 weights,
 * written to w [experts][rows][cols] (bf16, or fp32 when bits = 4). */
twell_status twell_weights_unpack(const twell_wdesc* d, twell_wplanes in, void* w, int32_t w_dtype, void* stream);

/* y[t, n] = sum_k x[t, k] q[n, k] s[n, k / group]: the product of T tokens with
 * one matrix of 4-bit weights (experts = 1, bits = 4), fp32 sums.
 *   x [T x cols], y [T x rows] in dtype, rows ldx / ldy apart.
 * Made for few tokens: the weights are read once per 4 to 64 of them, by how
 * many there are and how many workgroups that makes.  T = 0 is a no-op.
 * Products x q are exact (fp32 data is cut into three bf16 parts for them, whose
 * last bits end at 2^-133: inputs below 2^-109 have fewer than 24), so an input
 * takes nothing from a row whose code for it is 0, and a group's sum of x q is
 * finite where it is in fp32.  An infinite or NaN input makes its own token's
 * outputs NaN, and no other token's.  Deterministic. */
twell_status twell_linear_fwd(const twell_wdesc* d, twell_wplanes w, int64_t T, int32_t dtype, const void* x,
                              int64_t ldx, void* y, int64_t ldy, void* stream);

typedef enum { TWELL_RELU = 0, TWELL_SILU = 1 } twell_activation;

/* Mixture of experts: T tokens, `experts` gated feed-forward layers of d_model x
 * d_ff, top_k of them per token; dtype of x, w_router and y; bits and group of
 * the experts' weights; renorm = 1 divides the chosen weights by their sum. */
typedef struct {
  int64_t T;
  int64_t ldx;
  int64_t ldy;
  int32_t d_model;
  int32_t d_ff;
  int32_t experts;
  int32_t top_k;
  int32_t dtype; /* twell_dtype */
  int32_t bits;
  int32_t group;
  int32_t act; /* twell_activation */
  int32_t renorm;
} twell_moe_desc;

/* Workspace bytes of twell_moe_fwd.  Host only. */
twell_status twell_moe_sizes(const twell_moe_desc* d, size_t* ws);

/* The whole layer:
 *   l[t, e] = x[t] . w_router[e] + router_bias[e]        (fp32)
 *   ids[t]  = the top_k largest l[t], in descending order; equal ones in ascending
 *             order of e; a NaN counts as the largest
 *   weights[t] = softmax(l[t]) over all experts, at ids[t]  (/ their sum if renorm)
 *   y[t] = sum_i weights[t, i] W_down_e (act(W_gate_e x[t]) * (W_up_e x[t])), e = ids[t, i]
 * gate, up: planes of {experts, d_ff, d_model, bits, group}; down: planes of
 * {experts, d_model, d_ff, bits, group}.  w_router [experts x d_model] dtype,
 * contiguous; router_bias [experts] fp32 or NULL (-inf takes an expert out).
 * Outputs: y, ids int32 [T x top_k], weights fp32 [T x top_k].
 * An expert whose weight is 0 adds nothing (its product is not formed), so a
 * row whose logits are all -inf has weights 0 and y = 0.  A NaN logit makes its
 * token's weights and y NaN, no other token's.
 * Hidden values are kept to 16 bits of mantissa (bf16 data) or 24 (fp32); sums
 * are fp32.  With infinite inputs, and with hidden values that overflow, the
 * token's y is NaN.  Deterministic.  ws: twell_moe_sizes() bytes; nothing in it
 * needs to start at zero.  Made for few tokens: 64 of them at a time, an expert's
 * weights once per 16 of its tokens (its down projection once per token where
 * there is little to read).  T = 0 is a no-op. */
twell_status twell_moe_fwd(const twell_moe_desc* d, const void* x, const void* w_router, const float* router_bias,
                           twell_wplanes gate, twell_wplanes up, twell_wplanes down, void* y, int32_t* ids,
                           float* weights, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * A mixture-of-experts layer over many tokens, for training and long prompts:
 * tokens sorted by expert and back with their weights, products with weights in
 * 8-bit floating point, and layer norm, each with its gradients.
 *
 * As above, odd widths and strided rows: tensors need only the alignment of
 * their elements (int32 and fp32 arrays 4 bytes, workspaces 16).  Tensors of one
 * call must not overlap where not said otherwise.  Limits: 2^20 tokens, T x
 * d_model up to 2^33, 1024 experts, top_k up to 32, strides up to 2^40 elements
 * (TWELL_EUNSUPPORTED beyond).  T = 0 reads no tensor.  All are deterministic.  A
 * workspace belongs to one call at a time: calls, or graphs that hold some, that may
 * run at once need one each. */

/* T tokens, top_k choices among `experts` each.  A pair p = t * top_k + i is
 * choice i of token t; there are up to T * top_k sorted rows.  Rows of
 * token tensors are ld_tokens elements apart, those of row tensors ld_rows. */
typedef struct {
  int64_t T;
  int64_t ld_tokens;
  int64_t ld_rows;
  int32_t d_model;
  int32_t experts;
  int32_t top_k;
  int32_t dtype; /* twell_dtype */
} twell_tokens_desc;

/* Workspace bytes of twell_tokens_sort.  Host only. */
twell_status twell_tokens_sizes(const twell_tokens_desc* d, size_t* ws);

/* The order of pairs by expert, stable (a lower pair first):
 *   ids [T x top_k] -> offsets [experts + 1], pair_row [T x top_k]
 * Rows offsets[e] .. offsets[e + 1] - 1 are expert e's, offsets[0] = 0; row
 * pair_row[p] belongs to pair p.  A pair whose id is not one of 0 .. experts - 1
 * is left out: pair_row[p] = -1.  A token may choose an expert twice.  ws: nothing
 * in it needs to start at zero. */
twell_status twell_tokens_sort(const twell_tokens_desc* d, const int32_t* ids, int32_t* offsets, int32_t* pair_row,
                               void* ws, size_t ws_bytes, void* stream);

/* rows[pair_row[p]] = x[p / top_k]: x [T x d_model], rows [T * top_k x d_model].
 * Rows behind offsets[experts] are left as they are.  Its gradient is
 * twell_tokens_combine without weights; it is that call's. */
twell_status twell_tokens_gather(const twell_tokens_desc* d, const void* x, const int32_t* pair_row, void* rows,
                                 void* stream);

/* y[t] = sum_i weights[t, i] rows[pair_row[t, i]], fp32 sums over ascending i
 * rounded once.  weights [T x top_k] fp32, or NULL: ones.  A pair left out, and
 * one whose weight is 0, adds nothing, whatever the row holds. */
twell_status twell_tokens_combine(const twell_tokens_desc* d, const void* rows, const int32_t* pair_row,
                                  const float* weights, void* y, void* stream);

/* The gradients of twell_tokens_combine with weights:
 *   drows[pair_row[t, i]] = weights[t, i] dy[t],  dweights[t, i] = rows[pair_row[t, i]] . dy[t]
 * dy [T x d_model]; drows like rows, its rows ld_drows apart; dweights [T x top_k]
 * fp32, 0 for a pair left out.  Either output may be NULL; rows may be NULL
 * without dweights.  drows may be rows itself (ld_drows = ld_rows).  Rows behind
 * offsets[experts] are left as they are. */
twell_status twell_tokens_combine_bwd(const twell_tokens_desc* d, const void* rows, const int32_t* pair_row,
                                      const float* weights, const void* dy, void* drows, int64_t ld_drows,
                                      float* dweights, void* stream);

/* `experts` matrices of `rows` outputs x `cols` inputs in 8-bit floating point
 * (e4m3: values up to 448, no infinities).  Limits: rows and cols up to 2^20, rows
 * x cols of one matrix up to 2^34, T x rows and T x cols up to 2^37. */
typedef struct {
  int32_t experts;
  int32_t rows;
  int32_t cols;
} twell_fp8_desc;

/* Byte sizes of the planes.  Host only.  The planes (16-byte aligned) are blocks
 * of 16 rows x 128 inputs, [experts][ceil(rows/16)][ceil(cols/128)], 2048 bytes,
 * padded with zeros: in a block, lane l (0..63) holds row l % 16 and inputs 32 s +
 * 8 (l / 16) + 0..7 for s = 0..3, steps 0 and 1 at byte 16 l, steps 2 and 3 at 1024
 * + 16 l; and a scale byte b, standing for 2^(b - 127), for each row of a block,
 * [experts][ceil(rows/16)][ceil(blocks/4)][16 rows][4 blocks].  Rows 128 r .. 128 r +
 * 127 of a matrix have to hold the same byte for a block, and all 16 rows of a tile
 * have it, as packing leaves them: products may read it from any one of those rows. */
twell_status twell_fp8_weights_sizes(const twell_fp8_desc* d, twell_wsizes_t* out);

/* Lay weights w [experts][rows][cols] (contiguous, bf16 or fp32) out.  128 x 128
 * weights share a scale: s = the smallest power of two from 2^-126 on with
 * max|w| <= 448 s; code = w / s rounded to nearest even.  An infinity or a NaN gets
 * a NaN code and has no part in the scale.  out_t, if not NULL, gets the planes of
 * {experts, cols, rows} of the transposed matrices, which hold the same values. */
twell_status twell_fp8_weights_pack(const twell_fp8_desc* d, const void* w, int32_t w_dtype, twell_wplanes out,
                                    const twell_wplanes* out_t, void* stream);

/* The values that planes stand for, written to w [experts][rows][cols] (bf16, which
 * holds them exactly from 2^-126 on, or fp32). */
twell_status twell_fp8_weights_unpack(const twell_fp8_desc* d, twell_wplanes in, void* w, int32_t w_dtype,
                                      void* stream);

/* Workspace bytes of the calls below with T rows.  Host only. */
twell_status twell_fp8_linear_sizes(const twell_fp8_desc* d, int64_t T, size_t* ws_fwd, size_t* ws_bwd);

/* y[t] = W_e Q(x[t]): T rows through their expert's matrix.
 *   x [T x cols], y [T x rows] in dtype, rows ldx / ldy apart
 *   offsets [experts + 1] (device): rows offsets[e] .. offsets[e + 1] - 1 are expert
 *   e's, as twell_tokens_sort leaves them; rows beside them are left as they are in
 *   y.  NULL with one expert: all rows.
 * Q rounds a row to e4m3 with a scale for each 128 inputs, by the rule of
 * twell_fp8_weights_pack; that is the only rounding of inputs.  dtype fp32: products
 * of codes are exact and sums fp32, but a rounded input or weight, or a product of
 * two, below 2^-126 may count as 0, here and in dx.  dtype bf16: the matrix core's
 * 8-bit products, where such a product may count as 0 too.
 * It cuts the products of 8 consecutive inputs to multiples of 2^-13 of the largest
 * one's power of two before it adds them in fp32, so that a sum is off by less than
 * 7 * 2^-13 of the largest product of each 8 (1.4e-5 of the norm for Gaussian data,
 * where y's own rounding is 1.7e-3).  Inputs and weights within 2^-1 of fp32's
 * largest value may round to infinities (fp32).  An infinite or NaN
 * input makes its own row's y NaN, and no other. */
twell_status twell_fp8_linear_fwd(const twell_fp8_desc* d, twell_wplanes w, int64_t T, const int32_t* offsets,
                                  int32_t dtype, const void* x, int64_t ldx, void* y, int64_t ldy, void* ws,
                                  size_t ws_bytes, void* stream);

/* The gradients, the roundings of x and W taken as if they were none:
 *   dx[t] = W_e^T Q(dy[t])          (w_t: the planes of {experts, cols, rows})
 *   dw_e  = sum_t dy[t] x[t]^T      over expert e's rows
 * dw [experts][rows x cols] fp32, from x and dy themselves with fp32 sums, is
 * overwritten (zeros for an expert without rows).  dx [T x cols] like y above.
 * Either may be NULL; without dw x may be NULL, without dx w_t's pointers. */
twell_status twell_fp8_linear_bwd(const twell_fp8_desc* d, twell_wplanes w_t, int64_t T, const int32_t* offsets,
                                  int32_t dtype, const void* x, int64_t ldx, const void* dy, int64_t lddy, void* dx,
                                  int64_t lddx, float* dw, void* ws, size_t ws_bytes, void* stream);

/* Layer norm of T rows of d_model (up to 16384) elements; rows of x are ldx
 * apart, those of y and dy ldy, those of dx lddx.  dtype: of x, y, dy and dx;
 * w_dtype: of w and b. */
typedef struct {
  int64_t T;
  int64_t ldx;
  int64_t ldy;
  int64_t lddx;
  int32_t d_model;
  int32_t dtype;   /* twell_dtype */
  int32_t w_dtype; /* twell_dtype */
  float eps;       /* >= 0 */
} twell_norm_desc;

/* Workspace bytes of twell_layernorm_bwd.  Host only. */
twell_status twell_layernorm_sizes(const twell_norm_desc* d, size_t* ws);

/* y = (x - mean) rstd w + b, rstd = 1 / sqrt(mean((x - mean)^2) + eps), over each
 * row; fp32 sums.  w [d_model] or NULL: ones; b [d_model] or NULL: zeros.  stats
 * [T x 2] fp32 gets mean and rstd of each row for the backward call; may be NULL.
 * y may be x itself (ldy = ldx). */
twell_status twell_layernorm_fwd(const twell_norm_desc* d, const void* x, const void* w, const void* b, void* y,
                                 float* stats, void* stream);

/* With h = (x - mean) rstd and g = dy w:
 *   dx = rstd (g - mean(g) - h mean(g h)),  dw = sum_t dy h,  db = sum_t dy
 * dx [T x d_model] is overwritten, and may be x or dy itself (same stride); dw and db
 * [d_model] fp32 are overwritten (zeros for T = 0); either may be NULL. */
twell_status twell_layernorm_bwd(const twell_norm_desc* d, const void* x, const void* w, const float* stats,
                                 const void* dy, void* dx, float* dw, float* db, void* ws, size_t ws_bytes,
                                 void* stream);

/* Static description of a status code. */
const char* twell_status_str(twell_status s);

#ifdef __cplusplus
}
#endif

#endif /* TWELL_H */
