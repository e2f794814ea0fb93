"""Thin ctypes binding of libtwell (include/twell.h).

Argument marshalling only: every step of the layer runs in the HIP kernels of
libtwell.so.  The binding checks what a raw pointer cannot carry -- that each
tensor lives on the GPU, is contiguous, has the expected dtype and is large
enough for the descriptor -- so that no kernel is ever handed a host pointer
or an undersized buffer.  If libtwell.so is missing the import of this module
still works, but every call raises: there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
from dataclasses import dataclass, fields
from typing import NamedTuple, Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libtwell.so")

TWELL_OK, TWELL_EINVAL, TWELL_EUNSUPPORTED, TWELL_EHIP, TWELL_ESCRATCH = 0, 1, 2, 3, 4
NOALLOC_SCRATCH_BYTES = 128 << 20  # TWELL_NOALLOC_SCRATCH_BYTES
TWELL_FP32, TWELL_BF16 = 0, 1

EXPORTED = ("twell_sizes", "twell_pack", "twell_pack_classic", "twell_ffn_fwd", "twell_ffn_fwd_hybrid",
            "twell_ffn_bwd", "twell_dense_ffn_fwd", "twell_status_str", "twell_ffn_fwd_hybrid_noalloc",
            "twell_weights_sizes", "twell_weights_pack", "twell_weights_unpack", "twell_linear_fwd",
            "twell_moe_sizes", "twell_moe_fwd")


class TwellError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn}: status {code} ({status_str(code)})")
        self.code = code


class CDesc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("d_model", ctypes.c_int32), ("d_ff", ctypes.c_int32),
                ("tile_n", ctypes.c_int32), ("slots", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class CAct(ctypes.Structure):
    _fields_ = [("count", ctypes.c_void_p), ("idx", ctypes.c_void_p), ("val", ctypes.c_void_p)]


class CRoute(ctypes.Structure):
    _fields_ = [("ell_rows", ctypes.c_void_p), ("dense_rows", ctypes.c_void_p), ("n_rows", ctypes.c_void_p),
                ("row_kind", ctypes.c_void_p), ("max_dense_rows", ctypes.c_int64)]


class CSizes(ctypes.Structure):
    _fields_ = [("count", ctypes.c_size_t), ("idx", ctypes.c_size_t), ("val", ctypes.c_size_t),
                ("ws_dense_fwd", ctypes.c_size_t), ("ws_hybrid", ctypes.c_size_t), ("ws_bwd", ctypes.c_size_t),
                ("ws_pack_classic", ctypes.c_size_t)]


class CWDesc(ctypes.Structure):
    _fields_ = [("experts", ctypes.c_int32), ("rows", ctypes.c_int32), ("cols", ctypes.c_int32),
                ("bits", ctypes.c_int32), ("group", ctypes.c_int32)]


class CPlanes(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class CWSizes(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_size_t), ("scales", ctypes.c_size_t)]


class CMoeDesc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("ldx", ctypes.c_int64), ("ldy", ctypes.c_int64),
                ("d_model", ctypes.c_int32), ("d_ff", ctypes.c_int32), ("experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("dtype", ctypes.c_int32), ("bits", ctypes.c_int32),
                ("group", ctypes.c_int32), ("act", ctypes.c_int32), ("renorm", ctypes.c_int32)]


_lib = None


def library() -> ctypes.CDLL:
    """Load libtwell.so once; raise if it was not built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m activation_sparse_feedforward_amd.build` (no CPU fallback exists)")
        lib = ctypes.CDLL(LIB_PATH)
        P, I32, I64, SZ, ST = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
        D = ctypes.POINTER(CDesc)
        R = ctypes.POINTER(CRoute)
        sig = {
            "twell_sizes": (ST, [D, I64, ctypes.POINTER(CSizes)]),
            "twell_ffn_fwd_hybrid": (ST, [D, P, P, CAct, P, P, P, R, P, SZ, P]),
            "twell_ffn_fwd_hybrid_noalloc": (ST, [D, P, P, CAct, P, P, P, R, P]),
            "twell_ffn_bwd": (ST, [D, P, CAct, R, P, P, P, P, ctypes.c_float, P, P, P, P, P, SZ, P]),
            "twell_pack": (ST, [D, P, P, CAct, P, P, P]),
            "twell_pack_classic": (ST, [D, P, P, CAct, P, SZ, P]),
            "twell_ffn_fwd": (ST, [D, P, CAct, P, P, P, P]),
            "twell_dense_ffn_fwd": (ST, [D, P, P, P, P, P, P, SZ, P]),
            "twell_status_str": (ctypes.c_char_p, [ST]),
            "twell_weights_sizes": (ST, [ctypes.POINTER(CWDesc), ctypes.POINTER(CWSizes)]),
            "twell_weights_pack": (ST, [ctypes.POINTER(CWDesc), P, I32, I32, CPlanes, P]),
            "twell_weights_unpack": (ST, [ctypes.POINTER(CWDesc), CPlanes, P, I32, P]),
            "twell_linear_fwd": (ST, [ctypes.POINTER(CWDesc), CPlanes, I64, I32, P, I64, P, I64, P]),
            "twell_moe_sizes": (ST, [ctypes.POINTER(CMoeDesc), ctypes.POINTER(SZ)]),
            "twell_moe_fwd": (ST, [ctypes.POINTER(CMoeDesc), P, P, P, CPlanes, CPlanes, CPlanes, P, P, P, P, SZ, P]),
        }
        for name, (res, args) in sig.items():
            f = getattr(lib, name)
            f.restype, f.argtypes = res, args
        _lib = lib
    return _lib


def status_str(code: int) -> str:
    return library().twell_status_str(int(code)).decode()


# ----------------------------------------------------------------------------- descriptor
@dataclass(frozen=True)
class Desc:
    T: int
    d_model: int
    d_ff: int
    tile_n: int
    slots: int
    dtype: str  # "fp32" | "bf16"

    @property
    def n_t(self) -> int:
        return self.d_ff // self.tile_n

    @property
    def torch_dtype(self) -> torch.dtype:
        return torch.bfloat16 if self.dtype == "bf16" else torch.float32

    def c(self) -> CDesc:
        return CDesc(int(self.T), int(self.d_model), int(self.d_ff), int(self.tile_n), int(self.slots),
                     TWELL_BF16 if self.dtype == "bf16" else TWELL_FP32)

    def with_T(self, T: int) -> "Desc":
        return Desc(T, self.d_model, self.d_ff, self.tile_n, self.slots, self.dtype)


class Act(NamedTuple):
    """The three TwELL planes as device tensors."""
    count: torch.Tensor  # int32 [T, n_t]
    idx: torch.Tensor    # uint8 [T, n_t, C]
    val: torch.Tensor    # dtype [T, n_t, C]


class Route(NamedTuple):
    """Row routing of the hybrid format as device tensors."""
    ell_rows: torch.Tensor    # int32 [T]
    dense_rows: torch.Tensor  # int32 [max_dense_rows]
    n_rows: torch.Tensor      # int32 [3]: n_ell, n_dense, dense rows over the cap
    row_kind: torch.Tensor    # uint8 [T]: 1 = dense fallback

    @property
    def max_dense_rows(self) -> int:
        return int(self.dense_rows.numel())


# The entry points below share one C struct and one size table per descriptor
# (the library only reads the struct): at small batches the host cost of a
# call, not the kernels, sets the pace of a step.
@functools.lru_cache(maxsize=256)
def _cdesc(desc: Desc) -> CDesc:
    return desc.c()


@functools.lru_cache(maxsize=256)
def _sizes(desc: Desc, max_dense_rows: int) -> dict:
    out = CSizes()
    st = library().twell_sizes(ctypes.byref(_cdesc(desc)), ctypes.c_int64(max_dense_rows), ctypes.byref(out))
    if st != TWELL_OK:
        raise TwellError("twell_sizes", st)
    return {k: int(getattr(out, k)) for k, _ in CSizes._fields_}


def sizes(desc: Desc, max_dense_rows: int = 0) -> dict:
    return dict(_sizes(desc, int(max_dense_rows)))


def alloc_act(desc: Desc, device="cuda") -> Act:
    return Act(torch.empty((desc.T, desc.n_t), dtype=torch.int32, device=device),
               torch.empty((desc.T, desc.n_t, desc.slots), dtype=torch.uint8, device=device),
               torch.empty((desc.T, desc.n_t, desc.slots), dtype=desc.torch_dtype, device=device))


def alloc_route(desc: Desc, max_dense_rows: int, device="cuda") -> Route:
    return Route(torch.empty(max(desc.T, 1), dtype=torch.int32, device=device),
                 torch.empty(max_dense_rows, dtype=torch.int32, device=device),
                 torch.zeros(3, dtype=torch.int32, device=device),
                 torch.empty(max(desc.T, 1), dtype=torch.uint8, device=device))


# ----------------------------------------------------------------------------- checks
def _ptr(t: Optional[torch.Tensor], name: str, nbytes: int, dtype: Optional[torch.dtype] = None) -> int:
    if t is None:
        return 0
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a GPU tensor (got {t.device})")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.nbytes < nbytes:
        raise ValueError(f"{name}: {t.nbytes} bytes, need {nbytes}")
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _act(desc: Desc, act: Act) -> CAct:
    sz = _sizes(desc, 0)
    return CAct(_ptr(act.count, "count", sz["count"], torch.int32),
                _ptr(act.idx, "idx", sz["idx"], torch.uint8),
                _ptr(act.val, "val", sz["val"], desc.torch_dtype))


def _route(desc: Desc, route: Route) -> CRoute:
    cap = route.max_dense_rows
    return CRoute(_ptr(route.ell_rows, "ell_rows", desc.T * 4, torch.int32),
                  _ptr(route.dense_rows, "dense_rows", cap * 4, torch.int32) if cap else 0,
                  _ptr(route.n_rows, "n_rows", 12, torch.int32),
                  _ptr(route.row_kind, "row_kind", desc.T, torch.uint8), cap)


def _check(fn: str, st: int):
    if st != TWELL_OK:
        raise TwellError(fn, st)


# ----------------------------------------------------------------------------- entry points
def twell_pack(desc: Desc, x, w_gate_t, act: Act, stats=None, gate_dbg=None, stream=None):
    """Gate GEMM + ReLU + TwELL pack in one dispatch (see include/twell.h)."""
    e = 2 if desc.dtype == "bf16" else 4
    dt = desc.torch_dtype
    _check("twell_pack", library().twell_pack(
        ctypes.byref(_cdesc(desc)), _ptr(x, "x", desc.T * desc.d_model * e, dt),
        _ptr(w_gate_t, "w_gate_t", desc.d_ff * desc.d_model * e, dt), _act(desc, act),
        _ptr(stats, "stats", 16, torch.int64), _ptr(gate_dbg, "gate_dbg", desc.T * desc.d_ff * e, dt),
        _stream(stream)))


def twell_pack_classic(desc: Desc, x, w_gate_t, act: Act, ws, stream=None):
    """Baseline: dense gate GEMM writing ReLU(g) to ws, then a conversion kernel
    to the same TwELL planes (see include/twell.h)."""
    e = 2 if desc.dtype == "bf16" else 4
    dt = desc.torch_dtype
    need = _sizes(desc, 0)["ws_pack_classic"]
    _check("twell_pack_classic", library().twell_pack_classic(
        ctypes.byref(_cdesc(desc)), _ptr(x, "x", desc.T * desc.d_model * e, dt),
        _ptr(w_gate_t, "w_gate_t", desc.d_ff * desc.d_model * e, dt), _act(desc, act), _ptr(ws, "ws", need),
        ctypes.c_size_t(ws.numel() * ws.element_size() if ws is not None else 0), _stream(stream)))


def twell_ffn_fwd(desc: Desc, x, act: Act, w_up_t, w_down, y, stream=None):
    """Fused TwELL up + down projection: one fused kernel, dispatched once per
    generation of resident workgroups for large batches (see include/twell.h)."""
    e = 2 if desc.dtype == "bf16" else 4
    dt = desc.torch_dtype
    _check("twell_ffn_fwd", library().twell_ffn_fwd(
        ctypes.byref(_cdesc(desc)), _ptr(x, "x", desc.T * desc.d_model * e, dt), _act(desc, act),
        _ptr(w_up_t, "w_up_t", desc.d_ff * desc.d_model * e, dt),
        _ptr(w_down, "w_down", desc.d_ff * desc.d_model * e, dt),
        _ptr(y, "y", desc.T * desc.d_model * e, dt), _stream(stream)))


def twell_ffn_fwd_hybrid(desc: Desc, x, w_gate_t, act: Act, w_up_t, w_down, y, route: Route, ws, stream=None):
    """Router + fused TwELL path on ELL rows + dense MFMA fallback on dense rows."""
    e = 2 if desc.dtype == "bf16" else 4
    dt = desc.torch_dtype
    need = _sizes(desc, route.max_dense_rows)["ws_hybrid"]
    cr = _route(desc, route)
    _check("twell_ffn_fwd_hybrid", library().twell_ffn_fwd_hybrid(
        ctypes.byref(_cdesc(desc)), _ptr(x, "x", desc.T * desc.d_model * e, dt),
        _ptr(w_gate_t, "w_gate_t", desc.d_ff * desc.d_model * e, dt), _act(desc, act),
        _ptr(w_up_t, "w_up_t", desc.d_ff * desc.d_model * e, dt),
        _ptr(w_down, "w_down", desc.d_ff * desc.d_model * e, dt),
        _ptr(y, "y", desc.T * desc.d_model * e, dt), ctypes.byref(cr), _ptr(ws, "ws", need),
        ctypes.c_size_t(ws.numel() * ws.element_size() if ws is not None else 0), _stream(stream)))


def twell_ffn_fwd_hybrid_noalloc(desc: Desc, x, w_gate_t, act: Act, w_up_t, w_down, y, route: Route,
                                 stream=None):
    """twell_ffn_fwd_hybrid with the library's static device scratch as its
    workspace: allocates nothing (see include/twell.h for the size limit and
    the rule that calls on one device must not overlap)."""
    e = 2 if desc.dtype == "bf16" else 4
    dt = desc.torch_dtype
    cr = _route(desc, route)
    _check("twell_ffn_fwd_hybrid_noalloc", library().twell_ffn_fwd_hybrid_noalloc(
        ctypes.byref(_cdesc(desc)), _ptr(x, "x", desc.T * desc.d_model * e, dt),
        _ptr(w_gate_t, "w_gate_t", desc.d_ff * desc.d_model * e, dt), _act(desc, act),
        _ptr(w_up_t, "w_up_t", desc.d_ff * desc.d_model * e, dt),
        _ptr(w_down, "w_down", desc.d_ff * desc.d_model * e, dt),
        _ptr(y, "y", desc.T * desc.d_model * e, dt), ctypes.byref(cr), _stream(stream)))


def twell_ffn_bwd(desc: Desc, x, act: Act, route: Route, w_gate_t, w_up_t, w_down, dy, l1_coef: float,
                  dx, dw_gate_t, dw_up_t, dw_down, ws, stream=None):
    """Backward of the hybrid-format FFN with the L1 activation penalty (see include/twell.h)."""
    e = 2 if desc.dtype == "bf16" else 4
    dt = desc.torch_dtype
    need = _sizes(desc, route.max_dense_rows)["ws_bwd"]
    cr = _route(desc, route)
    wbytes = desc.d_ff * desc.d_model
    _check("twell_ffn_bwd", library().twell_ffn_bwd(
        ctypes.byref(_cdesc(desc)), _ptr(x, "x", desc.T * desc.d_model * e, dt), _act(desc, act), ctypes.byref(cr),
        _ptr(w_gate_t, "w_gate_t", wbytes * e, dt), _ptr(w_up_t, "w_up_t", wbytes * e, dt),
        _ptr(w_down, "w_down", wbytes * e, dt), _ptr(dy, "dy", desc.T * desc.d_model * e, dt),
        ctypes.c_float(l1_coef), _ptr(dx, "dx", desc.T * desc.d_model * e, dt),
        _ptr(dw_gate_t, "dw_gate_t", wbytes * 4, torch.float32), _ptr(dw_up_t, "dw_up_t", wbytes * 4, torch.float32),
        _ptr(dw_down, "dw_down", wbytes * 4, torch.float32), _ptr(ws, "ws", need),
        ctypes.c_size_t(ws.numel() * ws.element_size() if ws is not None else 0), _stream(stream)))


def twell_dense_ffn_fwd(desc: Desc, x, w_gate_t, w_up_t, w_down, y, ws, stream=None):
    """The library's dense MFMA FFN (gate|up GEMM with ReLU*u epilogue, then down)."""
    e = 2 if desc.dtype == "bf16" else 4
    dt = desc.torch_dtype
    need = _sizes(desc, 0)["ws_dense_fwd"]
    _check("twell_dense_ffn_fwd", library().twell_dense_ffn_fwd(
        ctypes.byref(_cdesc(desc)), _ptr(x, "x", desc.T * desc.d_model * e, dt),
        _ptr(w_gate_t, "w_gate_t", desc.d_ff * desc.d_model * e, dt),
        _ptr(w_up_t, "w_up_t", desc.d_ff * desc.d_model * e, dt),
        _ptr(w_down, "w_down", desc.d_ff * desc.d_model * e, dt),
        _ptr(y, "y", desc.T * desc.d_model * e, dt), _ptr(ws, "ws", need),
        ctypes.c_size_t(ws.numel() * ws.element_size() if ws is not None else 0), _stream(stream)))


# ----------------------------------------------------------------------------- serving a few tokens
# A call here takes a few microseconds of GPU time, so its host cost sets the
# pace: the C structs of a descriptor are kept on it, and the checks below are
# one condition each, with the reason worked out only when it fails.
ACTIVATIONS = {"relu": 0, "silu": 1}
_TORCH = {"bf16": torch.bfloat16, "fp32": torch.float32}
_CODE = {torch.bfloat16: TWELL_BF16, torch.float32: TWELL_FP32}
_CODE_DTYPE, _SCALE_DTYPE = torch.uint8, torch.bfloat16


def _c_ints(width: int, /, **numbers) -> dict:
    """The numbers as C takes them; ctypes alone would wrap the ones that do not fit."""
    for name, v in numbers.items():
        if not -(1 << (width - 1)) <= int(v) < 1 << (width - 1):
            raise ValueError(f"{name}: {v} does not fit {width} bits")
    return {name: int(v) for name, v in numbers.items()}


class _Keeping:
    """A descriptor that keeps C structs between calls: copies and pickles hold its fields alone."""

    def __reduce__(self):
        return type(self), tuple(getattr(self, f.name) for f in fields(self))


@dataclass(frozen=True)
class WDesc(_Keeping):
    """``experts`` matrices of ``rows`` outputs x ``cols`` inputs, held in 4 bits with a scale for every ``group``
    inputs of a row (32, 64 or 128), or in bf16 (``bits`` 16, ``group`` 0)."""
    experts: int
    rows: int
    cols: int
    bits: int
    group: int = 0

    @functools.cached_property
    def _ref(self):
        return ctypes.byref(CWDesc(**_c_ints(32, experts=self.experts, rows=self.rows, cols=self.cols, bits=self.bits,
                                             group=self.group)))

    @functools.cached_property
    def plane_bytes(self) -> tuple:
        """Bytes of the planes (codes, scales)."""
        out = CWSizes()
        _check("twell_weights_sizes", library().twell_weights_sizes(self._ref, ctypes.byref(out)))
        return int(out.codes), int(out.scales)


class Weights(NamedTuple):
    """The planes of laid-out weights as device tensors."""
    codes: torch.Tensor   # uint8
    scales: torch.Tensor  # bf16; empty for 16 bits


@dataclass(frozen=True)
class MoeDesc(_Keeping):
    """A mixture-of-experts layer for T tokens; ``bits`` and ``group`` are those of the experts' weights."""
    T: int
    d_model: int
    d_ff: int
    experts: int
    top_k: int
    dtype: str  # "fp32" | "bf16": x, the router's weights and y
    bits: int
    group: int = 0
    act: str = "silu"  # "relu" | "silu"
    renorm: bool = True

    @functools.cached_property
    def torch_dtype(self) -> torch.dtype:
        return _TORCH[self.dtype]

    @functools.cached_property
    def in_desc(self) -> WDesc:
        """Of the gate and the up projections: d_model -> d_ff."""
        return WDesc(self.experts, self.d_ff, self.d_model, self.bits, self.group)

    @functools.cached_property
    def out_desc(self) -> WDesc:
        """Of the down projections: d_ff -> d_model."""
        return WDesc(self.experts, self.d_model, self.d_ff, self.bits, self.group)

    def _strided(self, ldx: int, ldy: int):
        if self.act not in ACTIVATIONS or self.dtype not in _TORCH:
            raise ValueError(f"act {self.act!r}, dtype {self.dtype!r}: expected one of {tuple(ACTIVATIONS)} and "
                             f"{tuple(_TORCH)}")
        return ctypes.byref(CMoeDesc(
            **_c_ints(64, T=self.T, ldx=ldx, ldy=ldy),
            **_c_ints(32, d_model=self.d_model, d_ff=self.d_ff, experts=self.experts, top_k=self.top_k, bits=self.bits,
                      group=self.group),
            dtype=_CODE[self.torch_dtype], act=ACTIVATIONS[self.act], renorm=int(bool(self.renorm))))

    @functools.cached_property
    def _ref(self):  # contiguous rows
        return self._strided(self.d_model, self.d_model)

    @functools.cached_property
    def _call(self) -> tuple:
        """What every call asks for: bytes of the router, the choices and the workspace among it."""
        return (self.torch_dtype, self.T, self.d_model, self._ref, self.in_desc, self.out_desc,
                self.experts * self.d_model * self.torch_dtype.itemsize, self.T * self.top_k * 4, self.ws_bytes)

    @functools.cached_property
    def ws_bytes(self) -> int:
        """Bytes of twell_moe_fwd's workspace."""
        out = ctypes.c_size_t()
        _check("twell_moe_sizes", library().twell_moe_sizes(self._ref, ctypes.byref(out)))
        return int(out.value)


class MoeWeights(NamedTuple):
    gate: Weights
    up: Weights
    down: Weights


class MoeOut(NamedTuple):
    y: torch.Tensor        # dtype [T, d_model]
    ids: torch.Tensor      # int32 [T, top_k]: the chosen experts, best first
    weights: torch.Tensor  # fp32 [T, top_k]


def _weights_sizes(desc: WDesc) -> tuple:
    return desc.plane_bytes


def moe_ws_bytes(desc: MoeDesc) -> int:
    return desc.ws_bytes


def alloc_weights(desc: WDesc, device="cuda") -> Weights:
    codes, scales = desc.plane_bytes
    return Weights(torch.empty(codes, dtype=_CODE_DTYPE, device=device),
                   torch.empty(scales // 2, dtype=_SCALE_DTYPE, device=device))


def alloc_moe_weights(desc: MoeDesc, device="cuda") -> MoeWeights:
    return MoeWeights(alloc_weights(desc.in_desc, device), alloc_weights(desc.in_desc, device),
                      alloc_weights(desc.out_desc, device))


def alloc_moe_out(desc: MoeDesc, device="cuda") -> MoeOut:
    return MoeOut(torch.empty((desc.T, desc.d_model), dtype=desc.torch_dtype, device=device),
                  torch.empty((desc.T, desc.top_k), dtype=torch.int32, device=device),
                  torch.empty((desc.T, desc.top_k), dtype=torch.float32, device=device))


def alloc_moe_ws(desc: MoeDesc, device="cuda") -> torch.Tensor:
    return torch.empty(desc.ws_bytes, dtype=torch.uint8, device=device)


def _device(t, name: str) -> int:
    """The GPU that all tensors of a call are on, told by one of them."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name}: must be a GPU tensor (got {t.device})")
    return dev


def _fit(t, name: str, nbytes: int, dtype: torch.dtype, dev: int) -> int:
    """Pointer of a contiguous tensor of the dtype with at least nbytes on GPU dev."""
    if (isinstance(t, torch.Tensor) and t.get_device() == dev and t.dtype is dtype and t.nbytes >= nbytes
            and t.is_contiguous()):
        return t.data_ptr()
    if t is None:
        raise TypeError(f"{name}: expected a torch.Tensor")
    _ptr(t, name, nbytes, dtype)  # says what is wrong
    raise ValueError(f"{name}: on cuda:{t.get_device()}, expected cuda:{dev}")


def _shaped(t, name: str, shape: tuple) -> None:
    """Refuses a tensor that holds something else than ``shape``: another number of elements, or other axes behind the
    first.  A flat one says nothing of axes, and leading axes of 1 may be left out."""
    if not isinstance(t, torch.Tensor) or t.shape == shape:
        return
    inner = shape[1:]
    if t.numel() != math.prod(shape) or (inner and t.dim() > 1 and t.shape[-len(inner):] != inner):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {shape}")


def _planes(desc: WDesc, w: Weights, name: str, dev: int) -> CPlanes:
    codes, scales = desc.plane_bytes
    c, s = w.codes, w.scales
    if (scales and isinstance(c, torch.Tensor) and c.get_device() == dev and c.dtype is _CODE_DTYPE
            and c.nbytes >= codes and c.is_contiguous() and isinstance(s, torch.Tensor) and s.get_device() == dev
            and s.dtype is _SCALE_DTYPE and s.nbytes >= scales and s.is_contiguous()):  # _fit of both, no calls
        return CPlanes(c.data_ptr(), s.data_ptr())
    return CPlanes(_fit(w.codes, name + ".codes", codes, _CODE_DTYPE, dev),
                   _fit(w.scales, name + ".scales", scales, _SCALE_DTYPE, dev) if scales else 0)


def _rows(t: torch.Tensor, name: str, n: int, width: int, dtype: torch.dtype, dev: int) -> tuple:
    """Pointer and row stride of n rows of ``width`` elements on GPU dev, each row contiguous."""
    if (isinstance(t, torch.Tensor) and t.get_device() == dev and t.dtype is dtype and t.is_contiguous()
            and t.shape == (n, width)):
        return t.data_ptr(), width
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a GPU tensor (got {t.device})")
    if t.get_device() != dev:
        raise ValueError(f"{name}: on cuda:{t.get_device()}, expected cuda:{dev}")
    if t.dtype is not dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.shape != (n, width):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {(n, width)}")
    s0, s1 = t.stride()
    if width > 1 and s1 != 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    if n > 1 and s0 < width:
        raise ValueError(f"{name}: rows overlap (stride {s0} for {width} elements)")
    return t.data_ptr(), s0 if n > 1 else width


# The handle alone: building a Stream object costs more than the other checks of a call together.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


@functools.lru_cache(maxsize=None)
def _device_count() -> int:
    return torch.cuda.device_count()


_current_device = torch.cuda.current_device


def _current_is(dev: int) -> None:
    """Every GPU has a default stream of handle 0, which to a launch means the current GPU's: the tensors have to be
    there."""
    if dev != _current_device():
        raise ValueError(f"tensors on cuda:{dev}, default stream of the current device, cuda:{_current_device()}")


def _stream_on(dev: int, stream) -> int:
    """The stream's handle; by default the current one of GPU dev."""
    handle = _raw_stream(dev) if stream is None else _stream(stream)
    if not handle and _device_count() > 1:
        _current_is(dev)
    return handle


def _any_dtype(t, name: str) -> int:
    code = _CODE.get(t.dtype) if isinstance(t, torch.Tensor) else None
    if code is None:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}: expected a torch.Tensor")
        raise ValueError(f"{name}: dtype {t.dtype}, expected torch.bfloat16 or torch.float32")
    return code


def twell_weights_pack(desc: WDesc, w, planes: Weights, transposed: bool = False, stream=None):
    """Lay out w [experts, rows, cols] ([experts, cols, rows] if transposed; bf16, or fp32 for 4 bits) into planes.
    A flat w is taken in that order; any other shape is refused."""
    code = _any_dtype(w, "w")
    dev = _device(w, "w")
    _shaped(w, "w", (desc.experts, desc.cols, desc.rows) if transposed else (desc.experts, desc.rows, desc.cols))
    n = desc.experts * desc.rows * desc.cols * w.element_size()
    st = library().twell_weights_pack(desc._ref, _fit(w, "w", n, w.dtype, dev), code, 1 if transposed else 0,
                                      _planes(desc, planes, "planes", dev), _stream_on(dev, stream))
    if st:
        _check("twell_weights_pack", st)


def twell_weights_unpack(desc: WDesc, planes: Weights, w, stream=None):
    """Write the values that planes stand for to w [experts, rows, cols] (bf16, or fp32 for 4 bits; flat will do)."""
    code = _any_dtype(w, "w")
    dev = _device(w, "w")
    _shaped(w, "w", (desc.experts, desc.rows, desc.cols))
    n = desc.experts * desc.rows * desc.cols * w.element_size()
    st = library().twell_weights_unpack(desc._ref, _planes(desc, planes, "planes", dev),
                                        _fit(w, "w", n, w.dtype, dev), code, _stream_on(dev, stream))
    if st:
        _check("twell_weights_unpack", st)


def twell_linear_fwd(desc: WDesc, planes: Weights, x, y, stream=None):
    """y [T, rows] = x [T, cols] times one matrix of 4-bit weights; x and y in bf16 or fp32, rows may be strided."""
    code = _any_dtype(x, "x")
    shape, dtype = x.shape, x.dtype
    if len(shape) != 2:
        raise ValueError(f"x: shape {tuple(shape)}, expected {('T', desc.cols)}")
    T, dev = shape[0], x.get_device()
    if dev < 0:
        _device(x, "x")
    px, ldx = _rows(x, "x", T, desc.cols, dtype, dev)
    py, ldy = _rows(y, "y", T, desc.rows, dtype, dev)
    handle = _raw_stream(dev) if stream is None else _stream(stream)  # _stream_on without the call
    if not handle and _device_count() > 1:
        _current_is(dev)
    st = library().twell_linear_fwd(desc._ref, _planes(desc, planes, "planes", dev), T, code, px, ldx, py, ldy,
                                    handle)
    if st:
        _check("twell_linear_fwd", st)


def twell_moe_fwd(desc: MoeDesc, x, w_router, weights: MoeWeights, out: MoeOut, ws, router_bias=None, stream=None):
    """Router, chosen experts and their weighted sum for desc.T tokens (see include/twell.h).  x and out.y may have
    strided rows; ws holds moe_ws_bytes(desc) bytes."""
    dt, T, d, ref, din, dout, router, pairs, need = desc._call
    dev = _device(x, "x")
    px, ldx = _rows(x, "x", T, d, dt, dev)
    y, ids, wts = out
    py, ldy = _rows(y, "out.y", T, d, dt, dev)
    gate, up, down = weights
    _shaped(w_router, "w_router", (desc.experts, d))
    if router_bias is not None:
        _shaped(router_bias, "router_bias", (desc.experts,))
    st = library().twell_moe_fwd(
        ref if ldx == d and ldy == d else desc._strided(ldx, ldy), px, _fit(w_router, "w_router", router, dt, dev),
        _fit(router_bias, "router_bias", desc.experts * 4, torch.float32, dev) if router_bias is not None else None,
        _planes(din, gate, "gate", dev), _planes(din, up, "up", dev), _planes(dout, down, "down", dev), py,
        _fit(ids, "out.ids", pairs, torch.int32, dev), _fit(wts, "out.weights", pairs, torch.float32, dev),
        _fit(ws, "ws", need, torch.uint8, dev), need, _stream_on(dev, stream))
    if st:
        _check("twell_moe_fwd", st)
