"""CPU tests of the many-token entry points: sizes, and bad arguments mapped to status codes or exceptions before any
HIP call."""
import copy
import ctypes
import os
import pickle

import pytest
import torch

from activation_sparse_feedforward_amd import twell as T
from test_few_token_abi import _On

pytestmark = pytest.mark.skipif(not os.path.exists(T.LIB_PATH), reason="libtwell.so not built")

P = 0x10000
OK, INVAL, UNSUP = T.TWELL_OK, T.TWELL_EINVAL, T.TWELL_EUNSUPPORTED


def _tok(**kw):
    base = dict(T=4, ld_tokens=64, ld_rows=64, d_model=64, experts=8, top_k=2, dtype=T.TWELL_BF16)
    base.update(kw)
    return T.CTokensDesc(**base)


@pytest.mark.parametrize("kw,code", [
    ({}, OK), ({"T": 0}, OK), ({"d_model": 1}, OK), ({"top_k": 32, "experts": 2}, OK), ({"dtype": T.TWELL_FP32}, OK),
    ({"T": 1 << 20}, OK), ({"experts": 1024}, OK),
    ({"T": -1}, INVAL), ({"d_model": 0}, INVAL), ({"experts": 0}, INVAL), ({"top_k": 0}, INVAL), ({"dtype": 2}, INVAL),
    ({"ld_tokens": 63}, INVAL), ({"ld_rows": 63}, INVAL), ({"d_model": 65}, INVAL),
    ({"T": (1 << 20) + 1}, UNSUP), ({"experts": 1025}, UNSUP), ({"top_k": 33}, UNSUP),
    ({"ld_tokens": (1 << 40) + 1}, UNSUP), ({"ld_rows": (1 << 40) + 1}, UNSUP),
    ({"T": 1 << 20, "d_model": (1 << 13) + 1, "ld_tokens": 1 << 14, "ld_rows": 1 << 14}, UNSUP),
])
def test_tokens_descriptor(kw, code):
    n = ctypes.c_size_t()
    d = ctypes.byref(_tok(**kw))
    assert T.library().twell_tokens_sizes(d, ctypes.byref(n)) == code
    assert T.library().twell_tokens_sizes(d, None) != OK
    lib = T.library()
    calls = (lib.twell_tokens_sort(d, None, None, None, None, 0, None), lib.twell_tokens_gather(d, None, None, None, None),
             lib.twell_tokens_combine(d, None, None, None, None, None),
             lib.twell_tokens_combine_bwd(d, None, None, None, None, P, 64, P, None))
    if code != OK:
        assert set(calls) == {code}


def test_tokens_refuse():
    lib, d = T.library(), ctypes.byref(_tok())
    n = ctypes.c_size_t()
    assert lib.twell_tokens_sizes(d, ctypes.byref(n)) == OK

    def sort(ids=P, off=P, pr=P, ws=P, size=n.value):
        return lib.twell_tokens_sort(d, ids, off, pr, ws, size, None)

    for kw in (dict(ids=None), dict(off=None), dict(pr=None), dict(ws=None), dict(ids=P + 2), dict(off=P + 2),
               dict(pr=P + 2), dict(ws=P + 8), dict(size=n.value - 1)):
        assert sort(**kw) == INVAL, kw
    for x, pr, rows in ((None, P, P), (P, None, P), (P, P, None), (P + 1, P, P), (P, P + 2, P), (P, P, P + 1)):
        assert lib.twell_tokens_gather(d, x, pr, rows, None) == INVAL
        assert lib.twell_tokens_combine(d, x, pr, None, rows, None) == INVAL
        assert lib.twell_tokens_combine_bwd(d, x, pr, P, rows, None, 64, P, None) == INVAL
    assert lib.twell_tokens_combine(d, P, P, P + 2, P, None) == INVAL
    for w, dr, ld, dw in ((None, P, 64, P), (P + 2, P, 64, P), (P, P + 1, 64, P), (P, P, 63, P), (P, P, 64, P + 2)):
        assert lib.twell_tokens_combine_bwd(d, P, P, w, P, dr, ld, dw, None) == INVAL
    assert lib.twell_tokens_combine_bwd(d, P, P, P, P, P, (1 << 40) + 1, P, None) == UNSUP
    assert lib.twell_tokens_combine_bwd(d, P, P, P, P, None, 0, None, None) == OK  # nothing is asked for
    e = ctypes.byref(_tok(T=0))
    assert lib.twell_tokens_gather(e, None, None, None, None) == OK
    assert lib.twell_tokens_combine(e, None, None, None, None, None) == OK
    assert lib.twell_tokens_combine_bwd(e, None, None, None, None, P, 64, P, None) == OK


def test_tokens_workspace_stops_growing():
    sizes = [T.TokensDesc(t, 64, 100, 4, "bf16").ws_bytes for t in (0, 1, 1 << 18, 1 << 20)]
    assert 400 <= sizes[0] == sizes[1] and sizes[2] == sizes[3] <= 256 * 400 + 256


def _norm(**kw):
    base = dict(T=4, ldx=64, ldy=64, lddx=64, d_model=64, dtype=T.TWELL_BF16, w_dtype=T.TWELL_FP32, eps=1e-5)
    base.update(kw)
    return T.CNormDesc(**base)


@pytest.mark.parametrize("kw,code", [
    ({}, OK), ({"T": 0}, OK), ({"d_model": 1}, OK), ({"w_dtype": T.TWELL_BF16}, OK), ({"eps": 0.0}, OK),
    ({"d_model": 16384, "ldx": 16384, "ldy": 16384, "lddx": 16384}, OK),
    ({"T": -1}, INVAL), ({"d_model": 0}, INVAL), ({"dtype": 2}, INVAL), ({"w_dtype": 2}, INVAL), ({"eps": -1e-5}, INVAL),
    ({"eps": float("nan")}, INVAL), ({"eps": float("inf")}, INVAL), ({"ldx": 63}, INVAL), ({"ldy": 63}, INVAL),
    ({"lddx": 63}, INVAL),
    ({"d_model": 16385, "ldx": 16385, "ldy": 16385, "lddx": 16385}, UNSUP), ({"T": (1 << 20) + 1}, UNSUP),
    ({"ldx": (1 << 40) + 1}, UNSUP), ({"ldy": (1 << 40) + 1}, UNSUP), ({"lddx": (1 << 40) + 1}, UNSUP),
])
def test_norm_descriptor(kw, code):
    n, d, lib = ctypes.c_size_t(), ctypes.byref(_norm(**kw)), T.library()
    assert lib.twell_layernorm_sizes(d, ctypes.byref(n)) == code
    assert lib.twell_layernorm_sizes(d, None) != OK
    if code != OK:
        assert lib.twell_layernorm_fwd(d, P, P, P, P, P, None) == code
        assert lib.twell_layernorm_bwd(d, P, P, P, P, P, P, P, P, 1 << 30, None) == code


def test_norm_refuses():
    lib, d = T.library(), ctypes.byref(_norm())
    n = ctypes.c_size_t()
    assert lib.twell_layernorm_sizes(d, ctypes.byref(n)) == OK
    for a in ((None, P, P, P, P), (P, P, P, None, P), (P + 1, P, P, P, P), (P, P + 2, P, P, P), (P, P, P + 2, P, P),
              (P, P, P, P + 1, P), (P, P, P, P, P + 2)):
        assert lib.twell_layernorm_fwd(d, *a, None) == INVAL, a

    def bwd(x=P, w=P, stats=P, dy=P, dx=P, dw=P, db=P, ws=P, size=n.value):
        return lib.twell_layernorm_bwd(d, x, w, stats, dy, dx, dw, db, ws, size, None)

    for kw in (dict(x=None), dict(stats=None), dict(dy=None), dict(dx=None), dict(ws=None), dict(x=P + 1), dict(w=P + 2),
               dict(stats=P + 2), dict(dy=P + 1), dict(dx=P + 1), dict(dw=P + 2), dict(db=P + 2), dict(ws=P + 8),
               dict(size=n.value - 1)):
        assert bwd(**kw) == INVAL, kw
    e = ctypes.byref(_norm(T=0))
    assert lib.twell_layernorm_fwd(e, None, None, None, None, None, None) == OK
    assert lib.twell_layernorm_bwd(e, None, None, None, None, None, None, None, None, 0, None) == OK


def _tokens_args(dev=0, T_=0, k=2, d=64, E=8):
    on = lambda *s, dtype=torch.bfloat16: _On.make(dev, *s, dtype=dtype)  # noqa: E731
    i32, f32 = torch.int32, torch.float32
    return dict(ids=on(T_, k, dtype=i32), offsets=on(E + 1, dtype=i32), pair_row=on(T_, k, dtype=i32), x=on(T_, d),
                rows=on(T_ * k, d), y=on(T_, d), weights=on(T_, k, dtype=f32), dy=on(T_, d), drows=on(T_ * k, d),
                dweights=on(T_, k, dtype=f32))


def _tokens_calls(desc, a):
    o = T.TokensOrder(a["offsets"], a["pair_row"])
    return {
        "gather": (lambda: T.twell_tokens_gather(desc, a["x"], o, a["rows"], stream=0), "x pair_row rows"),
        "combine": (lambda: T.twell_tokens_combine(desc, a["rows"], o, a["weights"], a["y"], stream=0),
                    "rows pair_row weights y"),
        "combine_bwd": (lambda: T.twell_tokens_combine_bwd(desc, a["rows"], o, a["weights"], a["dy"], a["drows"],
                                                           a["dweights"], stream=0),
                        "rows pair_row weights dy drows dweights"),
    }


def test_tokens_binding_refuses_what_does_not_fit(monkeypatch):
    monkeypatch.setattr(T, "_device_count", lambda: 2)
    monkeypatch.setattr(T, "_current_device", lambda: 0)
    desc = T.TokensDesc(0, 64, 8, 2, "bf16")
    good = _tokens_args()
    for name, (call, _) in _tokens_calls(desc, good).items():
        call()
    for name in ("gather", "combine", "combine_bwd"):
        for arg in _tokens_calls(desc, good)[name][1].split():
            shape, dtype = tuple(good[arg].shape), good[arg].dtype
            other = torch.float32 if dtype != torch.float32 else torch.bfloat16
            for bad in (_On.make(1, *shape, dtype=dtype), _On.make(0, *shape, dtype=other),
                        _On.make(0, shape[0] + 1, shape[1], dtype=dtype), _On.make(0, shape[0], shape[1] + 1, dtype=dtype)):
                with pytest.raises(ValueError):
                    _tokens_calls(desc, {**good, arg: bad})[name][0]()
    with pytest.raises(ValueError, match="GPU"):
        T.twell_tokens_gather(desc, torch.zeros(0, 64).bfloat16(), T.alloc_tokens_order(desc, "cpu"), good["rows"])
    with pytest.raises(TypeError):
        T.twell_tokens_combine_bwd(desc, None, T.TokensOrder(good["offsets"], good["pair_row"]), good["weights"],
                                   good["dy"], good["drows"], good["dweights"], stream=0)
    for arg, bad in (("ids", _On.make(0, 0, 3, dtype=torch.int32)), ("offsets", _On.make(0, 8, dtype=torch.int32)),
                     ("pair_row", _On.make(0, 1, 2, dtype=torch.int32)), ("ids", _On.make(0, 0, 2, dtype=torch.int64)),
                     ("ids", _On.make(1, 0, 2, dtype=torch.int32))):
        a = {**good, arg: bad}
        with pytest.raises(ValueError):
            T.twell_tokens_sort(desc, a["ids"], T.TokensOrder(a["offsets"], a["pair_row"]),
                                _On.make(0, desc.ws_bytes, dtype=torch.uint8), stream=0)
    with pytest.raises(ValueError, match="ws"):
        T.twell_tokens_sort(desc, good["ids"], T.TokensOrder(good["offsets"], good["pair_row"]),
                            _On.make(0, desc.ws_bytes - 1, dtype=torch.uint8), stream=0)


def test_norm_binding_refuses_what_does_not_fit(monkeypatch):
    monkeypatch.setattr(T, "_device_count", lambda: 2)
    monkeypatch.setattr(T, "_current_device", lambda: 0)
    desc = T.NormDesc(0, 64, "bf16")
    f32 = torch.float32
    good = dict(x=_On.make(0, 0, 64), w=_On.make(0, 64, dtype=f32), b=_On.make(0, 64, dtype=f32), y=_On.make(0, 0, 64),
                stats=_On.make(0, 0, 2, dtype=f32))

    def fwd(**kw):
        a = {**good, **kw}
        T.twell_layernorm_fwd(desc, a["x"], a["w"], a["b"], a["y"], a["stats"], stream=0)

    fwd()
    fwd(w=None)
    fwd(b=None)
    fwd(w=None, b=None, stats=None)
    fwd(w=_On.make(0, 64), b=_On.make(0, 64))
    for bad in (dict(x=_On.make(0, 1, 64)), dict(x=_On.make(0, 0, 65)), dict(y=_On.make(0, 0, 63)),
                dict(y=_On.make(0, 0, 64, dtype=f32)), dict(w=_On.make(0, 63, dtype=f32)), dict(b=_On.make(0, 64)),
                dict(w=_On.make(0, 64, dtype=torch.float64)), dict(stats=_On.make(0, 0, 1, dtype=f32)),
                *({k: _On.make(1, *v.shape, dtype=v.dtype)} for k, v in good.items())):
        with pytest.raises(ValueError):
            fwd(**bad)
    with pytest.raises(TypeError):
        fwd(x=None)
    with pytest.raises(TypeError):
        fwd(y=None)


def _f8(**kw):
    return T.CFp8Desc(**{**dict(experts=2, rows=64, cols=128), **kw})


@pytest.mark.parametrize("kw,code", [
    ({}, OK), ({"rows": 1, "cols": 1}, OK), ({"experts": 1024}, OK), ({"rows": 1 << 20, "cols": 1 << 14}, OK),
    ({"experts": 0}, INVAL), ({"rows": 0}, INVAL), ({"cols": -1}, INVAL),
    ({"experts": 1025}, UNSUP), ({"rows": (1 << 20) + 1}, UNSUP), ({"cols": (1 << 20) + 1}, UNSUP),
    ({"rows": 1 << 20, "cols": (1 << 14) + 1}, UNSUP),
])
def test_fp8_descriptor(kw, code):
    lib, d, n, a, b = T.library(), ctypes.byref(_f8(**kw)), T.CWSizes(), ctypes.c_size_t(), ctypes.c_size_t()
    assert lib.twell_fp8_weights_sizes(d, ctypes.byref(n)) == code
    assert lib.twell_fp8_weights_sizes(d, None) != OK
    assert lib.twell_fp8_linear_sizes(d, 5, ctypes.byref(a), ctypes.byref(b)) == code
    if code != OK:
        pl = T.CPlanes(P, P)
        assert lib.twell_fp8_weights_pack(d, P, T.TWELL_BF16, pl, None, None) == code
        assert lib.twell_fp8_weights_unpack(d, pl, P, T.TWELL_BF16, None) == code
        assert lib.twell_fp8_linear_fwd(d, pl, 1, P, T.TWELL_BF16, P, 1 << 30, P, 1 << 30, P, 1 << 40, None) == code
        assert lib.twell_fp8_linear_bwd(d, pl, 1, P, T.TWELL_BF16, P, 1 << 30, P, 1 << 30, P, 1 << 30, P, P, 1 << 40,
                                        None) == code


def test_fp8_sizes():
    for rows, cols in ((16, 128), (17, 129), (1, 1), (1001, 707), (64, 1024)):
        tiles, blocks = -(-rows // 16), -(-cols // 128)
        assert T.Fp8Desc(3, rows, cols).plane_bytes == (3 * tiles * blocks * 2048, 3 * tiles * -(-blocks // 4) * 64)
        assert T.Fp8Desc(3, rows, cols).transposed == T.Fp8Desc(3, cols, rows)
    lib, a, b = T.library(), ctypes.c_size_t(), ctypes.c_size_t()
    d = ctypes.byref(_f8())
    assert lib.twell_fp8_linear_sizes(d, -1, ctypes.byref(a), ctypes.byref(b)) == INVAL
    assert lib.twell_fp8_linear_sizes(d, 1, None, ctypes.byref(b)) == INVAL
    assert lib.twell_fp8_linear_sizes(d, 1, ctypes.byref(a), None) == INVAL
    assert lib.twell_fp8_linear_sizes(d, (1 << 20) + 1, ctypes.byref(a), ctypes.byref(b)) == UNSUP
    # rows of 128 and of 64 inputs: one block each, up to a tile more for each expert
    assert T.fp8_ws_bytes(T.Fp8Desc(2, 64, 128), 100) >= 8 * (2048 + 64)


def test_fp8_pack_and_unpack_refuse():
    lib, d, pl, bf = T.library(), ctypes.byref(_f8()), T.CPlanes(P, P), T.TWELL_BF16
    for f in (lambda w, t, pl: lib.twell_fp8_weights_pack(d, w, t, pl, None, None),
              lambda w, t, pl: lib.twell_fp8_weights_unpack(d, pl, w, t, None)):
        for w, t, p in ((None, bf, pl), (P + 1, bf, pl), (P + 2, T.TWELL_FP32, pl), (P, 2, pl),
                        (P, bf, T.CPlanes(0, P)), (P, bf, T.CPlanes(P, 0)), (P, bf, T.CPlanes(P + 8, P)),
                        (P, bf, T.CPlanes(P, P + 4))):
            assert f(w, t, p) == INVAL
    for t in (T.CPlanes(0, P), T.CPlanes(P, 0), T.CPlanes(P + 8, P)):
        assert lib.twell_fp8_weights_pack(d, P, bf, pl, ctypes.byref(t), None) == INVAL


def test_fp8_linear_refuses():
    lib, d = T.library(), _f8()
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    assert lib.twell_fp8_linear_sizes(ctypes.byref(d), 10, ctypes.byref(a), ctypes.byref(b)) == OK
    good = dict(d=ctypes.byref(d), p=T.CPlanes(P, P), T_=10, off=P, t=T.TWELL_BF16, x=P, ldx=128, y=P, ldy=64, dx=P,
                lddx=128, dw=P, ws=P, n=max(a.value, b.value))

    def fwd(**kw):
        g = {**good, **kw}
        return lib.twell_fp8_linear_fwd(g["d"], g["p"], g["T_"], g["off"], g["t"], g["x"], g["ldx"], g["y"], g["ldy"],
                                        g["ws"], g["n"], None)

    def bwd(**kw):
        g = {**good, **kw}
        return lib.twell_fp8_linear_bwd(g["d"], g["p"], g["T_"], g["off"], g["t"], g["x"], g["ldx"], g["y"], g["ldy"],
                                        g["dx"], g["lddx"], g["dw"], g["ws"], g["n"], None)

    both = [dict(d=None), dict(T_=-1), dict(off=None), dict(off=P + 2), dict(t=2), dict(x=None), dict(x=P + 1),
            dict(y=None), dict(y=P + 1), dict(ldx=127), dict(ldy=63), dict(p=T.CPlanes(0, P)), dict(p=T.CPlanes(P, 0)),
            dict(p=T.CPlanes(P + 8, P)), dict(ws=None), dict(ws=P + 8), dict(n=100)]
    for kw in both:
        assert fwd(**kw) == INVAL, kw
        assert bwd(**kw) == INVAL, kw
    for kw in (dict(dx=P + 1), dict(lddx=127), dict(dw=P + 2)):
        assert bwd(**kw) == INVAL, kw
    for kw in (dict(T_=(1 << 20) + 1), dict(ldx=(1 << 40) + 1), dict(ldy=(1 << 40) + 1)):
        assert fwd(**kw) == UNSUP and bwd(**kw) == UNSUP, kw
    assert bwd(lddx=(1 << 40) + 1) == UNSUP
    wide = ctypes.byref(_f8(rows=1 << 18))
    assert fwd(d=wide, ldy=1 << 18, T_=(1 << 19) + 1, n=1 << 50) == UNSUP
    assert fwd(T_=0, x=None, y=None, p=T.CPlanes(0, 0), ws=None, n=0) == OK
    assert bwd(T_=0, x=None, y=None, p=T.CPlanes(0, 0), ws=None, n=0, dx=None, dw=None) == OK
    assert bwd(dx=None, dw=None, x=None, y=None, p=T.CPlanes(0, 0), ws=None, n=0) == OK  # nothing is asked for


def _f8_planes(desc, dev=0, short=0):
    codes, scales = desc.plane_bytes
    return T.Weights(_On.make(dev, codes - short, dtype=torch.uint8), _On.make(dev, scales, dtype=torch.uint8))


def test_fp8_binding_refuses_what_does_not_fit(monkeypatch):
    monkeypatch.setattr(T, "_device_count", lambda: 2)
    monkeypatch.setattr(T, "_current_device", lambda: 0)
    desc, u8, f32 = T.Fp8Desc(2, 64, 128), torch.uint8, torch.float32
    on = _On.make
    good = dict(p=_f8_planes(desc), t=_f8_planes(desc.transposed), x=on(0, 0, 128), y=on(0, 0, 64), dx=on(0, 0, 128),
                ws=on(0, 1 << 16, dtype=u8), off=on(0, 3, dtype=torch.int32))

    def fwd(**kw):
        g = {**good, **kw}
        T.twell_fp8_linear_fwd(desc, g["p"], g["x"], g["y"], g["ws"], offsets=g["off"], stream=0)

    def bwd(dw=None, **kw):
        g = {**good, **kw}
        T.twell_fp8_linear_bwd(desc, g["t"], g["x"], g["y"], g["dx"], dw, g["ws"], offsets=g["off"], stream=0)

    fwd()
    bwd()
    bwd(x=None)
    for kw in (dict(x=on(0, 0, 127)), dict(x=on(0, 128)), dict(x=on(0, 0, 128, dtype=torch.float16)),
               dict(x=on(1, 0, 128)), dict(y=on(0, 0, 65)), dict(y=on(0, 1, 64)), dict(y=on(0, 0, 64, dtype=f32)),
               dict(y=on(1, 0, 64)), dict(ws=on(0, 10, dtype=u8)), dict(ws=on(1, 1 << 16, dtype=u8)), dict(off=None),
               dict(off=on(0, 2, dtype=torch.int32)), dict(off=on(0, 3, dtype=torch.int64)),
               dict(off=on(1, 3, dtype=torch.int32))):
        with pytest.raises(ValueError):
            fwd(**kw)
        if kw.get("x") is None or kw["x"].shape != (128,):
            with pytest.raises(ValueError):
                bwd(**kw)
    for p in (_f8_planes(desc, short=1), _f8_planes(desc, dev=1)):
        with pytest.raises(ValueError):
            fwd(p=p)
    for kw in (dict(dx=on(0, 0, 127)), dict(dx=on(0, 0, 128, dtype=f32)), dict(dx=on(1, 0, 128)),
               dict(t=_f8_planes(desc.transposed, short=1)), dict(dw=on(0, 2, 128, 64, dtype=f32)), dict(dw=on(0, 2, 64, 128)),
               dict(dw=on(1, 2, 64, 128, dtype=f32))):
        with pytest.raises(ValueError):
            bwd(**kw)
    for kw in (dict(x=None, dw=on(0, 2, 64, 128, dtype=f32)), dict(t=None), dict(ws=None)):
        with pytest.raises(TypeError):
            bwd(**kw)
    with pytest.raises(ValueError, match="shape"):
        T.twell_fp8_weights_pack(desc, on(0, 2, 128, 64), good["p"], stream=0)
    with pytest.raises(ValueError):
        T.twell_fp8_weights_pack(desc, on(0, 2, 64, 128), good["p"], _f8_planes(desc.transposed, dev=1), stream=0)
    with pytest.raises(ValueError):
        T.twell_fp8_weights_pack(desc, on(0, 2, 64, 128), _f8_planes(desc, short=1), stream=0)
    with pytest.raises(ValueError):
        T.twell_fp8_weights_unpack(desc, good["p"], on(0, 2, 64, 128, dtype=torch.float16), stream=0)


@pytest.mark.parametrize("make", [lambda d: T.TokensDesc(1, 64, 8, 2, d).ws_bytes, lambda d: T.NormDesc(1, 64, d).ws_bytes])
def test_unknown_dtypes_are_refused(make):
    make("fp32")
    with pytest.raises(ValueError, match="dtype"):
        make("fp16")


def test_numbers_beyond_c_integers_do_not_wrap():
    for kw in (dict(d_model=64 + (1 << 32)), dict(experts=8 + (1 << 32)), dict(top_k=2 + (1 << 32))):
        with pytest.raises(ValueError, match="32 bits"):
            T.TokensDesc(**{**dict(T=1, d_model=64, experts=8, top_k=2, dtype="bf16"), **kw}).ws_bytes
    with pytest.raises(ValueError, match="64 bits"):
        T.TokensDesc(1 << 64, 64, 8, 2, "bf16").ws_bytes
    with pytest.raises(ValueError, match="32 bits"):
        T.NormDesc(1, 64 + (1 << 32), "bf16").ws_bytes
    with pytest.raises(T.TwellError):
        T.NormDesc(1, 64, "bf16", float("nan")).ws_bytes
    for big in (1 << 32, -(1 << 32)):
        for make in (lambda: T.Fp8Desc(1 + big, 64, 64), lambda: T.Fp8Desc(1, 64 + big, 64), lambda: T.Fp8Desc(1, 64, 64 + big)):
            with pytest.raises(ValueError, match="32 bits"):
                make().plane_bytes
    with pytest.raises(ValueError, match="64 bits"):
        T.fp8_ws_bytes(T.Fp8Desc(1, 64, 64), 1 << 64)


@pytest.mark.parametrize("desc", [T.TokensDesc(3, 64, 8, 2, "bf16"), T.NormDesc(3, 64, "fp32", 1e-6), T.Fp8Desc(2, 64, 32)])
def test_descriptors_are_copied_and_pickled_after_use(desc):
    if isinstance(desc, T.Fp8Desc):
        used, name = desc.plane_bytes, "plane_bytes"
        desc.transposed
    else:
        used, name = desc.ws_bytes, "ws_bytes"
    for again in (copy.copy(desc), copy.deepcopy(desc), pickle.loads(pickle.dumps(desc))):
        assert again == desc and hash(again) == hash(desc) and getattr(again, name) == used
