"""CPU tests of the many-token entry points: sizes, and bad arguments mapped to status codes or exceptions before any
HIP call."""
import copy
import ctypes
import pickle

import os

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


@pytest.mark.parametrize("desc", [T.TokensDesc(3, 64, 8, 2, "bf16"), T.NormDesc(3, 64, "fp32", 1e-6)])
def test_descriptors_are_copied_and_pickled_after_use(desc):
    used = desc.ws_bytes
    for again in (copy.copy(desc), copy.deepcopy(desc), pickle.loads(pickle.dumps(desc))):
        assert again == desc and hash(again) == hash(desc) and again.ws_bytes == used
