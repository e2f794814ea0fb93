"""CPU tests of the few-token entry points: sizes, and bad arguments mapped to
status codes before any HIP call."""
import copy
import ctypes
import dataclasses
import os
import pickle

import pytest
import torch

from activation_sparse_feedforward_amd import twell as T

pytestmark = pytest.mark.skipif(not os.path.exists(T.LIB_PATH), reason="libtwell.so not built")

P = 0x10000
PL = T.CPlanes(P, P)


def _w(experts=1, rows=64, cols=128, bits=4, group=64):
    return T.CWDesc(experts, rows, cols, bits, group)


@pytest.mark.parametrize("kw,code", [
    ({}, T.TWELL_OK),
    ({"bits": 16, "group": 0}, T.TWELL_OK),
    ({"rows": 1, "cols": 1}, T.TWELL_OK),
    ({"experts": 0}, T.TWELL_EINVAL),
    ({"rows": 0}, T.TWELL_EINVAL),
    ({"cols": -1}, T.TWELL_EINVAL),
    ({"bits": 8}, T.TWELL_EINVAL),
    ({"group": 16}, T.TWELL_EINVAL),
    ({"group": 0}, T.TWELL_EINVAL),
    ({"bits": 16, "group": 64}, T.TWELL_EINVAL),
    ({"experts": 1025}, T.TWELL_EUNSUPPORTED),
    ({"rows": (1 << 20) + 1}, T.TWELL_EUNSUPPORTED),
    ({"rows": 1 << 20, "cols": 1 << 15}, T.TWELL_EUNSUPPORTED),
])
def test_weights_descriptor(kw, code):
    d, out = _w(**kw), T.CWSizes()
    assert T.library().twell_weights_sizes(ctypes.byref(d), ctypes.byref(out)) == code


def test_weights_sizes_pad_to_blocks():
    lib = T.library()
    assert lib.twell_weights_sizes(None, ctypes.byref(T.CWSizes())) == T.TWELL_EINVAL
    assert lib.twell_weights_sizes(ctypes.byref(_w()), None) == T.TWELL_EINVAL
    for rows, cols in ((16, 128), (17, 128), (16, 129), (1, 1), (1001, 707)):
        blocks = -(-rows // 16) * -(-cols // 128)
        assert T._weights_sizes(T.WDesc(3, rows, cols, 16)) == (3 * blocks * 4096, 0)
        for group in (32, 64, 128):
            assert T._weights_sizes(T.WDesc(3, rows, cols, 4, group)) == (3 * blocks * 1024,
                                                                          3 * blocks * 16 * (128 // group) * 2)


def test_pack_and_unpack_refuse():
    lib = T.library()
    d, d16 = ctypes.byref(_w()), ctypes.byref(_w(bits=16, group=0))
    for f in (lambda w, t, pl, d=d: lib.twell_weights_pack(d, w, t, 0, pl, None),
              lambda w, t, pl, d=d: lib.twell_weights_unpack(d, pl, w, t, None)):
        assert f(None, T.TWELL_BF16, PL) == T.TWELL_EINVAL
        assert f(P + 1, T.TWELL_BF16, PL) == T.TWELL_EINVAL
        assert f(P + 2, T.TWELL_FP32, PL) == T.TWELL_EINVAL
        assert f(P, 7, PL) == T.TWELL_EINVAL
        assert f(P, T.TWELL_BF16, T.CPlanes(0, P)) == T.TWELL_EINVAL
        assert f(P, T.TWELL_BF16, T.CPlanes(P, 0)) == T.TWELL_EINVAL
        assert f(P, T.TWELL_BF16, T.CPlanes(P + 8, P)) == T.TWELL_EINVAL
        assert f(P, T.TWELL_FP32, PL, d16) == T.TWELL_EUNSUPPORTED  # bf16 planes hold bf16 weights
    assert lib.twell_weights_pack(d, P, T.TWELL_BF16, 2, PL, None) == T.TWELL_EINVAL
    assert lib.twell_weights_pack(None, P, T.TWELL_BF16, 0, PL, None) == T.TWELL_EINVAL


def test_linear_refuses():
    lib = T.library()
    f = lib.twell_linear_fwd
    d, bf = ctypes.byref(_w()), T.TWELL_BF16
    assert f(d, T.CPlanes(0, 0), 0, bf, None, 128, None, 64, None) == T.TWELL_OK  # no tokens: nothing is read
    assert f(d, PL, -1, bf, P, 128, P, 64, None) == T.TWELL_EINVAL
    assert f(d, PL, 1, 5, P, 128, P, 64, None) == T.TWELL_EINVAL
    assert f(d, PL, 1, bf, P, 127, P, 64, None) == T.TWELL_EINVAL  # rows overlap
    assert f(d, PL, 1, bf, P, 128, P, 63, None) == T.TWELL_EINVAL
    assert f(d, PL, 1, bf, None, 128, P, 64, None) == T.TWELL_EINVAL
    assert f(d, PL, 1, bf, P, 128, None, 64, None) == T.TWELL_EINVAL
    assert f(d, PL, 1, bf, P + 1, 128, P, 64, None) == T.TWELL_EINVAL
    assert f(d, PL, 1, T.TWELL_FP32, P, 128, P + 2, 64, None) == T.TWELL_EINVAL
    assert f(d, T.CPlanes(P, 0), 1, bf, P, 128, P, 64, None) == T.TWELL_EINVAL
    assert f(d, PL, (1 << 20) + 1, bf, P, 128, P, 64, None) == T.TWELL_EUNSUPPORTED
    assert f(d, PL, 1, bf, P, (1 << 40) + 1, P, 64, None) == T.TWELL_EUNSUPPORTED
    assert f(ctypes.byref(_w(experts=2)), PL, 1, bf, P, 128, P, 64, None) == T.TWELL_EUNSUPPORTED
    assert f(ctypes.byref(_w(bits=16, group=0)), PL, 1, bf, P, 128, P, 64, None) == T.TWELL_EUNSUPPORTED


def _m(**kw):
    base = dict(T=4, ldx=128, ldy=128, d_model=128, d_ff=64, experts=8, top_k=2, dtype=T.TWELL_BF16, bits=4, group=64,
                act=0, renorm=1)
    base.update(kw)
    return T.CMoeDesc(**base)


@pytest.mark.parametrize("kw,code", [
    ({}, T.TWELL_OK),
    ({"T": 0}, T.TWELL_OK),
    ({"T": 100000}, T.TWELL_OK),
    ({"bits": 16, "group": 0}, T.TWELL_OK),
    ({"T": -1}, T.TWELL_EINVAL),
    ({"top_k": 0}, T.TWELL_EINVAL),
    ({"top_k": 9}, T.TWELL_EINVAL),
    ({"dtype": 2}, T.TWELL_EINVAL),
    ({"act": 2}, T.TWELL_EINVAL),
    ({"renorm": 2}, T.TWELL_EINVAL),
    ({"ldx": 127}, T.TWELL_EINVAL),
    ({"ldy": 127}, T.TWELL_EINVAL),
    ({"d_ff": 0}, T.TWELL_EINVAL),
    ({"bits": 5}, T.TWELL_EINVAL),
    ({"experts": 2000}, T.TWELL_EUNSUPPORTED),
    ({"experts": 64, "top_k": 33}, T.TWELL_EUNSUPPORTED),
    ({"T": 1 << 21}, T.TWELL_EUNSUPPORTED),
    ({"ldx": 1 << 41}, T.TWELL_EUNSUPPORTED),
])
def test_moe_descriptor(kw, code):
    n = ctypes.c_size_t()
    assert T.library().twell_moe_sizes(ctypes.byref(_m(**kw)), ctypes.byref(n)) == code


def test_moe_refuses():
    lib = T.library()
    d = _m()
    n = ctypes.c_size_t()
    assert lib.twell_moe_sizes(ctypes.byref(d), None) == T.TWELL_EINVAL
    assert lib.twell_moe_sizes(ctypes.byref(d), ctypes.byref(n)) == T.TWELL_OK
    good = dict(d=ctypes.byref(d), x=P, r=P, bias=None, g=PL, u=PL, dn=PL, y=P, ids=P, w=P, ws=P, n=n.value)

    def call(**kw):
        a = dict(good, **kw)
        return lib.twell_moe_fwd(a["d"], a["x"], a["r"], a["bias"], a["g"], a["u"], a["dn"], a["y"], a["ids"], a["w"],
                                 a["ws"], a["n"], None)

    for bad in (dict(x=None), dict(r=None), dict(y=None), dict(ids=None), dict(w=None), dict(ws=None), dict(x=P + 1),
                dict(y=P + 1), dict(r=P + 1), dict(ids=P + 2), dict(w=P + 2), dict(bias=P + 2), dict(ws=P + 8),
                dict(n=n.value - 1), dict(g=T.CPlanes(0, P)), dict(u=T.CPlanes(P, 0)), dict(dn=T.CPlanes(P + 4, P)),
                dict(d=None)):
        assert call(**bad) == T.TWELL_EINVAL, bad
    e = _m(T=0)
    none = T.CPlanes(0, 0)
    assert call(d=ctypes.byref(e), x=None, r=None, y=None, ids=None, w=None, ws=None, n=0, g=none, u=none,
                dn=none) == T.TWELL_OK


def test_moe_workspace_stops_growing_with_the_batch():
    big = [T.moe_ws_bytes(T.MoeDesc(t, 128, 64, 8, 2, "bf16", 4, 64)) for t in (64, 65, 4096)]
    assert big[0] == big[1] == big[2] >= 64 * 2 * 128 * 2 * 2


def test_binding_refuses_host_tensors_and_bad_shapes():
    wd = T.WDesc(1, 64, 128, 4, 64)
    pl = T.alloc_weights(wd, device="cpu")
    with pytest.raises(ValueError):
        T.twell_weights_pack(wd, torch.zeros(64, 128, dtype=torch.bfloat16), pl)
    with pytest.raises(ValueError):
        T.twell_weights_pack(wd, torch.zeros(64, 128, dtype=torch.float16), pl)
    with pytest.raises(TypeError):
        T.twell_weights_unpack(wd, pl, None)
    with pytest.raises(ValueError):
        T.twell_linear_fwd(wd, pl, torch.zeros(1, 128, dtype=torch.bfloat16), torch.zeros(1, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        T.twell_linear_fwd(wd, pl, torch.zeros(128), torch.zeros(64))
    with pytest.raises(ValueError):
        T.moe_ws_bytes(T.MoeDesc(1, 128, 64, 8, 2, "bf16", 4, 64, act="tanh"))
    with pytest.raises(T.TwellError):
        T.moe_ws_bytes(T.MoeDesc(1, 128, 64, 8, 9, "bf16", 4, 64))


@pytest.mark.parametrize("make", [
    lambda big: T.WDesc(1, 64, 128, 4, big + 64), lambda big: T.WDesc(1, big + 64, 128, 4, 64),
    lambda big: T.WDesc(big + 1, 64, 128, 16), lambda big: T.WDesc(1, 64, big + 128, 16, 0),
    lambda big: T.WDesc(1, 64, 128, big + 16),
])
def test_numbers_beyond_32_bits_do_not_wrap(make):
    for big in (1 << 32, -(1 << 32)):
        with pytest.raises(ValueError, match="32 bits"):
            make(big).plane_bytes
        with pytest.raises(ValueError, match="32 bits"):
            T.alloc_weights(make(big), device="cpu")


@pytest.mark.parametrize("name", ["d_model", "d_ff", "experts", "top_k", "bits", "group"])
def test_moe_numbers_beyond_32_bits_do_not_wrap(name):
    good = dict(T=1, d_model=128, d_ff=64, experts=8, top_k=2, dtype="bf16", bits=4, group=64)
    T.moe_ws_bytes(T.MoeDesc(**good))
    with pytest.raises(ValueError, match="32 bits"):
        T.moe_ws_bytes(T.MoeDesc(**{**good, name: good[name] + (1 << 32)}))
    with pytest.raises(ValueError, match="64 bits"):
        T.moe_ws_bytes(T.MoeDesc(**{**good, "T": 1 << 64}))


@pytest.mark.parametrize("desc", [T.WDesc(2, 64, 128, 4, 64), T.MoeDesc(3, 128, 64, 8, 2, "bf16", 4, 64)])
def test_descriptors_are_copied_and_sent_after_their_first_use_as_before(desc):
    """What a descriptor keeps of its C structs is its own affair: a model or a worker's arguments that hold one can be
    copied and pickled."""
    used = desc.plane_bytes if isinstance(desc, T.WDesc) else desc._call
    for again in (copy.copy(desc), copy.deepcopy(desc), pickle.loads(pickle.dumps(desc)), dataclasses.replace(desc)):
        assert again == desc and type(again) is type(desc) and hash(again) == hash(desc)
        if isinstance(desc, T.WDesc):
            assert again.plane_bytes == used
        else:
            assert again.ws_bytes == used[-1]


class _On(torch.Tensor):
    """A host tensor that claims to be on GPU `dev`; calls that hold it have no tokens, so that nothing is launched."""
    dev = 0
    is_cuda = True

    def get_device(self):
        return self.dev

    @classmethod
    def make(cls, dev, *shape, dtype=torch.bfloat16):
        t = torch.zeros(*shape, dtype=dtype).as_subclass(cls)
        t.dev = dev
        return t


def test_tensors_have_to_be_on_one_device_where_the_launch_goes(monkeypatch):
    """A launch on the default stream goes to the current device, and all tensors of a call are on one: tensors of
    another are refused, whichever argument it is."""
    monkeypatch.setattr(T, "_device_count", lambda: 2)
    wd, md = T.WDesc(1, 64, 128, 4, 64), T.MoeDesc(0, 128, 64, 2, 1, "bf16", 4, 64)

    def planes(desc, dev):
        return T.Weights(_On.make(dev, desc.plane_bytes[0], dtype=torch.uint8),
                         _On.make(dev, desc.plane_bytes[1] // 2))

    def linear(x=0, w=0, y=0):
        T.twell_linear_fwd(wd, planes(wd, w), _On.make(x, 0, 128), _On.make(y, 0, 64), stream=0)

    def moe(x=0, r=0, b=0, gate=0, up=0, down=0, y=0, ids=0, wts=0, ws=0):
        out = T.MoeOut(_On.make(y, 0, 128), _On.make(ids, 0, 1, dtype=torch.int32),
                       _On.make(wts, 0, 1, dtype=torch.float32))
        T.twell_moe_fwd(md, _On.make(x, 0, 128), _On.make(r, 2, 128),
                        T.MoeWeights(planes(md.in_desc, gate), planes(md.in_desc, up), planes(md.out_desc, down)), out,
                        _On.make(ws, 256, dtype=torch.uint8), router_bias=_On.make(b, 2, dtype=torch.float32), stream=0)

    for current, other in ((0, 1), (1, 0)):
        monkeypatch.setattr(T, "_current_device", lambda: current)
        for call, names in ((linear, "x w y"), (moe, "x r b gate up down y ids wts ws")):
            names = names.split()
            call(**dict.fromkeys(names, current))
            for name in names:
                with pytest.raises(ValueError, match=f"cuda:{other}"):
                    call(**{**dict.fromkeys(names, current), name: other})
            with pytest.raises(ValueError, match=f"cuda:{other}"):
                call(**dict.fromkeys(names, other))
    monkeypatch.setattr(T, "_current_device", lambda: 0)
    with pytest.raises(ValueError, match="cuda:1"):
        T.twell_weights_pack(wd, _On.make(0, 1, 64, 128), planes(wd, 1), stream=0)
    with pytest.raises(ValueError, match="cuda:1"):
        T.twell_weights_unpack(wd, planes(wd, 1), _On.make(0, 1, 64, 128), stream=0)
