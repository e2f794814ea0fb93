"""GPU parity of the few-token operators against 64-bit references.

Tolerances.  A bf16 output carries one rounding, at most 2^-8 of its value (8
significand bits); on top of it comes the fp32 arithmetic.  The norm of the fp32
error of a product is taken as at most 1e-6 of the result's: 2^-24 per accumulation, times at most 6
for the codes' offset (|q + 24| against the codes' own size), times 2 for the few
chained roundings of a random walk.  The hidden values of the expert layer add
2^-17 in bf16 (kept as two bf16 numbers).  Element by element, 40 times that
of the output's rms is allowed, plus the rounding.
"""
import numpy as np
import pytest
import torch

import _few_token as R
from activation_sparse_feedforward_amd import twell as T
from _helpers import check_guards, guarded, host64, say

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
NOT_A_CASE = 0xA5


def _close(got, ref, dtype, extra=0.0):
    got = host64(got)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    ok = np.isfinite(ref)
    assert np.array_equal(got[~ok & ~np.isnan(ref)], ref[~ok & ~np.isnan(ref)])
    g, r = got[ok], ref[ok]
    if not r.size:
        return
    rnd = 2.0 ** -8 if dtype == "bf16" else 0.0
    tol = 1e-6 + extra
    rms = np.sqrt(np.mean(r * r))
    assert np.linalg.norm(g - r) <= (rnd + tol) * np.linalg.norm(r), np.linalg.norm(g - r) / np.linalg.norm(r)
    assert np.all(np.abs(g - r) <= rnd * np.abs(r) + 40 * tol * rms + 1e-38)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, scale=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * scale


def _packed(w, wd, transposed=False):
    pl = T.Weights(*(guarded(t.shape, t.dtype) for t in T.alloc_weights(wd)))
    T.twell_weights_pack(wd, w, pl, transposed=transposed)
    return pl


# ----------------------------------------------------------------------------- packing
@pytest.mark.parametrize("E,N,K", [(1, 1, 1), (1, 16, 128), (2, 17, 129), (3, 100, 31), (1, 5, 300), (2, 70, 1000)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("wtype", ["bf16", "fp32"])
@pytest.mark.parametrize("transposed", [False, True])
def test_pack_4bit_is_exact(E, N, K, group, wtype, transposed):
    say(f"[gpu case] pack 4 bits E={E} N={N} K={K} group={group} {wtype} transposed={transposed}")
    w = _randn(_gen(N * K + group), E, N, K).to(DT[wtype])
    w[:, N // 2, : K // 2] = 0
    src = w.transpose(1, 2).contiguous() if transposed else w
    wd = T.WDesc(E, N, K, 4, group)
    pl = _packed(src, wd, transposed)
    back = {d: guarded((E, N, K), DT[d]) for d in ("fp32", "bf16")}
    for b in back.values():
        T.twell_weights_unpack(wd, pl, b)
    torch.cuda.synchronize()
    check_guards(*pl, *back.values())
    ref = R.quantise(w.float().cpu().numpy(), group)
    assert np.array_equal(host64(back["fp32"]), ref)
    assert np.array_equal(host64(back["bf16"]), R.bf16_round(ref).astype(np.float64))
    q, s = R.planes_to_codes(pl.codes.cpu().numpy(), pl.scales.view(torch.int16).cpu().numpy(), E, N, K, group)
    assert np.array_equal((q * s.astype(np.float64))[:, :N, :K], ref)
    assert not np.any(q[:, N:, :]) and not np.any(q[:, :, K:])  # padding


@pytest.mark.parametrize("E,N,K", [(1, 1, 1), (2, 17, 129), (1, 70, 1000), (3, 128, 256)])
@pytest.mark.parametrize("transposed", [False, True])
def test_pack_16bit_keeps_every_bit(E, N, K, transposed):
    say(f"[gpu case] pack 16 bits E={E} N={N} K={K} transposed={transposed}")
    bits = torch.randint(-32768, 32768, (E, N, K), generator=_gen(5), device="cuda", dtype=torch.int16)
    wd = T.WDesc(E, N, K, 16)
    src = bits.transpose(1, 2).contiguous() if transposed else bits
    pl = _packed(src.view(torch.bfloat16), wd, transposed)
    back = guarded((E, N, K), torch.bfloat16)
    T.twell_weights_unpack(wd, pl, back)
    torch.cuda.synchronize()
    check_guards(*pl, back)
    # NaN payloads may become quiet on the way out; everything else keeps its bits
    nan = torch.isnan(bits.view(torch.bfloat16))
    assert torch.equal(back.view(torch.int16)[~nan], bits[~nan]) and torch.isnan(back[nan]).all()


def test_pack_marks_groups_that_are_not_finite_and_keeps_tiny_ones():
    w = torch.full((1, 16, 256), 0.5, device="cuda")
    w[0, 0, 3] = float("nan")
    w[0, 1, 130] = float("inf")
    w[0, 2, :] = 1e-42  # a scale that bf16 cannot hold
    w[0, 3, :] = 1e-37
    w[0, 4, :] = 3e38
    wd = T.WDesc(1, 16, 256, 4, 64)
    pl = _packed(w, wd)
    back = torch.empty_like(w)
    T.twell_weights_unpack(wd, pl, back)
    assert np.array_equal(host64(back), R.quantise(w.cpu().numpy(), 64), equal_nan=True)
    assert torch.isnan(back[0, 0, :64]).all() and torch.isnan(back[0, 1, 128:192]).all()
    assert torch.isfinite(back[0, 0, 64:]).all()


def test_planes_beyond_4_gib():
    """The last expert of planes whose offsets pass 32 bits."""
    E, N, K = 1024, 1024, 2200
    say(f"[gpu case] planes beyond 4 GiB: E={E} N={N} K={K}")
    w = torch.zeros((E, N, K), dtype=torch.bfloat16, device="cuda")
    w[-1] = _randn(_gen(3), N, K).bfloat16()
    wd = T.WDesc(E, N, K, 16)
    pl = T.alloc_weights(wd)
    assert pl.codes.numel() > 1 << 32
    T.twell_weights_pack(wd, w, pl)
    back = torch.empty_like(w)
    T.twell_weights_unpack(wd, pl, back)
    assert torch.equal(back[-1], w[-1]) and not back[:-1].any()


# ----------------------------------------------------------------------------- linear
def _linear_case(T_, N, K, group, dtype, seed=0, x=None):
    g = _gen(seed + T_ * 7 + N + K)
    w = _randn(g, 1, N, K, scale=K ** -0.5).bfloat16()
    wd = T.WDesc(1, N, K, 4, group)
    pl = _packed(w, wd)
    x = _randn(g, T_, K).to(DT[dtype]) if x is None else x
    ref = host64(x) @ R.quantise(w[0].float().cpu().numpy(), group).T
    return wd, pl, x, ref


@pytest.mark.parametrize("T_", [1, 2, 4, 5, 15, 16, 17, 32, 33, 64, 100])
@pytest.mark.parametrize("N,K", [(1, 1), (17, 127), (300, 1001), (64, 4096)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_linear(T_, N, K, group, dtype):
    say(f"[gpu case] linear T={T_} N={N} K={K} group={group} {dtype}")
    wd, pl, x, ref = _linear_case(T_, N, K, group, dtype)
    y = guarded((T_, N), DT[dtype])
    T.twell_linear_fwd(wd, pl, x, y)
    torch.cuda.synchronize()
    check_guards(*pl, y)
    _close(y, ref, dtype)


@pytest.mark.parametrize("T_", [3, 7, 13, 29, 61, 100])
@pytest.mark.parametrize("N", [4090, 4100, 8200, 12288, 12300])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_linear_many_rows(T_, N, group, dtype):
    """Rows for every CU: the most tokens a workgroup takes, and one to four tiles of rows each."""
    say(f"[gpu case] linear many rows T={T_} N={N} group={group} {dtype}")
    wd, pl, x, ref = _linear_case(T_, N, 203, group, dtype)
    y = guarded((T_, N), DT[dtype])
    T.twell_linear_fwd(wd, pl, x, y)
    torch.cuda.synchronize()
    check_guards(*pl, y)
    _close(y, ref, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T_", [1, 3, 20])
def test_linear_strided_rows_at_odd_addresses(T_, dtype):
    """x and y as windows of wider tensors, starting one element in: nothing but the window is written."""
    N, K = 45, 203
    say(f"[gpu case] linear strided T={T_} {dtype}")
    wide_x = _randn(_gen(9), T_ + 1, K + 14).to(DT[dtype])
    wide_y = torch.full((T_ + 1, N + 9), 7.0, dtype=DT[dtype], device="cuda")
    x, y = wide_x[:T_, 1:1 + K], wide_y[:T_, 3:3 + N]
    wd, pl, _, ref = _linear_case(T_, N, K, 32, dtype, x=x)
    # what surrounds x must not matter
    wide_x[T_:] = float("nan")
    wide_x[:, 0] = float("nan")
    wide_x[:, 1 + K:] = float("nan")
    T.twell_linear_fwd(wd, pl, x, y)
    _close(y, ref, dtype)
    mask = torch.ones_like(wide_y, dtype=torch.bool)
    mask[:T_, 3:3 + N] = False
    assert (wide_y[mask] == 7.0).all()


def test_linear_rows_beyond_4_gib_apart():
    ld = (1 << 31) + 24
    buf = torch.empty(ld + 256, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((2, 200), (ld, 1))
    x.copy_(_randn(_gen(1), 2, 200))
    wd, pl, _, ref = _linear_case(2, 33, 200, 64, "bf16", x=x)
    y = torch.empty(2, 33, dtype=torch.bfloat16, device="cuda")
    T.twell_linear_fwd(wd, pl, x, y)
    _close(y, ref, "bf16")


def test_linear_no_tokens_and_rows_that_are_not_finite():
    wd, pl, x, ref = _linear_case(6, 40, 300, 64, "bf16")
    T.twell_linear_fwd(wd, pl, x[:0], torch.empty(0, 40, dtype=torch.bfloat16, device="cuda"))
    x[2, 5] = float("nan")
    x[4, 7] = float("inf")
    y = torch.empty(6, 40, dtype=torch.bfloat16, device="cuda")
    T.twell_linear_fwd(wd, pl, x, y)
    assert torch.isnan(y[2]).all() and torch.isnan(y[4]).all()
    keep = [0, 1, 3, 5]
    _close(y[keep], ref[keep], "bf16")


def test_linear_weight_group_that_is_not_finite_spoils_its_row_alone():
    w = _randn(_gen(2), 1, 40, 300, scale=0.1).bfloat16()
    w[0, 11, 70] = float("nan")
    wd = T.WDesc(1, 40, 300, 4, 64)
    pl = _packed(w, wd)
    x = _randn(_gen(3), 3, 300)
    y = torch.empty(3, 40, device="cuda")
    T.twell_linear_fwd(wd, pl, x, y)
    _close(y, host64(x) @ R.quantise(w[0].float().cpu().numpy(), 64).T, "fp32")
    assert torch.isnan(y[:, 11]).all()


def test_binding_refuses_on_the_device():
    wd = T.WDesc(1, 64, 128, 4, 64)
    pl = T.alloc_weights(wd)
    x = torch.zeros(2, 128, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda")
    small = T.Weights(pl.codes[:-1], pl.scales)
    bad = [(wd, pl, x[:, :64], y), (wd, pl, x, y[:1]), (wd, pl, x, y.float()), (wd, small, x, y),
           (wd, T.Weights(pl.codes, pl.scales[:-1]), x, y),
           (wd, pl, torch.zeros(128, 2, dtype=torch.bfloat16, device="cuda").t(), y),
           (wd, pl, torch.zeros(1, 128, dtype=torch.bfloat16, device="cuda").expand(2, 128), y)]
    for a in bad:
        with pytest.raises(ValueError):
            T.twell_linear_fwd(*a)
    with pytest.raises(T.TwellError) as e:
        T.twell_linear_fwd(T.WDesc(1, 64, 128, 16), T.alloc_weights(T.WDesc(1, 64, 128, 16)), x, y)
    assert e.value.code == T.TWELL_EUNSUPPORTED


# ----------------------------------------------------------------------------- mixture of experts
def _moe_case(md, seed=0):
    g = _gen(seed + md.T + 3 * md.experts + md.d_model)
    E, d, f = md.experts, md.d_model, md.d_ff
    x = _randn(g, md.T, d).to(md.torch_dtype)
    router = _randn(g, E, d, scale=2 * d ** -0.5).to(md.torch_dtype)
    gate, up = (_randn(g, E, f, d, scale=d ** -0.5).bfloat16() for _ in range(2))
    down = _randn(g, E, f, d, scale=f ** -0.5).bfloat16()
    w = T.MoeWeights(_packed(gate, md.in_desc), _packed(up, md.in_desc), _packed(down, md.out_desc, True))
    mats = [gate, up, down.transpose(1, 2)]
    mats = [m.float().cpu().numpy() for m in mats]
    mats = [R.quantise(m, md.group) if md.bits == 4 else m.astype(np.float64) for m in mats]
    return x, router, w, mats


def _moe_out(md):
    return T.MoeOut(*(guarded(t.shape, t.dtype) for t in T.alloc_moe_out(md)))


def _moe_check(md, x, router, w, mats, bias=None):
    out, ws = _moe_out(md), guarded((T.moe_ws_bytes(md),), torch.uint8)
    T.twell_moe_fwd(md, x, router, w, out, ws, router_bias=bias)
    torch.cuda.synchronize()
    check_guards(*out, ws)
    x64 = host64(x)
    ids, wts = R.route(x64, host64(router), None if bias is None else bias.cpu().numpy(), md.top_k, md.renorm)
    assert np.array_equal(out.ids.cpu().numpy(), ids)
    # the logits' fp32 sums of up to some 8 in size, through exp: 2e-6 of a weight
    got = host64(out.weights)
    assert np.array_equal(np.isnan(got), np.isnan(wts))
    assert np.all(np.abs(got - wts)[~np.isnan(wts)] <= 4e-6 * np.abs(wts)[~np.isnan(wts)] + 1e-37)
    _close(out.y, R.moe(x64, ids, wts, *mats, md.act), md.dtype, extra=4e-6 + (2.0 ** -17 if md.dtype == "bf16" else 0))
    return out


@pytest.mark.parametrize("T_,E,k,d,f", [
    (1, 1, 1, 64, 32), (1, 8, 2, 128, 256), (3, 7, 3, 101, 77), (4, 64, 8, 256, 130), (5, 5, 5, 130, 129),
    (16, 16, 4, 200, 64), (17, 9, 2, 96, 200), (64, 4, 2, 72, 48), (64, 3, 3, 65, 33), (65, 16, 4, 48, 40),
    (130, 6, 1, 40, 24), (2, 200, 12, 64, 40), (20, 1024, 32, 40, 20),
])
@pytest.mark.parametrize("bits,group", [(16, 0), (4, 32), (4, 64), (4, 128)])
@pytest.mark.parametrize("dtype,act,renorm", [("bf16", "relu", True), ("fp32", "silu", False), ("bf16", "silu", False),
                                              ("fp32", "relu", True)])
def test_moe(T_, E, k, d, f, bits, group, dtype, act, renorm):
    say(f"[gpu case] moe T={T_} E={E} k={k} d={d} f={f} bits={bits} group={group} {dtype} {act} renorm={renorm}")
    md = T.MoeDesc(T_, d, f, E, k, dtype, bits, group, act, renorm)
    _moe_check(md, *_moe_case(md))


@pytest.mark.parametrize("T_", [1, 16, 64])
@pytest.mark.parametrize("bits,group", [(16, 0), (4, 128)])
def test_moe_larger_widths(T_, bits, group):
    md = T.MoeDesc(T_, 1024, 512, 8, 2, "bf16", bits, group, "silu", True)
    say(f"[gpu case] moe larger T={T_} bits={bits}")
    _moe_check(md, *_moe_case(md))


@pytest.mark.parametrize("T_", [5, 20, 64])
@pytest.mark.parametrize("bits,group", [(16, 0), (4, 32), (4, 64), (4, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_moe_work_for_every_cu(T_, bits, group, dtype):
    """Many experts: the most tiles a workgroup takes, some of them beyond the last."""
    md = T.MoeDesc(T_, 300, 200, 40, 8, dtype, bits, group, "silu", True)
    say(f"[gpu case] moe many T={T_} bits={bits} group={group} {dtype}")
    _moe_check(md, *_moe_case(md))


@pytest.mark.parametrize("T_,E,k,d", [(1, 16, 4, 600), (2, 5, 2, 601), (4, 4, 4, 520), (3, 1024, 32, 40), (4, 256, 3, 130),
                                      (1, 17, 3, 1030)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_moe_router_of_a_few_tokens(T_, E, k, d, dtype):
    """Small routers and large ones, with experts taken out by the bias and a token that is not finite."""
    say(f"[gpu case] moe router T={T_} E={E} k={k} d={d} {dtype}")
    md = T.MoeDesc(T_, d, 70, E, k, dtype, 4, 64, "relu", False)
    x, router, w, mats = _moe_case(md)
    bias = _randn(_gen(E), E)
    bias[::3] = float("-inf")
    _moe_check(md, x, router, w, mats, bias)
    x[T_ - 1, d - 1] = float("nan")
    out = _moe_check(md, x, router, w, mats, bias)
    assert torch.isnan(out.y[T_ - 1]).all()
    assert not torch.isnan(out.y[:T_ - 1]).any()


@pytest.mark.parametrize("T_", [2, 20])
def test_moe_planes_beyond_4_gib(T_):
    """The last expert's weights begin 4.3 GiB into each plane."""
    say(f"[gpu case] moe planes beyond 4 GiB T={T_}")
    md = T.MoeDesc(T_, 4096, 4096, 140, 2, "bf16", 16, 0, "silu", True)
    g = _gen(5)
    x = _randn(g, T_, 4096).bfloat16()
    router = _randn(g, 140, 4096, scale=4096 ** -0.5).bfloat16()
    bias = torch.full((140,), float("-inf"), device="cuda")
    bias[[1, 139]] = 0.0
    w, kept = T.alloc_moe_weights(md), []
    for desc, planes, transposed in ((md.in_desc, w.gate, False), (md.in_desc, w.up, False), (md.out_desc, w.down, True)):
        full = torch.randn(140, 4096, 4096, generator=g, device="cuda", dtype=torch.bfloat16) / 64
        T.twell_weights_pack(desc, full, planes, transposed=transposed)
        kept.append(full[[1, 139]].double())
        del full
    out = T.alloc_moe_out(md)
    T.twell_moe_fwd(md, x, router, w, out, T.alloc_moe_ws(md), router_bias=bias)
    x64 = host64(x)
    ids, wts = R.route(x64, host64(router), bias.cpu().numpy(), 2, True)
    assert np.array_equal(out.ids.cpu().numpy(), ids)
    xg, ref = x.double(), torch.zeros(T_, 4096, dtype=torch.float64, device="cuda")
    for i, e in enumerate((1, 139)):
        gate, up, down = (k[i] for k in kept)
        a = xg @ gate.T
        y = (a / (1 + torch.exp(-a)) * (xg @ up.T)) @ down
        ref += y * torch.from_numpy((wts * (ids == e)).sum(1)).cuda()[:, None]
    _close(out.y, ref.cpu().numpy(), "bf16", extra=4e-6 + 2.0 ** -17)


@pytest.mark.parametrize("T_", [2, 40])
def test_moe_masked_experts_ties_and_empty_rows(T_):
    md = T.MoeDesc(T_, 96, 40, 12, 4, "fp32", 4, 32, "silu", True)
    x, router, w, mats = _moe_case(md)
    bias = torch.zeros(12, device="cuda")
    bias[[0, 3, 5]] = float("-inf")
    out = _moe_check(md, x, router, w, mats, bias)
    assert not np.isin(out.ids.cpu().numpy(), [0, 3, 5]).any()
    # fewer experts left than choices: the others have weight 0 and lowest indices
    bias[:] = float("-inf")
    bias[[7, 2]] = torch.tensor([0.5, -0.5], device="cuda")
    out = _moe_check(md, x, router, w, mats, bias)
    assert (out.weights[:, 2:] == 0).all() and (out.ids[:, 2:].cpu() == torch.tensor([0, 1])).all()
    # no expert left: empty rows
    bias[:] = float("-inf")
    out = _moe_check(md, x, router, w, mats, bias)
    assert (out.y == 0).all() and (out.weights == 0).all() and (out.ids.cpu() == torch.arange(4)).all()
    # equal logits everywhere: the lowest indices
    out = _moe_check(md, x, torch.zeros_like(router), w, mats)
    assert (out.ids.cpu() == torch.arange(4)).all()


@pytest.mark.parametrize("bits,group", [(16, 0), (4, 64)])
def test_moe_tokens_that_are_not_finite_spoil_themselves_alone(bits, group):
    md = T.MoeDesc(20, 130, 50, 6, 2, "bf16", bits, group, "relu", True)
    x, router, w, mats = _moe_case(md)
    base = _moe_check(md, x, router, w, mats)
    x[3, 100] = float("nan")
    out = _moe_out(md)
    ws = T.alloc_moe_ws(md)
    T.twell_moe_fwd(md, x, router, w, out, ws)
    assert torch.isnan(out.y[3]).all() and torch.isnan(out.weights[3]).all()
    assert (out.ids[3].cpu() == torch.arange(2)).all()
    keep = [t for t in range(20) if t != 3]
    assert torch.equal(out.y[keep], base.y[keep]) and torch.equal(out.ids[keep], base.ids[keep])


def test_moe_all_tokens_on_one_expert_and_one_weight_that_is_not_finite():
    md = T.MoeDesc(64, 64, 48, 4, 1, "bf16", 16, 0, "silu", False)
    x, router, w, mats = _moe_case(md)
    bias = torch.tensor([-1e4, -1e4, 1e4, -1e4], device="cuda")
    out = _moe_check(md, x, router, w, mats, bias)
    assert (out.ids == 2).all()
    # a broken expert that nobody chooses does no harm
    bad = torch.full((1, 48, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    size = w.gate.codes.numel() // 4
    one = T.alloc_weights(T.WDesc(1, 48, 64, 16))
    T.twell_weights_pack(T.WDesc(1, 48, 64, 16), bad, one)
    w.gate.codes[:size] = one.codes
    again = _moe_check(md, x, router, w, mats, bias)
    assert torch.equal(again.y, out.y)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_moe_strided_rows(dtype):
    md = T.MoeDesc(9, 61, 40, 5, 2, dtype, 4, 32, "silu", True)
    x, router, w, mats = _moe_case(md)
    plain = _moe_check(md, x, router, w, mats)
    wide = torch.full((9, 90), float("nan"), dtype=DT[dtype], device="cuda")
    wide[:, 5:66] = x
    wide_y = torch.full((9, 70), 7.0, dtype=DT[dtype], device="cuda")
    o = T.alloc_moe_out(md)
    T.twell_moe_fwd(md, wide[:, 5:66], router, w, T.MoeOut(wide_y[:, 1:62], o.ids, o.weights), T.alloc_moe_ws(md))
    assert torch.equal(wide_y[:, 1:62], plain.y)
    assert (wide_y[:, 0] == 7).all() and (wide_y[:, 62:] == 7).all()


# ----------------------------------------------------------------------------- streams, graphs, repeats
def _everything(md, wd, x, router, w, gate, pl, out, ws, y, stream=None):
    T.twell_weights_pack(wd, gate, pl, stream=stream)
    T.twell_linear_fwd(wd, pl, x, y, stream=stream)
    T.twell_moe_fwd(md, x, router, w, out, ws, stream=stream)


@pytest.mark.parametrize("T_", [1, 70])
def test_streams_graph_replays_and_repeats_give_the_same_bits(T_):
    say(f"[gpu case] streams and graphs T={T_}")
    md = T.MoeDesc(T_, 256, 200, 8, 2, "bf16", 4, 64, "silu", True)
    x, router, w, _ = _moe_case(md)
    wd = T.WDesc(1, 300, 256, 4, 64)
    gate = _randn(_gen(8), 1, 300, 256).bfloat16()

    def buffers():
        return dict(pl=T.alloc_weights(wd), out=T.alloc_moe_out(md), ws=T.alloc_moe_ws(md),
                    y=torch.empty(T_, 300, dtype=torch.bfloat16, device="cuda"))

    def outs(b):
        return [*b["pl"], *b["out"], b["y"]]

    def same(a, b):
        return all(torch.equal(s.view(torch.uint8), t.view(torch.uint8)) for s, t in zip(outs(a), outs(b)))

    ref, again = buffers(), buffers()
    _everything(md, wd, x, router, w, gate, **ref)
    again["ws"].fill_(NOT_A_CASE)  # nothing in the workspace needs to start at zero
    _everything(md, wd, x, router, w, gate, **again)
    torch.cuda.synchronize()
    assert same(ref, again)

    side, b = torch.cuda.Stream(), buffers()
    torch.cuda.synchronize()
    _everything(md, wd, x, router, w, gate, **b, stream=side)
    side.synchronize()
    assert same(ref, b)

    b = buffers()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _everything(md, wd, x, router, w, gate, **b)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _everything(md, wd, x, router, w, gate, **b)
    for _ in range(3):
        for t in outs(b) + [b["ws"]]:
            t.view(torch.uint8).fill_(NOT_A_CASE)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same(ref, b)
