"""Layer norm against its formulas in 64 bits.

Bounds, with u = 2^-24 and n the additions on the longest way of a sum (a lane's elements, then lanes, then waves): a
sum is off by at most n u times the sum of magnitudes; each further operation adds u of its result; a result rounded to
its dtype adds half a step of that."""
import numpy as np
import pytest
import torch

from activation_sparse_feedforward_amd import twell as T
from _helpers import check_guards, guarded, say
from _many_token import DT, HALF, U32, capture, check, h64, layernorm, layernorm_grads

pytestmark = pytest.mark.gpu

WIDTHS = [1, 2, 7, 63, 64, 255, 257, 512, 513, 1001, 1024, 1025, 2048, 2049, 4096, 4099, 5000, 8192, 8200, 11008, 16383,
          16384]


def _data(T_, d, dtype, wdtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(T_, d, generator=g, device="cuda") * 3 + 1).to(DT[dtype])
    dy = torch.randn(T_, d, generator=g, device="cuda").to(DT[dtype])
    w, b = ((torch.randn(d, generator=g, device="cuda") * s + c).to(DT[wdtype]) for s, c in ((0.2, 1), (0.2, 0)))
    return x, dy, w, b


def check_forward(x, w, b, eps, y, stats, half):
    x, w, b = h64(x), (1.0 if w is None else h64(w)), (0.0 if b is None else h64(b))
    d = x.shape[1]
    n = d / 64 + 24
    ref, mean, rstd = layernorm(x, w, b, eps)
    c = np.abs(x - mean)
    e_mean = (n + 2) * U32 * np.abs(x).mean(1, keepdims=True)
    e_c = e_mean + U32 * (c + e_mean)
    # relative error of var + eps, then of its root
    e_var = ((n + 4) * U32 * (c ** 2).mean(1, keepdims=True) + 2 * (e_c * c).mean(1, keepdims=True)
             + (e_c ** 2).mean(1, keepdims=True)) * rstd ** 2
    e_rstd = 0.51 * e_var + 4 * U32
    e_h = rstd * (e_c + (c + e_c) * (e_rstd + 2 * U32))
    e_y = np.abs(w) * e_h + 2 * U32 * (np.abs(w) * rstd * c + np.abs(b))
    check(y, ref, 1.01 * e_y + half * (np.abs(ref) + 1.01 * e_y), "y")
    if stats is not None:
        s = h64(stats)
        check(s[:, :1], mean, e_mean, "mean")
        check(s[:, 1:], rstd, e_rstd * rstd, "rstd")


def check_backward(x, w, stats, dy, dx, dw, db, half, blocks):
    x, dy, s = h64(x), h64(dy), h64(stats)
    w = np.ones(x.shape[1]) if w is None else h64(w)
    T_, d = x.shape
    n = d / 64 + 24
    mean, rstd = s[:, :1], s[:, 1:]
    ref, rdw, rdb = layernorm_grads(x, w, mean, rstd, dy)
    h, g = np.abs((x - mean) * rstd), np.abs(dy * w)
    m0, m1 = np.abs((dy * w).mean(1, keepdims=True)), np.abs((dy * w * (x - mean) * rstd).mean(1, keepdims=True))
    e0 = (n + 3) * U32 * g.mean(1, keepdims=True)
    e1 = (n + 6) * U32 * (g * h).mean(1, keepdims=True)
    e = rstd * (6 * U32 * (g + m0 + h * m1) + e0 + h * e1)
    check(dx, ref, 1.01 * e + half * (np.abs(ref) + 1.01 * e), "dx")
    k = T_ / max(blocks, 1) + blocks / 16 + 24
    if dw is not None:
        check(dw, rdw, 1.01 * (k + 4) * U32 * (np.abs(dy) * h).sum(0), "dw")
    if db is not None:
        check(db, rdb, 1.01 * k * U32 * np.abs(dy).sum(0), "db")


def _run(x, dy, w, b, dtype, eps=1e-5):
    T_, d = x.shape
    desc = T.NormDesc(T_, d, dtype, eps)
    y, dx = guarded((T_, d), DT[dtype]), guarded((T_, d), DT[dtype])
    stats, dw, db = guarded((T_, 2), torch.float32), guarded((d,), torch.float32), guarded((d,), torch.float32)
    ws = guarded((desc.ws_bytes,), torch.uint8)
    T.twell_layernorm_fwd(desc, x, w, b, y, stats)
    T.twell_layernorm_bwd(desc, x, w, stats, dy, dx, dw, db, ws)
    torch.cuda.synchronize()
    check_guards(y, dx, stats, dw, db, ws)
    return y, stats, dx, dw, db


def _blocks(T_, d, dtype):
    return T.NormDesc(T_, d, dtype).ws_bytes // (8 * d)


@pytest.mark.parametrize("dtype,wdtype", [("bf16", "fp32"), ("bf16", "bf16"), ("fp32", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("d", WIDTHS)
def test_widths(d, dtype, wdtype):
    say(f"[gpu case] layer norm d={d} {dtype} weights {wdtype}")
    T_ = 13
    x, dy, w, b = _data(T_, d, dtype, wdtype, d)
    y, stats, dx, dw, db = _run(x, dy, w, b, dtype)
    check_forward(x, w, b, 1e-5, y, stats, HALF[dtype])
    check_backward(x, w, stats, dy, dx, dw, db, HALF[dtype], min(T_, _blocks(T_, d, dtype)))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T_", [1, 2, 3, 4, 5, 1023, 1025, 5001])
def test_rows(T_, dtype):
    say(f"[gpu case] layer norm T={T_} {dtype}")
    x, dy, w, b = _data(T_, 330, dtype, "fp32", T_)
    y, stats, dx, dw, db = _run(x, dy, w, b, dtype)
    check_forward(x, w, b, 1e-5, y, stats, HALF[dtype])
    check_backward(x, w, stats, dy, dx, dw, db, HALF[dtype], min(T_, _blocks(T_, 330, dtype)))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_without_weights_and_in_place(dtype):
    say(f"[gpu case] layer norm without weights, in place {dtype}")
    T_, d = 21, 3003
    x, dy, w, b = _data(T_, d, dtype, "fp32", 5)
    desc = T.NormDesc(T_, d, dtype, 1e-3)
    for ww, bb in ((None, None), (w, None), (None, b)):
        y, stats = torch.empty_like(x), torch.empty(T_, 2, device="cuda")
        T.twell_layernorm_fwd(desc, x, ww, bb, y, stats)
        check_forward(x, ww, bb, 1e-3, y, stats, HALF[dtype])
        alone = torch.empty_like(x)
        T.twell_layernorm_fwd(desc, x, ww, bb, alone)
        assert torch.equal(alone, y)
        over = x.clone()
        T.twell_layernorm_fwd(desc, over, ww, bb, over)
        assert torch.equal(over, y)
    ws = T.alloc_norm_ws(desc)
    dx, dw, db = torch.empty_like(x), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    T.twell_layernorm_bwd(desc, x, None, stats, dy, dx, dw, db, ws)
    check_backward(x, None, stats, dy, dx, dw, db, HALF[dtype], min(T_, _blocks(T_, d, dtype)))
    for over_x in (True, False):
        xx, gg = x.clone(), dy.clone()
        dw2, db2 = torch.empty_like(dw), torch.empty_like(db)
        T.twell_layernorm_bwd(desc, xx, None, stats, gg, xx if over_x else gg, dw2 if over_x else None,
                              None if over_x else db2, ws)
        assert torch.equal(xx if over_x else gg, dx)
        assert torch.equal(dw2, dw) if over_x else torch.equal(db2, db)


def test_no_rows():
    say("[gpu case] layer norm of no rows")
    desc = T.NormDesc(0, 700, "bf16")
    e = torch.empty(0, 700, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(700, device="cuda")
    stats = torch.empty(0, 2, device="cuda")
    dw, db = guarded((700,), torch.float32), guarded((700,), torch.float32)
    T.twell_layernorm_fwd(desc, e, w, w, e, stats)
    T.twell_layernorm_bwd(desc, e, w, stats, e, e, dw, db, T.alloc_norm_ws(desc))
    assert not dw.any() and not db.any()
    check_guards(dw, db)


def test_constant_rows_large_values_and_nan():
    """A constant row has h = 0; a mean far above the spread costs no more than its own rounding; a NaN or an infinity
    makes its own row NaN, and no other."""
    say("[gpu case] layer norm of special rows")
    d = 1500
    x = torch.randn(6, d, device="cuda")
    x[0] = 1e4
    x[1] = 1e4 + x[1]
    x[2] *= 1e15
    x[3, 7] = float("nan")
    x[4, 9] = float("inf")
    w, b = torch.randn(d, device="cuda"), torch.randn(d, device="cuda")
    desc = T.NormDesc(6, d, "fp32", 1e-5)
    y, stats = torch.empty_like(x), torch.empty(6, 2, device="cuda")
    T.twell_layernorm_fwd(desc, x, w, b, y, stats)
    good = [1, 2, 5]
    check_forward(x[good], w, b, 1e-5, y[good], stats[good], HALF["fp32"])
    check_forward(x[:1], w, b, 1e-5, y[:1], stats[:1], HALF["fp32"])
    assert torch.isnan(y[3]).all() and torch.isnan(y[4]).all()


def test_strided_rows_and_far_rows():
    say("[gpu case] layer norm of strided rows")
    T_, d = 40, 1001
    x, dy, w, b = _data(T_, d, "bf16", "bf16", 9)
    desc = T.NormDesc(T_, d, "bf16")
    y, stats, dx, dw, db = _run(x, dy, w, b, "bf16")
    wide = [torch.zeros(T_, d + 5, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    xs, ys, gs, dxs = (t[:, 1:1 + d] for t in wide)
    xs.copy_(x)
    gs.copy_(dy)
    stats2, dw2, db2 = torch.empty_like(stats), torch.empty_like(dw), torch.empty_like(db)
    T.twell_layernorm_fwd(desc, xs, w, b, ys, stats2)
    T.twell_layernorm_bwd(desc, xs, w, stats2, gs, dxs, dw2, db2, T.alloc_norm_ws(desc))
    assert all(torch.equal(p, q) for p, q in ((ys, y), (stats2, stats), (dxs, dx), (dw2, dw), (db2, db)))
    assert all(not t[:, 0].any() and not t[:, 1 + d:].any() for t in wide)
    far = torch.empty((1 << 26) * (T_ - 1) + d, dtype=torch.bfloat16, device="cuda").as_strided((T_, d), (1 << 26, 1))
    far.copy_(x)
    T.twell_layernorm_fwd(desc, far, w, b, far, stats2)
    assert torch.equal(far.contiguous(), y)


def test_formula_against_differences():
    """The gradient's formula, in 64 bits, against differences of the loss; and the kernel's gradient along a direction
    against differences of the kernel's own loss in fp32."""
    say("[gpu case] layer norm, differences")
    r = np.random.default_rng(0)
    x, dy, w, b = r.normal(size=(3, 11)), r.normal(size=(3, 11)), r.normal(size=11), r.normal(size=11)
    _, mean, rstd = layernorm(x, w, b, 1e-3)
    grads = layernorm_grads(x, w, mean, rstd, dy)

    def loss(x, w, b):
        return (layernorm(x, w, b, 1e-3)[0] * dy).sum()

    for i, v in enumerate((x, w, b)):
        for at in np.ndindex(v.shape):
            step = np.zeros(v.shape)
            step[at] = 1e-5
            args = [x, w, b]
            up, down = list(args), list(args)
            up[i], down[i] = v + step, v - step
            # truncation 1e-10 times third derivatives (of order 10), cancellation 1e-15 / 1e-5
            assert abs((loss(*up) - loss(*down)) / 2e-5 - grads[i][at]) < 1e-7
    T_, d, h = 8, 257, 2.0 ** -6
    xs, gs, ws_, bs = _data(T_, d, "fp32", "fp32", 3)
    v = torch.randn_like(xs)
    v = v / v.norm(dim=1, keepdim=True)
    desc = T.NormDesc(T_, d, "fp32")
    y, stats, dx, dw, db = _run(xs, gs, ws_, bs, "fp32")

    def kernel_loss(x):
        T.twell_layernorm_fwd(desc, x, ws_, bs, y)
        return (h64(y) * h64(gs)).sum()

    slope = (kernel_loss(xs + h * v) - kernel_loss(xs - h * v)) / (2 * h)
    # each element of y is off by up to 60 half steps of fp32 of values about 4 (their bound above), and 2 T d of them
    # add up with dy in a difference over 2 h; truncation is h^2 / 6 times a third derivative below |dy| |v|^3 rstd^3
    rounding = 60 * U32 * 4 * np.abs(h64(gs)).sum() / h
    truncation = h * h * np.abs(h64(gs)).sum()
    assert abs(slope - (h64(dx) * h64(v)).sum()) < rounding + truncation


def test_other_stream_and_replayed_graph():
    say("[gpu case] layer norm on a side stream and in a graph")
    T_, d = 3000, 1030
    x, dy, w, b = _data(T_, d, "bf16", "fp32", 11)
    want = _run(x, dy, w, b, "bf16")
    desc = T.NormDesc(T_, d, "bf16")
    out = [torch.empty_like(t) for t in want]
    y, stats, dx, dw, db = out
    ws = T.alloc_norm_ws(desc)

    def step():
        T.twell_layernorm_fwd(desc, x, w, b, y, stats)
        T.twell_layernorm_bwd(desc, x, w, stats, dy, dx, dw, db, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(out, want))
    graph = capture(step)
    for _ in range(3):
        for t in (*out, ws):
            t.view(torch.uint8).fill_(0xA5)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want))
