"""Tokens sorted by expert and back, against plain references in 64 bits.

Bounds: an fp32 sum of n terms is off by at most n half steps of the sum of their magnitudes, a result rounded to its
dtype by half a step of that on top."""
import numpy as np
import pytest
import torch

from activation_sparse_feedforward_amd import twell as T
from _helpers import check_guards, guarded, say
from _many_token import DT, HALF, U32, capture, check, combine, h64, order, order_fast

pytestmark = pytest.mark.gpu


def _ids(T_, k, E, seed, dropped=0.0):
    r = np.random.default_rng(seed)
    ids = r.integers(0, E, (T_, k)).astype(np.int32)
    ids[r.random((T_, k)) < dropped] = -1
    return ids


def _sorted(desc, ids):
    o = T.TokensOrder(guarded((desc.experts + 1,), torch.int32), guarded((desc.T, desc.top_k), torch.int32))
    ws = guarded((desc.ws_bytes,), torch.uint8)
    T.twell_tokens_sort(desc, torch.from_numpy(ids).cuda(), o, ws)
    torch.cuda.synchronize()
    check_guards(*o, ws)
    return o


@pytest.mark.parametrize("T_,k,E", [(0, 2, 5), (1, 1, 1), (1, 8, 64), (1, 32, 3), (63, 1, 2), (64, 1, 2), (65, 3, 7),
                                    (1000, 4, 1024), (511, 8, 64), (513, 8, 64), (777, 5, 63), (1365, 3, 129)])
@pytest.mark.parametrize("dropped", [0.0, 0.3, 1.0])
def test_sort(T_, k, E, dropped):
    say(f"[gpu case] sort T={T_} k={k} E={E} dropped={dropped}")
    ids = _ids(T_, k, E, T_ + k + E, dropped)
    o = _sorted(T.TokensDesc(T_, 64, E, k, "bf16"), ids)
    offsets, pair_row = order(ids, E)
    assert np.array_equal(o.offsets.cpu().numpy(), offsets)
    assert np.array_equal(o.pair_row.cpu().numpy(), pair_row)


@pytest.mark.parametrize("T_,k,E", [(4096, 1, 8), (4097, 1, 8), (16384, 8, 64), (33333, 3, 1000), (200003, 6, 17),
                                    (1 << 20, 2, 256)])
def test_sort_over_several_workgroups(T_, k, E):
    say(f"[gpu case] sort T={T_} k={k} E={E}")
    ids = _ids(T_, k, E, 3, 0.1)
    ids[T_ // 2:T_ // 2 + 500] = E - 1  # a run of one expert
    o = _sorted(T.TokensDesc(T_, 64, E, k, "bf16"), ids)
    offsets, pair_row = order_fast(ids, E)
    assert np.array_equal(o.offsets.cpu().numpy(), offsets)
    assert np.array_equal(o.pair_row.cpu().numpy(), pair_row)


def test_sort_leaves_out_what_is_no_expert():
    say("[gpu case] sort with ids out of range")
    ids = np.array([[0, 5], [-1, 2], [2, -2 ** 31], [2 ** 31 - 1, 4], [2, 2]], np.int32)
    o = _sorted(T.TokensDesc(5, 64, 5, 2, "bf16"), ids)
    assert o.offsets.tolist() == [0, 1, 1, 5, 5, 6]
    assert o.pair_row.tolist() == [[0, -1], [-1, 1], [2, -1], [-1, 5], [3, 4]]


WIDTHS = [1, 7, 64, 255, 256, 257, 511, 513, 1001, 1024, 2048, 2056, 4099, 11008]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", WIDTHS)
def test_gather_combine_and_gradients(d, dtype):
    say(f"[gpu case] gather, combine, gradients d={d} {dtype}")
    T_, k, E = 37, 3, 5
    desc = T.TokensDesc(T_, d, E, k, dtype)
    _through(desc, _ids(T_, k, E, d, 0.2), d)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T_,k,E,dropped", [(1, 1, 1, 0.0), (1, 8, 64, 0.0), (3, 32, 40, 0.1), (5, 9, 2, 0.0),
                                            (130, 8, 16, 1.0), (129, 7, 300, 0.5), (2047, 3, 7, 0.2), (2048, 3, 7, 0.2)])
def test_gather_combine_and_gradients_by_choices(T_, k, E, dropped, dtype):
    say(f"[gpu case] gather, combine, gradients T={T_} k={k} E={E} dropped={dropped} {dtype}")
    _through(T.TokensDesc(T_, 320, E, k, dtype), _ids(T_, k, E, T_, dropped), k)


def _through(desc, ids, seed):
    T_, k, E, d, dt, half = desc.T, desc.top_k, desc.experts, desc.d_model, desc.torch_dtype, HALF[desc.dtype]
    P = T_ * k
    g = torch.Generator(device="cuda").manual_seed(seed)
    o = _sorted(desc, ids)
    pair_row = o.pair_row.cpu().numpy()
    live = int(o.offsets[-1])
    x, z, dy = (torch.randn(n, d, generator=g, device="cuda").to(dt) for n in (T_, P, T_))
    w = torch.rand(T_, k, generator=g, device="cuda")
    w[0, 0] = 0
    rows = guarded((P, d), dt)
    T.twell_tokens_gather(desc, x, o, rows)
    want = torch.zeros(P, d, dtype=dt)
    want.view(torch.uint8).fill_(0xA5)  # rows behind the last one stay as they were
    for p, r in enumerate(pair_row.reshape(-1)):
        if r >= 0:
            want[r] = x[p // k].cpu()
    assert torch.equal(rows.cpu().view(torch.uint8), want.view(torch.uint8))

    zh, wh, dyh = h64(z), h64(w), h64(dy)
    for weights, wv in ((w, wh), (None, np.ones((T_, k)))):
        y = guarded((T_, d), dt)
        T.twell_tokens_combine(desc, z, o, weights, y)
        ref, mag = combine(zh, pair_row, wv)
        check(y, ref, (k + 1) * U32 * mag + half * (np.abs(ref) + (k + 1) * U32 * mag), "y")
        check_guards(y)
    drows, dweights = guarded((P, d), dt), guarded((T_, k), torch.float32)
    T.twell_tokens_combine_bwd(desc, z, o, w, dy, drows, dweights)
    assert torch.equal(drows[live:].cpu().view(torch.uint8), want[live:].view(torch.uint8))
    got = h64(drows)
    for t in range(T_):
        for i in range(k):
            r = pair_row[t, i]
            if r < 0:
                assert float(dweights[t, i]) == 0
                continue
            v = wh[t, i] * dyh[t]
            check(got[r], v, (U32 + half) * 1.01 * np.abs(v), "drows")
            terms = zh[r] * dyh[t]
            check(float(dweights[t, i]), np.array(terms.sum()), (d / 64 + 24) * U32 * np.abs(terms).sum(), "dweights")
    check_guards(rows, drows, dweights)
    # each output alone, and into the rows themselves
    again, alone = torch.empty_like(drows), torch.empty_like(dweights)
    again.copy_(drows)
    T.twell_tokens_combine_bwd(desc, None, o, w, dy, again, None)
    T.twell_tokens_combine_bwd(desc, z, o, w, dy, None, alone)
    assert torch.equal(again.view(torch.uint8), drows.view(torch.uint8)) and torch.equal(alone, dweights)
    over, own = z.clone(), torch.empty_like(dweights)
    T.twell_tokens_combine_bwd(desc, over, o, w, dy, over, own)
    assert torch.equal(over[:live], drows[:live]) and torch.equal(own, dweights)
    assert torch.equal(over[live:], z[live:])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_strided_and_unaligned_rows(dtype):
    say(f"[gpu case] strided rows {dtype}")
    T_, k, E, d = 19, 2, 4, 301
    desc = T.TokensDesc(T_, d, E, k, dtype)
    ids = _ids(T_, k, E, 0, 0.1)
    o = _sorted(desc, ids)
    live = int(o.offsets[-1])
    base = [torch.randn(n, d + 9, device="cuda").to(DT[dtype]) for n in (T_, T_ * k, T_, T_ * k, T_)]
    x, z, dy, drows, y = (b[:, 3:3 + d] for b in base)
    w = torch.rand(T_, k, device="cuda")
    before = [b.clone() for b in base]
    plain = [torch.zeros(n, d, device="cuda", dtype=DT[dtype]) for n in (T_ * k, T_)]
    rows = torch.zeros(T_ * k, d + 1, device="cuda", dtype=DT[dtype])
    T.twell_tokens_gather(desc, x, o, rows[:, 1:])
    T.twell_tokens_gather(desc, x.contiguous(), o, plain[0])
    assert torch.equal(rows[:, 1:], plain[0]) and not rows[:, 0].any()
    T.twell_tokens_combine(desc, z, o, w, y)
    T.twell_tokens_combine(desc, z.contiguous(), o, w, plain[1])
    assert torch.equal(y, plain[1])
    dw, dw2 = torch.empty_like(w), torch.empty_like(w)
    T.twell_tokens_combine_bwd(desc, z, o, w, dy, drows, dw)
    T.twell_tokens_combine_bwd(desc, z.contiguous(), o, w, dy.contiguous(), plain[0], dw2)
    assert torch.equal(drows[:live], plain[0][:live]) and torch.equal(dw, dw2)
    for b, c in zip(base, before):  # nothing beside the rows
        assert torch.equal(b[:, :3], c[:, :3]) and torch.equal(b[:, 3 + d:], c[:, 3 + d:])
    assert torch.equal(drows[live:], before[3][live:, 3:3 + d])


# (first column, elements beside the row) of rows and of drows; None: no rows
@pytest.mark.parametrize("of_rows,of_drows", [((3, 9), (0, 0)), ((0, 0), (5, 11)), ((1, 2), (4, 40)), ((4, 40), (1, 2)),
                                              (None, (0, 0)), (None, (2, 7))])
@pytest.mark.parametrize("T_", [41, 2049])  # a wave a choice, a wave a token
@pytest.mark.parametrize("d", [301, 2600])  # dy kept in registers and read again, in both types
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gradients_into_rows_of_another_stride(dtype, d, T_, of_rows, of_drows):
    say(f"[gpu case] combine's gradients {dtype} T={T_} d={d} rows {of_rows} drows {of_drows}")
    k, E, dt = 2, 3, DT[dtype]
    P = T_ * k
    desc = T.TokensDesc(T_, d, E, k, dtype)
    o = _sorted(desc, _ids(T_, k, E, d, 0.1))
    live, pr = int(o.offsets[-1]), o.pair_row.view(-1).long()
    g = torch.Generator(device="cuda").manual_seed(d + T_)
    dy = torch.randn(T_, d, generator=g, device="cuda").to(dt)
    w = torch.rand(T_, k, generator=g, device="cuda")
    z = None
    if of_rows:
        z = torch.randn(P, d + of_rows[1], generator=g, device="cuda").to(dt)[:, of_rows[0]:of_rows[0] + d]
    first, beside = of_drows
    base, dweights = guarded((P, d + beside), dt), guarded((T_, k), torch.float32)
    drows = base[:, first:first + d]
    T.twell_tokens_combine_bwd(desc, z, o, w, dy, drows, dweights if of_rows else None)
    torch.cuda.synchronize()
    check_guards(base, dweights)
    kept = base.clone()
    kept.view(torch.uint8).fill_(0xA5)
    kept[:live, first:first + d] = drows[:live]
    assert torch.equal(base.view(torch.uint8), kept.view(torch.uint8)), "beside the rows or behind the last one"
    there = pr >= 0
    want = h64((dy.double()[:, None] * w.double()[..., None]).view(P, d)[there])
    check(drows[pr[there]], want, (U32 + HALF[dtype]) * 1.01 * np.abs(want), "drows")
    if of_rows:
        terms = torch.where(there[:, None], z.double()[pr.clamp(min=0)], 0).view(T_, k, d) * dy.double()[:, None]
        check(dweights, h64(terms.sum(-1)), h64((d / 64 + 24) * U32 * terms.abs().sum(-1)), "dweights")


def test_rows_beyond_32_bits():
    """Rows 2^26 elements apart: the last ones begin beyond 2^31 elements and 4 GiB."""
    say("[gpu case] rows beyond 4 GiB")
    T_, k, E, d, ld = 20, 2, 3, 40, 1 << 26
    desc = T.TokensDesc(T_, d, E, k, "bf16")
    o = _sorted(desc, _ids(T_, k, E, 1))
    x = torch.randn(T_, d, device="cuda").bfloat16()
    w = torch.rand(T_, k, device="cuda")
    near = torch.empty(T_ * k, d, device="cuda", dtype=torch.bfloat16)
    far = torch.empty(ld * (T_ * k - 1) + d, device="cuda", dtype=torch.bfloat16).as_strided((T_ * k, d), (ld, 1))
    T.twell_tokens_gather(desc, x, o, near)
    T.twell_tokens_gather(desc, x, o, far)
    assert torch.equal(near, far.contiguous())
    ys = [torch.empty_like(x) for _ in range(2)]
    dws = [torch.empty_like(w) for _ in range(2)]
    for rows, y, dw in zip((near, far), ys, dws):
        T.twell_tokens_combine(desc, rows, o, w, y)
        T.twell_tokens_combine_bwd(desc, rows, o, w, x, rows, dw)
    assert torch.equal(*ys) and torch.equal(*dws) and torch.equal(near, far.contiguous())


def test_what_is_left_out_is_not_read():
    """A weight of 0 and a pair left out add nothing, whatever rows hold; other rows carry infinities and NaN on."""
    say("[gpu case] NaN in rows that do not count")
    desc = T.TokensDesc(4, 100, 3, 2, "fp32")
    ids = np.array([[0, 1], [1, -1], [-1, -1], [2, 0]], np.int32)
    o = _sorted(desc, ids)
    pr = o.pair_row.tolist()
    z = torch.ones(8, 100, device="cuda")
    w = torch.ones(4, 2, device="cuda")
    z[pr[0][1]] = float("nan")
    w[0, 1] = 0
    z[pr[3][1], 5] = float("inf")
    z[5:] = float("nan")  # behind the last row
    y = torch.full((4, 100), 7.0, device="cuda")
    T.twell_tokens_combine(desc, z, o, w, y)
    assert torch.equal(y[0], torch.ones(100, device="cuda")) and torch.equal(y[1], torch.ones(100, device="cuda"))
    assert not y[2].any()
    assert torch.isinf(y[3, 5]) and torch.equal(y[3, :5], torch.full((5,), 2.0, device="cuda"))


def test_a_list_of_another_origin_stays_within_the_rows():
    say("[gpu case] rows out of range in pair_row")
    desc = T.TokensDesc(3, 64, 2, 2, "bf16")
    o = T.alloc_tokens_order(desc)
    o.pair_row.copy_(torch.tensor([[0, 6], [-7, 2 ** 31 - 1], [5, -2 ** 31]], dtype=torch.int32))
    x = torch.randn(3, 64, device="cuda").bfloat16()
    rows = guarded((6, 64), torch.bfloat16)
    T.twell_tokens_gather(desc, x, o, rows)
    check_guards(rows)
    assert torch.equal(rows[0], x[0]) and torch.equal(rows[5], x[2])
    y = torch.empty_like(x)
    T.twell_tokens_combine(desc, rows, o, None, y)
    assert torch.equal(y[0], x[0]) and not y[1].any() and torch.equal(y[2], x[2])


def test_gradients_agree_with_differences():
    """The loss sum(y dy) is linear in rows and in weights: its differences are its gradients, up to rounding."""
    say("[gpu case] differences")
    T_, k, E, d = 9, 3, 4, 33
    desc = T.TokensDesc(T_, d, E, k, "fp32")
    o = _sorted(desc, _ids(T_, k, E, 5, 0.2))
    live = int(o.offsets[-1])
    g = torch.Generator(device="cuda").manual_seed(1)
    z, vz = (torch.randn(T_ * k, d, generator=g, device="cuda") for _ in range(2))
    w, vw = (torch.rand(T_, k, generator=g, device="cuda") for _ in range(2))
    x, vx, dy = (torch.randn(T_, d, generator=g, device="cuda") for _ in range(3))
    y, drows, dw, dx = torch.empty_like(dy), torch.zeros_like(z), torch.empty_like(w), torch.empty_like(dy)

    def loss(z, w):
        T.twell_tokens_combine(desc, z, o, w, y)
        return (h64(y) * h64(dy)).sum(), (np.abs(h64(y)) * np.abs(h64(dy))).sum()

    T.twell_tokens_combine_bwd(desc, z, o, w, dy, drows, dw)
    for a, b, slope in ((loss(z + vz, w), loss(z - vz, w), (h64(drows)[:live] * h64(vz)[:live]).sum()),
                        (loss(z, w + vw), loss(z, w - vw), (h64(dw) * h64(vw)).sum())):
        # a sum of four terms, its inputs rounded once, in each loss and the gradient: 16 half steps
        assert abs((a[0] - b[0]) / 2 - slope) <= 16 * U32 * 4 * (a[1] + b[1])

    def moved(x):
        rows = torch.zeros_like(z)
        T.twell_tokens_gather(desc, x, o, rows)
        return (h64(rows)[:live] * h64(z)[:live]).sum(), np.abs(h64(rows)[:live] * h64(z)[:live]).sum()

    T.twell_tokens_combine(desc, z, o, None, dx)  # the gradient of gather
    a, b = moved(x + vx), moved(x - vx)
    assert abs((a[0] - b[0]) / 2 - (h64(dx) * h64(vx)).sum()) <= 16 * U32 * 4 * (a[1] + b[1])


def test_other_stream_and_replayed_graph():
    say("[gpu case] tokens on a side stream and in a graph")
    desc = T.TokensDesc(3000, 200, 16, 4, "bf16")
    g = torch.Generator(device="cuda").manual_seed(2)
    ids = [torch.from_numpy(_ids(3000, 4, 16, s, 0.1)).cuda() for s in (0, 1)]
    x, dy = (torch.randn(3000, 200, generator=g, device="cuda").bfloat16() for _ in range(2))
    w = torch.rand(3000, 4, generator=g, device="cuda")
    now = ids[0].clone()

    def buffers():
        return (T.alloc_tokens_order(desc), T.alloc_tokens_ws(desc), torch.zeros(12000, 200, device="cuda").bfloat16(),
                torch.zeros(3000, 200, device="cuda").bfloat16(), torch.zeros(12000, 200, device="cuda").bfloat16(),
                torch.zeros(3000, 4, device="cuda"))

    def step(b, ids):
        o, ws, rows, y, drows, dw = b
        T.twell_tokens_sort(desc, ids, o, ws)
        T.twell_tokens_gather(desc, x, o, rows)
        T.twell_tokens_combine(desc, rows, o, w, y)
        T.twell_tokens_combine_bwd(desc, rows, o, w, dy, drows, dw)

    def results(b):
        o, _, rows, y, drows, dw = b
        n = int(o.offsets[-1])
        return [t.clone() for t in (*o, rows[:n], y, drows[:n], dw)]

    want = []
    for i in ids:
        b = buffers()
        step(b, i)
        want.append(results(b))
    b = buffers()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(b, ids[0])
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(results(b), want[0]))
    b = buffers()
    graph = capture(lambda: step(b, now))
    for turn in (1, 0, 1):
        now.copy_(ids[turn])
        for t in (*b[0], b[1], *b[2:]):
            t.view(torch.uint8).fill_(0x3C)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(results(b), want[turn])), turn
