"""Products with weights in 8-bit floating point, against plain references in 64 bits on the same codes."""
import numpy as np
import pytest
import torch

from activation_sparse_feedforward_amd import twell as T
from _helpers import check_guards, guarded, say
from _many_token import (DT, E4M3, U32, capture, check, e4m3_nearest, e4m3_rows, e4m3_scale, e4m3_weights, h64,
                         product_bound)

pytestmark = pytest.mark.gpu


def _planes(desc):
    codes, scales = desc.plane_bytes
    return T.Weights(guarded((codes,), torch.uint8), guarded((scales,), torch.uint8))


def _packed(desc, w, both=True):
    p, t = _planes(desc), _planes(desc.transposed) if both else None
    T.twell_fp8_weights_pack(desc, w, p, t)
    torch.cuda.synchronize()
    check_guards(*p, *(t or ()))
    return p, t


def _values(desc, planes, dtype=torch.float32):
    out = guarded((desc.experts, desc.rows, desc.cols), dtype)
    T.twell_fp8_weights_unpack(desc, planes, out)
    torch.cuda.synchronize()
    check_guards(out)
    return out


def test_reference_rounds_as_the_format_says():
    """The reference's own rounding: e4m3's values, and halves between them to the even code."""
    mid = (E4M3[:-1] + E4M3[1:]) / 2
    got = e4m3_nearest(mid)
    assert np.array_equal(got, np.where(np.arange(126) % 2 == 0, E4M3[:-1], E4M3[1:]))
    assert np.array_equal(e4m3_nearest(E4M3), E4M3) and E4M3[-1] == 448 and E4M3[1] == 2.0 ** -9


SHAPES = [(1, 1, 1), (1, 16, 128), (2, 17, 129), (1, 128, 128), (3, 100, 300), (1, 257, 515), (2, 129, 1030), (1, 5, 2000)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("E,N,K", SHAPES)
def test_weights_there_and_back(E, N, K, dtype):
    say(f"[gpu case] fp8 weights {E} x {N} x {K} {dtype}")
    g = torch.Generator(device="cuda").manual_seed(N + K)
    # blocks of very different sizes
    w = torch.randn(E, N, K, generator=g, device="cuda") * torch.exp(4 * torch.randn(E, 1, K, generator=g, device="cuda"))
    w = w.to(DT[dtype])
    desc = T.Fp8Desc(E, N, K)
    p, t = _packed(desc, w)
    want = np.stack([e4m3_weights(m) for m in h64(w)])
    assert np.array_equal(h64(_values(desc, p)), want)
    assert np.array_equal(h64(_values(desc.transposed, t)), want.transpose(0, 2, 1))
    assert np.array_equal(h64(_values(desc, p, torch.bfloat16)), want)  # four bits of a bf16's eight
    alone, _ = _packed(desc, w.view(-1), both=False)
    assert torch.equal(alone.codes, p.codes)


def _scale_bytes(v, codes_rows, blocks):
    """Scale bytes of one matrix's planes, [tiles of 16 rows][4 blocks][16 rows][4], from its values [rows, cols]."""
    tiles, quads = -(-codes_rows // 16), -(-blocks // 4)
    out = np.zeros((tiles, quads, 16, 4), np.uint8)
    for a in range(0, codes_rows, 128):
        for b in range(blocks):
            most = np.abs(v[a:a + 128, 128 * b:128 * b + 128]).max()
            out[a // 16:a // 16 + 8, b // 4, :, b % 4] = 127 + int(np.log2(e4m3_scale(most)))
    return out


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("E,N,K", SHAPES + [(2, 500, 640), (1, 512, 512)])
def test_planes_are_written_whole(E, N, K, dtype):
    """Every byte of codes and scales comes from the weights: 128 x 128 weights share a scale, in all of their rows,
    and blocks that only fill up the last four have zeros."""
    say(f"[gpu case] fp8 planes {E} x {N} x {K} {dtype}")
    g = torch.Generator(device="cuda").manual_seed(N + K)
    w = torch.randn(E, N, K, generator=g, device="cuda") * torch.exp(4 * torch.randn(E, 1, K, generator=g, device="cuda"))
    w = w.to(DT[dtype])
    desc = T.Fp8Desc(E, N, K)
    p, t = _packed(desc, w)  # over bytes of 0xA5
    q, u = _planes(desc), _planes(desc.transposed)
    for plane in (*q, *u):
        plane.fill_(0x3C)
    T.twell_fp8_weights_pack(desc, w, q, u)
    alone = _planes(desc)
    T.twell_fp8_weights_pack(desc, w, alone)
    torch.cuda.synchronize()
    check_guards(*q, *u, *alone)
    assert torch.equal(p.codes, q.codes) and torch.equal(t.codes, u.codes) and torch.equal(p.codes, alone.codes)
    wh = h64(w)
    want = np.stack([_scale_bytes(m, N, -(-K // 128)) for m in wh])
    want_t = np.stack([_scale_bytes(m.T, K, -(-N // 128)) for m in wh])
    for got in (p, q, alone):
        assert np.array_equal(got.scales.cpu().numpy(), want.reshape(-1))
    for got in (t, u):
        assert np.array_equal(got.scales.cpu().numpy(), want_t.reshape(-1))


def test_rounding_of_every_value_and_border():
    """All codes, the halves between them and their neighbours, over several powers of two; both types."""
    say("[gpu case] fp8 rounding")
    vals = [v for a, b in zip(E4M3[:-1], E4M3[1:]) for v in (a, (a + b) / 2)]
    vals = np.array(vals + list(np.nextafter(np.float32(vals), np.float32(1e9)).astype(float))
                    + list(np.nextafter(np.float32(vals), np.float32(-1)).astype(float)) + [448.0])
    vals = np.concatenate([vals, -vals])
    n = -(-len(vals) // 127)
    for e in (-100, -7, 0, 9, 110):
        x = np.zeros((n, 128))
        x[:, 0] = 448.0  # sets the scale
        flat = np.zeros(n * 127)
        flat[:len(vals)] = vals
        x[:, 1:] = flat.reshape(n, 127)
        w32 = torch.from_numpy((x * 2.0 ** e).astype(np.float32))
        for w in (w32, w32.bfloat16()):
            desc = T.Fp8Desc(n, 1, 128)
            p, _ = _packed(desc, w.view(n, 1, 128).cuda(), both=False)
            assert np.array_equal(h64(_values(desc, p))[:, 0], e4m3_rows(h64(w))), e


def test_scales_at_the_ends_and_non_finite_weights():
    say("[gpu case] fp8 scales at the ends of the range")
    w = torch.zeros(6, 128, 128)
    w[0, 3, 5] = 3.4e38
    w[1] = 2.0 ** -126 * torch.rand(128, 128)  # below what the smallest scale takes to a code of its own size
    w[2, 0] = torch.arange(128) * 2.0 ** -149
    w[3] = torch.randn(128, 128)
    w[3, 7, 7], w[3, 8, 8], w[3, 9, 9] = float("inf"), float("-inf"), float("nan")
    w[4, 0, 0] = 448.0
    w[4, 0, 1] = 1.0
    w[5, 0, 0] = 449.0
    w[5, 0, 1] = 1.0
    desc = T.Fp8Desc(6, 128, 128)
    p, t = _packed(desc, w.cuda())
    want = np.stack([e4m3_weights(m) for m in h64(w)])
    want[0, 3, 5] = np.inf  # 256 * 2^120 = 2^128
    got = h64(_values(desc, p))
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.isnan(got).sum() == 3
    assert np.array_equal(np.nan_to_num(got, nan=0.0), np.nan_to_num(want, nan=0.0))
    assert np.array_equal(np.nan_to_num(h64(_values(desc.transposed, t)), nan=5.0).transpose(0, 2, 1),
                          np.nan_to_num(got, nan=5.0))


def _offsets(counts, T_):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32).cuda()


def _case(T_, N, K, dtype, counts=None, seed=0, spread=2.0):
    """Forward and both gradients against 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    E = 1 if counts is None else len(counts)
    desc = T.Fp8Desc(E, N, K)
    w = torch.randn(E, N, K, generator=g, device="cuda") * K ** -0.5
    size = torch.exp(spread * torch.randn(T_, 1, generator=g, device="cuda"))  # rows of different sizes
    x = (torch.randn(T_, K, generator=g, device="cuda") * size).to(DT[dtype])
    dy = (torch.randn(T_, N, generator=g, device="cuda") * size).to(DT[dtype])
    off = None if counts is None else _offsets(counts, T_)
    p, t = _packed(desc, w)
    y, dx = guarded((T_, N), DT[dtype]), guarded((T_, K), DT[dtype])
    dw = guarded((E, N, K), torch.float32)
    ws = guarded((T.fp8_ws_bytes(desc, T_),), torch.uint8)
    T.twell_fp8_linear_fwd(desc, p, x, y, ws, offsets=off)
    T.twell_fp8_linear_bwd(desc, t, x, dy, dx, dw, ws, offsets=off)
    torch.cuda.synchronize()
    check_guards(y, dx, dw, ws)
    wv = np.stack([e4m3_weights(m) for m in h64(w)])
    xh, gh = h64(x), h64(dy)
    qx, qg = e4m3_rows(xh), e4m3_rows(gh)
    yh, dxh, dwh = h64(y), h64(dx), h64(dw)
    bounds = [0, T_] if counts is None else np.concatenate([[0], np.cumsum(counts)])
    for e in range(E):
        a, b = bounds[e], bounds[e + 1]
        if b > a:
            ref = qx[a:b] @ wv[e].T
            check(yh[a:b], ref, product_bound(qx[a:b], wv[e], ref, dtype), f"y of expert {e}")
            ref = qg[a:b] @ wv[e]
            check(dxh[a:b], ref, product_bound(qg[a:b], wv[e].T, ref, dtype), f"dx of expert {e}")
        mag = np.abs(gh[a:b]).T @ np.abs(xh[a:b])
        check(dwh[e], gh[a:b].T @ xh[a:b], (b - a + 8) * U32 * mag, f"dw of expert {e}")
    behind = [v[bounds[-1]:].contiguous().view(torch.uint8) for v in (y, dx)]
    assert all(bool((v == 0xA5).all()) for v in behind), "rows behind the last one"
    # one gradient alone is the same
    for d1, d2 in ((torch.full_like(dx, 3.0), None), (None, torch.empty_like(dw))):
        T.twell_fp8_linear_bwd(desc, t if d2 is None else None, x if d1 is None else None, dy, d1, d2, ws, offsets=off)
        n = int(bounds[-1])
        assert torch.equal(d1[:n], dx[:n]) if d2 is None else torch.equal(d2, dw)
    return desc, p, t, x, dy, off, y, dx, dw


ROWS = [1, 2, 7, 15, 16, 17, 31, 33, 64, 65, 100, 127, 129, 257, 300]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T_", ROWS)
def test_rows(T_, dtype):
    say(f"[gpu case] fp8 product T={T_} {dtype}")
    _case(T_, 200, 330, dtype, seed=T_)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N,K", [(1, 1), (1, 128), (16, 64), (15, 129), (128, 128), (127, 512), (130, 513), (300, 1100),
                                 (513, 24), (64, 2049)])
def test_widths(N, K, dtype):
    say(f"[gpu case] fp8 product N={N} K={K} {dtype}")
    for T_ in (1, 5, 40, 140):
        _case(T_, N, K, dtype, seed=N + K)


COUNTS = [[0, 0, 0], [1, 0, 0], [0, 1], [3, 0, 5, 1], [16, 16], [17, 15, 1, 0, 33], [0, 130, 0, 0, 1, 127, 128, 129, 0],
          [1] * 70, [300, 2]]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("tail", [0, 9])
def test_experts(counts, tail, dtype):
    say(f"[gpu case] fp8 experts {counts} tail {tail} {dtype}")
    T_ = sum(counts) + tail
    if T_:
        _case(T_, 150, 260, dtype, counts, seed=len(counts))


@pytest.mark.parametrize("T_,N,K,counts", [(520, 600, 1000, None), (700, 260, 512, [300, 1, 0, 380]), (4500, 64, 96, None),
                                           (2100, 384, 640, [1000, 0, 600, 300, 128, 64]), (3000, 100, 136, [2900, 0])])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_more_rows(T_, N, K, counts, dtype):
    say(f"[gpu case] fp8 product T={T_} N={N} K={K} {counts} {dtype}")
    _case(T_, N, K, dtype, counts, seed=T_)


# one or more for each kernel that the launcher chooses among: rounding on the way with few to many workgroups,
# codes in small and larger tiles, tiles through LDS of 64 and 128 rows (fp32: 128 x 128)
@pytest.mark.parametrize("T_,N,K,counts", [(15, 8180, 130, None), (100, 2000, 300, None), (50, 620, 250, [1, 3] * 10 + [0] * 20),
                                           (470, 250, 400, [2, 1, 0] * 150), (250, 500, 8200, None),
                                           (1020, 1020, 2100, None), (3000, 1030, 650, None), (4200, 1030, 520, None),
                                           (4000, 1100, 300, [1400, 0, 70, 2520])])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_each_kernel_of_the_products(T_, N, K, counts, dtype):
    say(f"[gpu case] fp8 product T={T_} N={N} K={K} {dtype} of {len(counts or [0])} experts")
    _case(T_, N, K, dtype, counts, seed=T_)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T_,N,K,counts", [(3, 4096, 300, None), (3, 4097, 300, None), (3, 8192, 300, None),
                                           (3, 8193, 300, None), (3, 16384, 300, None), (3, 16385, 300, None),
                                           (40, 1360, 1200, None), (40, 1370, 1200, None), (6, 510, 2100, [2, 0, 1, 3]),
                                           (6, 1030, 2100, [2, 0, 1, 3])])
def test_borders_between_kernels_of_few_rows(T_, N, K, counts, dtype):
    """On both sides of 128, 256 and 512 tiles of 16 rows x 32 outputs."""
    say(f"[gpu case] fp8 product T={T_} N={N} K={K} {dtype} at a border")
    _case(T_, N, K, dtype, counts, seed=N)


def test_many_experts():
    say("[gpu case] fp8 1024 experts")
    r = np.random.default_rng(0)
    counts = r.integers(0, 4, 1024)
    counts[500:700] = 0
    _case(int(counts.sum()) + 3, 40, 130, "bf16", counts.tolist())


def test_one_expert_with_offsets_and_rows_before():
    """Rows before the first expert's are left as they are, too."""
    say("[gpu case] fp8 offsets of one expert")
    desc = T.Fp8Desc(1, 100, 200)
    w = torch.randn(1, 100, 200, device="cuda")
    p, t = _packed(desc, w)
    x, dy = torch.randn(90, 200, device="cuda").bfloat16(), torch.randn(90, 100, device="cuda").bfloat16()
    ws = T.alloc_fp8_ws(desc, 90)
    off = torch.tensor([20, 57], dtype=torch.int32, device="cuda")
    y, part = (torch.full((n, 100), 7.0, device="cuda", dtype=torch.bfloat16) for n in (90, 37))
    T.twell_fp8_linear_fwd(desc, p, x, y, ws, offsets=off)
    T.twell_fp8_linear_fwd(desc, p, x[20:57], part, ws)
    assert torch.equal(y[20:57], part) and bool((y[:20] == 7).all()) and bool((y[57:] == 7).all())
    dw, dw2 = torch.empty(1, 100, 200, device="cuda"), torch.empty(1, 100, 200, device="cuda")
    T.twell_fp8_linear_bwd(desc, None, x, dy, None, dw, ws, offsets=off)
    T.twell_fp8_linear_bwd(desc, None, x[20:57], dy[20:57], None, dw2, ws)
    check(dw, h64(dw2), 64 * U32 * (np.abs(h64(dy)).T @ np.abs(h64(x))), "dw")


@pytest.mark.parametrize("off", [[0, 50, 20, 30], [-5, 3, 9, 1000], [90, 80, 70, 60], [5, 5, 2 ** 31 - 1, -2 ** 31]])
def test_offsets_of_another_origin_stay_within_the_rows(off):
    say(f"[gpu case] fp8 offsets {off}")
    desc = T.Fp8Desc(3, 64, 128)
    p, t = _packed(desc, torch.randn(3, 64, 128, device="cuda"))
    x, dy = torch.randn(40, 128, device="cuda").bfloat16(), torch.randn(40, 64, device="cuda").bfloat16()
    y, dx, dw = guarded((40, 64), torch.bfloat16), guarded((40, 128), torch.bfloat16), guarded((3, 64, 128), torch.float32)
    ws = guarded((T.fp8_ws_bytes(desc, 40),), torch.uint8)
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    T.twell_fp8_linear_fwd(desc, p, x, y, ws, offsets=o)
    T.twell_fp8_linear_bwd(desc, t, x, dy, dx, dw, ws, offsets=o)
    torch.cuda.synchronize()
    check_guards(y, dx, dw, ws)


def test_no_rows():
    say("[gpu case] fp8 of no rows")
    for E in (1, 4):
        desc = T.Fp8Desc(E, 70, 90)
        p, t = _packed(desc, torch.randn(E, 70, 90, device="cuda"))
        x, dy = (torch.empty(0, n, dtype=torch.bfloat16, device="cuda") for n in (90, 70))
        off = torch.zeros(E + 1, dtype=torch.int32, device="cuda") if E > 1 else None
        ws, dw = T.alloc_fp8_ws(desc, 0), guarded((E, 70, 90), torch.float32)
        T.twell_fp8_linear_fwd(desc, p, x, dy.clone(), ws, offsets=off)
        T.twell_fp8_linear_bwd(desc, t, x, dy, x.clone(), dw, ws, offsets=off)
        torch.cuda.synchronize()
        assert not dw.any()
        check_guards(dw)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_strided_and_unaligned_rows(dtype):
    say(f"[gpu case] fp8 strided rows {dtype}")
    for T_, counts in ((5, None), (200, [90, 0, 101])):
        N, K = 131, 257
        desc, p, t, x, dy, off, y, dx, dw = _case(T_, N, K, dtype, counts, seed=1)
        wide = [torch.zeros(T_, n + 7, device="cuda", dtype=DT[dtype]) for n in (K, N, N, K)]
        xs, dys, ys, dxs = (v[:, 3:-4] for v in wide)
        xs.copy_(x)
        dys.copy_(dy)
        ws, dws = T.alloc_fp8_ws(desc, T_), torch.empty_like(dw)
        T.twell_fp8_linear_fwd(desc, p, xs, ys, ws, offsets=off)
        T.twell_fp8_linear_bwd(desc, t, xs, dys, dxs, dws, ws, offsets=off)
        n = T_ if off is None else int(off[-1])
        assert torch.equal(ys[:n], y[:n]) and torch.equal(dxs[:n], dx[:n]) and torch.equal(dws, dw)
        assert all(not v[:, :3].any() and not v[:, -4:].any() for v in wide)


def test_rows_beyond_32_bits():
    say("[gpu case] fp8 rows beyond 4 GiB")
    T_, N, K, ld = 40, 64, 130, 1 << 26
    for counts in (None, [10, 30]):
        desc, p, t, x, dy, off, y, dx, dw = _case(T_, N, K, "bf16", counts, seed=2)
        far = torch.empty(ld * (T_ - 1) + 1024, dtype=torch.bfloat16, device="cuda")
        xs, ys = far.as_strided((T_, K), (ld, 1)), far.as_strided((T_, N), (ld, 1), 200)
        dys, dxs = far.as_strided((T_, N), (ld, 1), 300), far.as_strided((T_, K), (ld, 1), 400)
        xs.copy_(x)
        dys.copy_(dy)
        ws, dws = T.alloc_fp8_ws(desc, T_), torch.empty_like(dw)
        T.twell_fp8_linear_fwd(desc, p, xs, ys, ws, offsets=off)
        T.twell_fp8_linear_bwd(desc, t, xs, dys, dxs, dws, ws, offsets=off)
        assert torch.equal(ys.contiguous(), y) and torch.equal(dxs.contiguous(), dx) and torch.equal(dws, dw)
        del far, xs, ys, dys, dxs


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T_", [4, 150])
def test_non_finite_inputs_stay_in_their_row(T_, dtype):
    say(f"[gpu case] fp8 NaN and infinities T={T_} {dtype}")
    desc, p, t, x, dy, off, y, dx, dw = _case(T_, 140, 300, dtype, seed=3, spread=0.5)
    x, dy = x.clone(), dy.clone()
    x[1, 130], x[3, 299], dy[1, 0], dy[2, 139] = float("nan"), float("inf"), float("-inf"), float("nan")
    y2, dx2, ws = torch.empty_like(y), torch.empty_like(dx), T.alloc_fp8_ws(desc, T_)
    T.twell_fp8_linear_fwd(desc, p, x, y2, ws)
    T.twell_fp8_linear_bwd(desc, t, x, dy, dx2, None, ws)
    bad_y, bad_dx = [1, 3], [1, 2]
    assert torch.isnan(y2[bad_y]).all() and torch.isnan(dx2[bad_dx]).all()
    good_y, good_dx = ([i for i in range(T_) if i not in b] for b in (bad_y, bad_dx))
    assert torch.equal(y2[good_y], y[good_y]) and torch.equal(dx2[good_dx], dx[good_dx])


def test_rows_of_very_different_sizes_and_zeros():
    """A row of zeros gives zeros; scales from 2^-126 to 2^100 meet in one product."""
    say("[gpu case] fp8 scales far apart")
    desc = T.Fp8Desc(1, 64, 256)
    w = torch.randn(1, 64, 256, device="cuda")
    w[:, :, 128:] *= 2.0 ** -20
    for dtype in ("bf16", "fp32"):
        p, _ = _packed(desc, w)
        for T_ in (6, 60):
            x = torch.randn(T_, 256, device="cuda")
            x[0] = 0
            x[1] *= 2.0 ** -120
            x[2] *= 2.0 ** 100
            x[3, :128] *= 2.0 ** -60
            x[4, :128] = 0
            x = x.to(DT[dtype])
            y = torch.empty(T_, 64, device="cuda", dtype=DT[dtype])
            T.twell_fp8_linear_fwd(desc, p, x, y, T.alloc_fp8_ws(desc, T_))
            q, wv = e4m3_rows(h64(x)), e4m3_weights(h64(w)[0])
            ref = q @ wv.T
            check(y, ref, product_bound(q, wv, ref, dtype) + 2.0 ** -126, "y")  # products below 2^-126 may become 0
            assert not y[0].any()


def test_gradients_against_differences():
    """With codes that hold x, W and dy exactly the product is linear: differences of the loss are the gradients."""
    say("[gpu case] fp8 differences")
    g = torch.Generator().manual_seed(0)

    def ints(*s):
        return torch.randint(-3, 4, s, generator=g).float().cuda()

    counts, N, K = [20, 0, 13], 33, 40
    T_ = sum(counts)
    desc, off = T.Fp8Desc(3, N, K), _offsets(counts, T_)
    x, vx, w, vw, dy = ints(T_, K), ints(T_, K), ints(3, N, K), ints(3, N, K), ints(T_, N)
    ws = T.alloc_fp8_ws(desc, T_)

    def loss(x, w):
        p, _ = _packed(desc, w)
        y = torch.empty(T_, N, device="cuda")
        T.twell_fp8_linear_fwd(desc, p, x, y, ws, offsets=off)
        return (h64(y) * h64(dy)).sum()

    _, t = _packed(desc, w)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    T.twell_fp8_linear_bwd(desc, t, x, dy, dx, dw, ws, offsets=off)
    # whole numbers up to 6 are codes, and all sums here are whole numbers below 2^24: nothing is rounded
    assert (loss(x + vx, w) - loss(x - vx, w)) / 2 == (h64(dx) * h64(vx)).sum()
    assert (loss(x, w + vw) - loss(x, w - vw)) / 2 == (h64(dw) * h64(vw)).sum()


@pytest.mark.parametrize("T_,counts", [(3, None), (900, [400, 0, 350, 100])])
def test_other_stream_and_replayed_graph(T_, counts):
    say(f"[gpu case] fp8 on a side stream and in a graph, T={T_}")
    desc, p, t, x, dy, off, y, dx, dw = _case(T_, 300, 400, "bf16", counts, seed=4)
    n = T_ if off is None else int(off[-1])
    out = [torch.zeros_like(v) for v in (y, dx, dw)]
    ws = T.alloc_fp8_ws(desc, T_)

    def step():
        T.twell_fp8_linear_fwd(desc, p, x, out[0], ws, offsets=off)
        T.twell_fp8_linear_bwd(desc, t, x, dy, out[1], out[2], ws, offsets=off)

    def same():
        return torch.equal(out[0][:n], y[:n]) and torch.equal(out[1][:n], dx[:n]) and torch.equal(out[2], dw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    assert same()
    graph = capture(step)
    for _ in range(3):
        for v in (*out, ws):
            v.view(torch.uint8).fill_(0x3C)
        graph.replay()
        torch.cuda.synchronize()
        assert same()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T_,N,K,counts", [(600, 2000, 2600, None), (1020, 1020, 2100, None), (4200, 1030, 520, None),
                                           (4000, 1100, 300, [1400, 0, 70, 2520]), (9000, 1100, 300, [3000, 5000, 999]),
                                           (16500, 2040, 1030, None)])
def test_kernels_of_many_rows_in_other_places(T_, N, K, counts, dtype):
    """Rows of other strides, NaN and infinities, replays with other work between them, and offsets of another origin:
    each kernel that reads codes of rows, against its own results for the same rows."""
    say(f"[gpu case] fp8 T={T_} N={N} K={K} {dtype} in other places")
    g = torch.Generator(device="cuda").manual_seed(T_)
    E = 1 if counts is None else len(counts)
    desc = T.Fp8Desc(E, N, K)
    p, _ = _packed(desc, torch.randn(E, N, K, generator=g, device="cuda"), both=False)
    x = torch.randn(T_, K, generator=g, device="cuda").to(DT[dtype])
    off = None if counts is None else _offsets(counts, T_)
    n = T_ if counts is None else sum(counts)
    ws = guarded((T.fp8_ws_bytes(desc, T_),), torch.uint8)
    y, again = (guarded((T_, N), DT[dtype]) for _ in range(2))
    T.twell_fp8_linear_fwd(desc, p, x, y, ws, offsets=off)
    check_guards(y, ws)
    assert bool((y[n:].contiguous().view(torch.uint8) == 0xA5).all())

    wide = [torch.zeros(T_, m + 7, device="cuda", dtype=DT[dtype]) for m in (K, N)]
    xs, ys = (v[:, 3:-4] for v in wide)
    xs.copy_(x)
    T.twell_fp8_linear_fwd(desc, p, xs, ys, ws, offsets=off)
    assert torch.equal(ys[:n], y[:n]) and not any(bool(v[:, :3].any() | v[:, -4:].any()) for v in wide)

    bad = x.clone()
    bad[1, K - 1], bad[n - 2, 0], bad[n // 2, K // 2] = float("nan"), float("inf"), float("-inf")
    T.twell_fp8_linear_fwd(desc, p, bad, again, ws, offsets=off)
    rows = torch.zeros(n, dtype=torch.bool, device="cuda")
    rows[[1, n - 2, n // 2]] = True
    assert torch.isnan(again[:n][rows]).all() and torch.equal(again[:n][~rows], y[:n][~rows])

    graph = capture(lambda: T.twell_fp8_linear_fwd(desc, p, x, again, ws, offsets=off))
    for _ in range(3):
        again.fill_(3.0)
        ws.fill_(0x3C)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(again[:n], y[:n])

    if counts is not None:
        for o in ([T_] * E + [0], [0, T_, 5, T_, 9][:E + 1], [-9] + [2 ** 31 - 1] * E, list(range(7, 7 + E + 1))):
            T.twell_fp8_linear_fwd(desc, p, x, again, ws, offsets=torch.tensor(o, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    check_guards(again, ws)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_most_rows(dtype):
    """2^20 rows, the most there may be, of two widths."""
    for N, K in ((8, 8), (40, 136)):
        say(f"[gpu case] fp8 2^20 rows, {N} x {K} {dtype}")
        desc = T.Fp8Desc(1, N, K)
        p, t = _packed(desc, torch.randn(1, N, K, device="cuda"))
        x, dy = (torch.randn(1 << 20, m, device="cuda").to(DT[dtype]) for m in (K, N))
        ws, y, dx, dw = T.alloc_fp8_ws(desc, 1 << 20), torch.empty_like(dy), torch.empty_like(x), torch.empty(1, N, K, device="cuda")
        T.twell_fp8_linear_fwd(desc, p, x, y, ws)
        T.twell_fp8_linear_bwd(desc, t, x, dy, dx, dw, ws)
        some = torch.cat([torch.arange(40), torch.arange((1 << 20) - 40, 1 << 20), torch.randint(1 << 20, (200,))]).cuda()
        wv = h64(_values(desc, p))[0]
        for got, of, m in ((y, x, wv.T), (dx, dy, wv)):
            q = e4m3_rows(h64(of[some]))
            check(got[some], q @ m, product_bound(q, m.T, q @ m, dtype), "rows")
        ref, mag = dy.double().t() @ x.double(), dy.double().abs().t() @ x.double().abs()
        check(dw[0], h64(ref), (2 ** 20 + 8) * U32 * h64(mag), "dw")


@pytest.mark.parametrize("T_,N,K,counts", [(16500, 2040, 1030, None), (33000, 1030, 1152, None),
                                           (17000, 2100, 1100, [9000, 0, 7, 7900])])
def test_results_past_the_caches(T_, N, K, counts):
    """bf16 results of 64 MB and more, of 8 blocks of inputs and more, against 64 bits: first and last rows, the ends of
    tiles and of experts, others at random; whole groups of 64 outputs and the part of one behind them."""
    say(f"[gpu case] fp8 T={T_} N={N} K={K} {counts} past the caches")
    assert T_ * N >= 1 << 25 and K > 7 * 128 and N % 64
    g = torch.Generator(device="cuda").manual_seed(T_)
    E = 1 if counts is None else len(counts)
    desc = T.Fp8Desc(E, N, K)
    w = torch.randn(E, N, K, generator=g, device="cuda") * K ** -0.5
    p, _ = _packed(desc, w, both=False)
    x = torch.randn(T_, K, generator=g, device="cuda") * torch.exp(2 * torch.randn(T_, 1, generator=g, device="cuda"))
    x = x.bfloat16()
    off = None if counts is None else _offsets(counts, T_)
    y, ws = guarded((T_, N), torch.bfloat16), guarded((T.fp8_ws_bytes(desc, T_),), torch.uint8)
    T.twell_fp8_linear_fwd(desc, p, x, y, ws, offsets=off)
    torch.cuda.synchronize()
    check_guards(y, ws)
    ends = np.concatenate([[0], np.cumsum(counts if counts else [T_])])
    assert bool((y[ends[-1]:].contiguous().view(torch.uint8) == 0xA5).all())
    r = np.random.default_rng(T_)
    for e in range(E):
        a, b = int(ends[e]), int(ends[e + 1])
        if a == b:
            continue
        rows = np.concatenate([np.arange(a, a + 20), np.arange(a + 120, a + 136), np.arange(b - 140, b),
                               r.integers(a, b, 64)])
        rows = np.unique(rows[(rows >= a) & (rows < b)])
        q, wv = e4m3_rows(h64(x[rows])), e4m3_weights(h64(w[e]))
        ref = q @ wv.T
        check(y[rows], ref, product_bound(q, wv, ref, "bf16"), f"y of expert {e}")
