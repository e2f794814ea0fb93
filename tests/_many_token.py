"""64-bit references of the many-token operators, written from their definitions, and rounding bounds."""
import numpy as np
import torch

U32 = 2.0 ** -24  # half a step of fp32, relative
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def h64(t):
    return t.detach().double().cpu().numpy()


def order(ids, E):
    """offsets and pair_row by a loop over the pairs."""
    flat = ids.reshape(-1).tolist()
    lists = [[p for p, e in enumerate(flat) if e == x] for x in range(E)]
    offsets, pair_row, n = [0], [-1] * len(flat), 0
    for ps in lists:
        for p in ps:
            pair_row[p] = n
            n += 1
        offsets.append(n)
    return np.array(offsets, np.int32), np.array(pair_row, np.int32).reshape(ids.shape)


def order_fast(ids, E):
    """The same by a stable sort, for many pairs."""
    flat = ids.reshape(-1)
    key = np.where((flat >= 0) & (flat < E), flat, E)
    by = np.argsort(key, kind="stable")
    offsets = np.searchsorted(key[by], np.arange(E + 1)).astype(np.int32)
    pair_row = np.empty(len(flat), np.int32)
    pair_row[by] = np.where(key[by] < E, np.arange(len(flat)), -1)
    return offsets, pair_row.reshape(ids.shape)


def combine(rows, pair_row, w):
    """y and the sum of magnitudes behind each element of it."""
    T, k = pair_row.shape
    y, mag = np.zeros((T, rows.shape[1])), np.zeros((T, rows.shape[1]))
    for t in range(T):
        for i in range(k):
            if pair_row[t, i] >= 0 and w[t, i] != 0:
                y[t] += w[t, i] * rows[pair_row[t, i]]
                mag[t] += np.abs(w[t, i] * rows[pair_row[t, i]])
    return y, mag


def layernorm(x, w, b, eps):
    """y, mean, rstd."""
    mean = x.mean(1, keepdims=True)
    rstd = 1 / np.sqrt(((x - mean) ** 2).mean(1, keepdims=True) + eps)
    return (x - mean) * rstd * w + b, mean, rstd


def layernorm_grads(x, w, mean, rstd, dy):
    h = (x - mean) * rstd
    g = dy * w
    dx = rstd * (g - g.mean(1, keepdims=True) - h * (g * h).mean(1, keepdims=True))
    return dx, (dy * h).sum(0), dy.sum(0)


def check(got, want, bound, what):
    """|got - want| <= bound element by element."""
    got = h64(got) if isinstance(got, torch.Tensor) else got
    bad = ~(np.abs(got - want) <= bound)
    if bad.any():
        at = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} off, first at {at}: {got[at]!r}, expected {want[at]!r} "
                             f"within {np.broadcast_to(bound, got.shape)[at]!r}")


def capture(fn):
    """fn warmed up on a side stream, then captured into a graph."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fn()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fn()
    torch.cuda.synchronize()
    return g


# ----------------------------------------------------------------------------- 8-bit floating point
E4M3 = np.array([(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7) for e in range(16) for m in range(8)][:127])


def e4m3_nearest(v):
    """The nearest of e4m3's values to each |v| <= 448, ties to the even code; NaN stays."""
    a = np.abs(np.where(np.isnan(v), 0, v))
    hi = np.clip(np.searchsorted(E4M3, a), 1, 126)
    lo = hi - 1
    d = (a - E4M3[lo]) - (E4M3[hi] - a)
    code = np.where((d < 0) | ((d == 0) & (lo % 2 == 0)), lo, hi)
    return np.where(np.isnan(v), np.nan, np.copysign(E4M3[code], v))


def e4m3_scale(most):
    """The smallest power of two from 2^-126 on that takes magnitudes up to `most` to 448 or less."""
    s = np.full(np.shape(most), 2.0 ** -126)
    for e in range(-125, 121):
        s = np.where(most > 448 * s, 2.0 ** e, s)
    return s


def _finite(v):
    return np.where(np.isfinite(v), v, np.nan)


def e4m3_rows(x):
    """What rows stand for, a scale for each 128 of a row."""
    out = np.empty_like(x)
    for b in range(0, x.shape[1], 128):
        p = _finite(x[:, b:b + 128])
        s = e4m3_scale(np.abs(np.where(np.isnan(p), 0, p)).max(1, keepdims=True))
        out[:, b:b + 128] = e4m3_nearest(p / s) * s
    return out


def e4m3_weights(w):
    """What weights [N, K] stand for, a scale for each 128 x 128."""
    out = np.empty_like(w)
    for a in range(0, w.shape[0], 128):
        for b in range(0, w.shape[1], 128):
            p = _finite(w[a:a + 128, b:b + 128])
            s = e4m3_scale(np.abs(np.where(np.isnan(p), 0, p)).max())
            out[a:a + 128, b:b + 128] = e4m3_nearest(p / s) * s
    return out


def product_bound(x, w, y, dtype):
    """How far a product of codes x [T, K], w [N, K] may be off from y = x w^T: each product and its addition a half
    step of fp32 of the magnitudes' sum; in bf16 also what the matrix core cuts off (7 products of each 8 consecutive
    inputs, less than 2^-13 of the largest each) and the result's half step."""
    x, w = np.abs(x), np.abs(w)
    K = x.shape[1]
    e = (K + 8) * U32 * (x @ w.T)
    if dtype == "bf16":
        for k in range(0, K, 8):
            e += 7 * 2.0 ** -13 * (x[:, None, k:k + 8] * w[None, :, k:k + 8]).max(2)
    return 1.01 * e + HALF[dtype] * (np.abs(y) + 1.01 * e)
