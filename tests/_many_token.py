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
