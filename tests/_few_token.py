"""64-bit references of the few-token operators, written from their definitions."""
import numpy as np
import torch


def planes_to_codes(codes: np.ndarray, scales: np.ndarray, E, N, K, group):
    """Codes q and fp32 scales per weight, read from the planes by the documented layout."""
    tiles, blocks = -(-N // 16), -(-K // 128)
    words = codes.view(np.uint32).reshape(E, tiles, blocks, 64, 4)
    words = (words >> 3) | (words << 29)  # stored rotated left by three
    q = np.zeros((E, tiles * 16, blocks * 128), np.int64)
    lane = np.arange(64)
    for s in range(4):
        for i in range(8):
            shift = 4 * (i // 2) + 16 * (i % 2)
            u = (words[..., s] >> shift) & 15  # [E, tiles, blocks, 64]
            for l in lane:
                q[:, l % 16::16, 32 * s + 8 * (l // 16) + i::128] = u[..., l].astype(np.int64) - 8
    g = 128 // group
    sc = (scales.view(np.uint16).astype(np.uint32) << 16).view(np.float32).reshape(E, tiles, blocks, 16, g)
    full = np.zeros((E, tiles * 16, blocks * 128), np.float32)
    for r in range(16):
        per = sc[:, :, :, r, :].reshape(E, tiles, blocks * g)
        full[:, r::16, :] = np.repeat(per, group, axis=2)
    return q, full


def bf16_round(v: np.ndarray) -> np.ndarray:
    return torch.from_numpy(np.ascontiguousarray(v, np.float32)).bfloat16().float().numpy()


def quantise(w: np.ndarray, group: int) -> np.ndarray:
    """The values that w [..., K] (fp32) stands for in 4 bits, in 64 bits."""
    w = np.asarray(w, np.float32)
    K = w.shape[-1]
    out = np.zeros(w.shape, np.float64)
    for a in range(0, K, group):
        p = w[..., a:a + group]
        bad = ~np.isfinite(p).all(-1, keepdims=True)
        m = np.abs(np.where(np.isfinite(p), p, 0)).max(-1, keepdims=True)
        s = bf16_round(m * np.float32(1 / 7))
        live = (s > 0) & ~bad
        with np.errstate(all="ignore"):
            q = np.clip(np.rint((p / np.where(live, s, np.float32(1))).astype(np.float32)), -7, 7)
        v = np.where(live, np.where(live, q, 0).astype(np.float64) * s.astype(np.float64), 0.0)
        out[..., a:a + group] = np.where(bad, np.nan, v)
    return out


def route(x64, r64, bias, k, renorm):
    """ids [T, k] and weights [T, k] of the router, in 64 bits."""
    logits = x64 @ r64.T
    if bias is not None:
        logits = logits + bias.astype(np.float64)
    ids = np.zeros((len(logits), k), np.int64)
    w = np.zeros((len(logits), k))
    for t, l in enumerate(logits):
        key = np.where(np.isnan(l), np.inf, l)
        # a NaN before +inf, then by value, then by index
        order = np.lexsort((np.arange(len(l)), -key, ~np.isnan(l)))
        ids[t] = order[:k]
        m = l[order[0]]
        if m == -np.inf:
            continue
        with np.errstate(all="ignore"):
            p = np.exp(l - m)
            w[t] = (p / p.sum())[ids[t]]
            if renorm:
                w[t] /= w[t].sum()
    return ids, w


def moe(x64, ids, w, gate, up, down, act):
    """y of the layer; gate, up [E, f, d] and down [E, d, f] in 64 bits."""
    y = np.zeros((len(x64), down.shape[1]))
    with np.errstate(all="ignore"):
        for t in range(len(x64)):
            for i, e in enumerate(ids[t]):
                if w[t, i] == 0:
                    continue
                g, u = gate[e] @ x64[t], up[e] @ x64[t]
                a = np.where(g < 0, 0, g) if act == "relu" else g / (1 + np.exp(-g))
                y[t] += w[t, i] * (down[e] @ (a * u))
    return y
