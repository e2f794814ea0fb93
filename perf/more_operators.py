"""The operators of a mixture-of-experts layer over many tokens, as cases to time and compare.

Three sets: tokens sorted by expert and back with their weights ("tokens"), products with weights in 8-bit floating
point, one matrix or one per expert ("fp8"), and layer norm ("norm"); each forward, or with its gradients ("train").
With ``own`` false ``run`` computes them with elementary torch operations in 32 bits; with ``own`` true it calls the
library.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}
BLOCK = 128


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # one token of a decoding step on its way to 8 of 64 experts and back: latency is all
        dict(name="tokens 1", op="tokens", train=False, T=1, E=64, k=8, d=2048, dropped=0.0, dtype="bf16"),
        # a training batch at the 2B-class width, every pair kept: the largest call
        dict(name="tokens 16384 train", op="tokens", train=True, T=16384, E=64, k=8, d=2048, dropped=0.0, dtype="bf16"),
        # odd everything, fp32 rows that are not aligned, a tenth of the pairs masked out
        dict(name="tokens 3001 odd train", op="tokens", train=True, T=3001, E=7, k=3, d=1001, dropped=0.1,
             dtype="fp32"),
        # one token through the gate of the 0.5B-class layer
        dict(name="fp8 1 token", op="fp8", train=False, T=1, E=1, N=4096, K=1024, dtype="bf16"),
        # sixteen sequences decoding together through the widest layer of the benchmark
        dict(name="fp8 16 tokens wide", op="fp8", train=False, T=16, E=1, N=11008, K=4096, dtype="bf16"),
        # a long prompt through the up projection of the 2B-class layer
        dict(name="fp8 16384 tokens", op="fp8", train=False, T=16384, E=1, N=8192, K=2048, dtype="bf16"),
        # a decoding batch of 64 tokens, each at 8 of 64 experts: a few rows for every expert
        dict(name="fp8 64 experts 512 rows", op="fp8", train=False, T=512, E=64, N=1024, K=2048, dtype="bf16"),
        # a training step of odd experts in fp32
        dict(name="fp8 5 experts odd train", op="fp8", train=True, T=777, E=5, N=1001, K=707, dtype="fp32"),
        # a training step of the experts' up projections: packing, forward, both gradients
        dict(name="fp8 16 experts train", op="fp8", train=True, T=16384, E=16, N=1024, K=2048, dtype="bf16"),
        # the norm in front of one decoded token's layer
        dict(name="norm 1 token", op="norm", train=False, T=1, d=2048, dtype="bf16"),
        # a training batch at the 2B-class width
        dict(name="norm 16384 train", op="norm", train=True, T=16384, d=2048, dtype="bf16"),
        # rows that are not aligned, fp32
        dict(name="norm 1999 odd train", op="norm", train=True, T=1999, d=4099, dtype="fp32"),
    ]


def _spread(rng, lo, hi):
    """A size between lo and hi, spread over its logarithm; half of them multiples of 64, the others as they fall."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5:
        v = (v + 32) // 64 * 64
    return max(lo, min(hi, v))


def _count(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 250)


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        op, train, dtype = rng.choice(["tokens", "fp8", "fp8", "norm"]), rng.random() < 0.5, rng.choice(
            ["bf16", "bf16", "fp32"])
        T = _count(rng, 1, 16384)
        if op == "tokens":
            E = _count(rng, 2, 256)
            c = dict(op=op, train=train, T=T, E=E, k=rng.randint(1, min(8, E)), d=_spread(rng, 256, 4096),
                     dropped=rng.choice([0.0, 0.0, 0.05, 0.3]), dtype=dtype)
        elif op == "fp8":
            c = dict(op=op, train=train, T=T, E=rng.choice([1, _count(rng, 2, 64)]), N=_spread(rng, 256, 11008),
                     K=_spread(rng, 256, 8192), dtype=dtype)
            if c["E"] * c["N"] * c["K"] > 16 * 8192 * 2048 or (dtype == "fp32" and T * c["N"] * c["K"] > 1 << 35):
                continue
        else:
            c = dict(op=op, train=train, T=T, d=_spread(rng, 128, 11008), dtype=dtype)
        if _cost(c) <= most:
            return c


def work(case):
    c = case
    e = SIZE[c["dtype"]]
    if c["op"] == "tokens":
        T, P, d = c["T"], c["T"] * c["k"], c["d"]
        # ids read; offsets and places written; gather (T + P rows) and combine (P + T rows), weights read
        n = 4 * P + 4 * (c["E"] + 1) + 4 * P + 2 * (T + P) * d * e + 4 * P
        f = 2.0 * P * d
        if c["train"]:  # combine's gradient (2 P + T rows, weights read, their gradient written), gather's (P + T)
            n += (3 * P + 2 * T) * d * e + 8 * P
            f += 4.0 * P * d
        return {"bytes": n, "flops": f}
    if c["op"] == "norm":
        T, d = c["T"], c["d"]
        if c["train"]:  # x read, y written; x and dy read, dx written; statistics, weights and their gradients
            return {"bytes": 5 * T * d * e + 16 * T + 16 * d, "flops": 20.0 * T * d}
        return {"bytes": 2 * T * d * e + 8 * d, "flops": 8.0 * T * d}
    T, E, N, K = c["T"], c["E"], c["N"], c["K"]
    planes = E * (N * K + N * K / (BLOCK * BLOCK))
    if c["train"]:  # fp32 weights in, their gradient out; x, y, dy, dx
        return {"bytes": 8 * E * N * K + 2 * T * (N + K) * e, "flops": 6.0 * T * N * K}
    reached = planes * (1 - (1 - 1 / E) ** T)  # what T rows reach of the experts
    return {"bytes": reached + T * (N + K) * e, "flops": 2.0 * T * N * K}


# ----------------------------------------------------------------------------- inputs
def _normal(g, *shape, scale=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * scale


def _loads(T, E, seed):
    """Rows of each expert as a router leaves them: uneven, one expert without any, a few rows behind the last."""
    g = torch.Generator().manual_seed(int(seed))
    if E == 1:
        return torch.tensor([T])
    p = torch.exp(0.5 * torch.randn(E, generator=g))
    if E >= 4:
        p[E // 2] = 0
    return torch.bincount(torch.multinomial(p, max(T - T // 16, 1), replacement=True, generator=g), minlength=E)


def _inputs(case, seed):
    """The tensors of a case, drawn on the GPU from the seed."""
    c, dt = case, DTYPES[case["dtype"]]
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    if c["op"] == "tokens":
        T, E, k, d = c["T"], c["E"], c["k"], c["d"]
        # different experts for a token, some of them much liked
        ids = (_normal(g, T, E) + _normal(g, 1, E)).argsort(-1)[:, :k].to(torch.int32).contiguous()
        ids = ids.masked_fill(torch.rand(T, k, generator=g, device="cuda") < c["dropped"], -1)
        w = torch.rand(T, k, generator=g, device="cuda") + 0.05
        t = dict(ids=ids, weights=w / w.sum(-1, keepdim=True), x=_normal(g, T, d).to(dt),
                 z=_normal(g, T * k, d).to(dt))
        if c["train"]:
            t.update(dy=_normal(g, T, d, scale=0.1).to(dt), dxs=_normal(g, T * k, d, scale=0.1).to(dt))
        return t
    if c["op"] == "norm":
        T, d = c["T"], c["d"]
        t = dict(x=(_normal(g, T, d) * torch.exp(0.5 * _normal(g, T, 1)) + 0.3 * _normal(g, T, 1)).to(dt),
                 w=1 + 0.1 * _normal(g, d), b=0.1 * _normal(g, d))
        if c["train"]:
            t.update(dy=_normal(g, T, d, scale=0.1).to(dt))
        return t
    T, E, N, K = c["T"], c["E"], c["N"], c["K"]
    n = _loads(T, E, seed)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)]).to(torch.int32).cuda()
    t = dict(offsets=offsets, most=int(n.max()), x=_normal(g, T, K).to(dt), w=_normal(g, E, N, K, scale=K ** -0.5))
    if c["train"]:
        t.update(dy=_normal(g, T, N, scale=0.1).to(dt))
    else:
        t.update(w=t["w"].bfloat16())
    return t


def prepare(case, seed):
    c, t = dict(case), _inputs(case, seed)
    t["c"], dt = c, DTYPES[c["dtype"]]

    def empty(*shape, dtype=dt):
        return torch.zeros(*shape, dtype=dtype, device="cuda")

    if c["op"] == "tokens":
        # the rows behind the last one are left as they are
        T, P, d = c["T"], c["T"] * c["k"], c["d"]
        t.update(rows=empty(P, d), y=empty(T, d))
        if c["train"]:
            t.update(drows=empty(P, d), dweights=empty(T, c["k"], dtype=torch.float32), dx=empty(T, d))
        if own:
            import activation_sparse_feedforward_amd as A

            desc = A.TokensDesc(T, d, c["E"], c["k"], c["dtype"])
            t.update(desc=desc, order=A.alloc_tokens_order(desc), ws=A.alloc_tokens_ws(desc))
        return t
    if c["op"] == "norm":
        T, d = c["T"], c["d"]
        if own:
            import activation_sparse_feedforward_amd as A

            desc = A.NormDesc(T, d, c["dtype"], 1e-5)
            t.update(desc=desc, y=empty(T, d))
            if c["train"]:
                t.update(stats=empty(T, 2, dtype=torch.float32), dx=empty(T, d), dw=empty(d, dtype=torch.float32),
                         db=empty(d, dtype=torch.float32), ws=A.alloc_norm_ws(desc))
        return t
    T, E, N, K = c["T"], c["E"], c["N"], c["K"]
    t.update(y=empty(T, N))
    if c["train"]:
        t.update(dx=empty(T, K))
    if own:
        import activation_sparse_feedforward_amd as A

        desc = A.Fp8Desc(E, N, K)
        t.update(desc=desc, planes=A.alloc_fp8_weights(desc), ws=A.alloc_fp8_ws(desc, T))
        if c["train"]:
            t.update(planes_t=A.alloc_fp8_weights(desc.transposed), dw=empty(E, N, K, dtype=torch.float32))
        else:
            A.twell_fp8_weights_pack(desc, t.pop("w"), t["planes"])
    elif not c["train"]:
        t.update(planes=_codes_of_weights(t.pop("w").float()))
    return t


# ----------------------------------------------------------------------------- one pass
def _scale(most):
    """The smallest power of two, from 2^-126 on, that takes values up to ``most`` into e4m3's range, as an exponent."""
    m, x = torch.frexp(most)  # most = m 2^x, 0.5 <= m < 1; e4m3's largest value, 448, is 0.875 2^9
    return torch.clamp(torch.where(m <= 0.875, x - 9, x - 8), min=-126)


def _power(e):
    return ((e + 127) << 23).view(torch.float32)


def _padded(v, rows=False):
    """v with its last axis, or its last two, filled up to whole blocks."""
    return torch.nn.functional.pad(v, (0, -v.shape[-1] % BLOCK, 0, -v.shape[-2] % BLOCK if rows else 0))


def _codes_of_weights(w):
    """e4m3 codes of w [E, N, K] and the exponent of each block of 128 x 128."""
    E, N, K = w.shape
    p = _padded(w, rows=True)
    b = p.view(E, p.shape[1] // BLOCK, BLOCK, p.shape[2] // BLOCK, BLOCK)
    e = _scale(b.abs().amax((2, 4), keepdim=True))
    q = (b * _power(-e)).to(torch.float8_e4m3fn)
    return q.view(p.shape)[:, :N, :K].contiguous(), e


def _values_of_weights(q, e):
    E, N, K = q.shape
    s = _power(e).expand(-1, -1, BLOCK, -1, BLOCK).reshape(E, e.shape[1] * BLOCK, e.shape[3] * BLOCK)
    return q.float() * s[:, :N, :K]


def _rounded_rows(x):
    """What rows [..., K] stand for in e4m3 with a scale for each 128 of a row."""
    v = _padded(x.float())
    b = v.view(*v.shape[:-1], -1, BLOCK)
    e = _scale(b.abs().amax(-1, keepdim=True))
    return ((b * _power(-e)).to(torch.float8_e4m3fn).float() * _power(e)).view(v.shape)[..., : x.shape[-1]]


def _places(offsets, most, T):
    """Rows of each expert [E, most] and which of them are its own; expert and place of each row, and which have one."""
    at = offsets[:-1, None].long() + torch.arange(most, device=offsets.device)
    live = at < offsets[1:, None]
    row = torch.arange(T, device=offsets.device)
    expert = (row[:, None] >= offsets[None, 1:]).sum(1)
    there = expert < len(offsets) - 1
    expert = torch.where(there, expert, 0)
    slot = torch.where(there, row - offsets[expert], 0)
    return torch.where(live, at, 0), live, expert, slot, there


def _fp8_plain(t):
    c = t["c"]
    x, T = t["x"], c["T"]
    w = _values_of_weights(*(_codes_of_weights(t["w"]) if c["train"] else t["planes"]))
    if c["E"] == 1:
        out = dict(y=(_rounded_rows(x) @ w[0].T).to(x.dtype))
        if c["train"]:
            out.update(dx=(_rounded_rows(t["dy"]) @ w[0]).to(x.dtype), dw=(t["dy"].float().T @ x.float()).unsqueeze(0))
        return out
    at, live, expert, slot, there = _places(t["offsets"], t["most"], T)

    def through(v, m, old):
        r = torch.matmul(_rounded_rows(v)[at], m)
        return torch.where(there[:, None], r[expert, slot].to(v.dtype), old)

    out = dict(y=through(x, w.transpose(1, 2), t["y"]))
    if c["train"]:
        g = t["dy"].float()[at] * live[..., None]
        out.update(dx=through(t["dy"], w, t["dx"]), dw=torch.matmul(g.transpose(1, 2), x.float()[at]))
    return out


def _tokens_plain(t):
    c = t["c"]
    T, E, k, d, dt = c["T"], c["E"], c["k"], c["d"], t["x"].dtype
    ids = t["ids"].view(-1)
    key, order = torch.sort(torch.where((ids >= 0) & (ids < E), ids, E), stable=True)
    offsets = torch.searchsorted(key, torch.arange(E + 1, device=key.device, dtype=key.dtype)).to(torch.int32)
    place = torch.arange(T * k, device=key.device)
    pair_row = torch.zeros(T * k, dtype=torch.int32, device=key.device)
    pair_row[order] = torch.where(key < E, place, -1).to(torch.int32)
    there = place < offsets[-1]
    rows = torch.where(there[:, None], t["x"][order // k], t["rows"])
    w = t["weights"].view(-1) * (pair_row >= 0)
    at = pair_row.clamp(min=0).long()

    def back(v, w):
        return (v[at].float() * w[:, None]).view(T, k, d).sum(1).to(dt)

    out = dict(offsets=offsets, pair_row=pair_row.view(T, k), rows=rows, y=back(t["z"], w))
    if c["train"]:
        dy = t["dy"].float()
        dr = (dy[order // k] * t["weights"].view(-1)[order][:, None]).to(dt)
        dweights = (t["z"][at].float().view(T, k, d) * dy[:, None]).sum(-1) * (pair_row >= 0).view(T, k)
        out.update(drows=torch.where(there[:, None], dr, t["drows"]), dweights=dweights,
                   dx=back(t["dxs"], (pair_row >= 0).float()))
    return out


def _norm_plain(t):
    x = t["x"].float()
    mean = x.mean(-1, keepdim=True)
    c = x - mean
    rstd = 1 / torch.sqrt((c * c).mean(-1, keepdim=True) + 1e-5)
    h = c * rstd
    out = dict(y=(h * t["w"] + t["b"]).to(t["x"].dtype))
    if t["c"]["train"]:
        dy = t["dy"].float()
        g = dy * t["w"]
        dx = rstd * (g - g.mean(-1, keepdim=True) - h * (g * h).mean(-1, keepdim=True))
        out.update(stats=torch.cat([mean, rstd], 1), dx=dx.to(t["x"].dtype), dw=(dy * h).sum(0), db=dy.sum(0))
    return out


def run(state):
    t, c = state, state["c"]
    if not own:
        return {"tokens": _tokens_plain, "fp8": _fp8_plain, "norm": _norm_plain}[c["op"]](t)
    import activation_sparse_feedforward_amd as A

    if c["op"] == "tokens":
        desc, order = t["desc"], t["order"]
        A.twell_tokens_sort(desc, t["ids"], order, t["ws"])
        A.twell_tokens_gather(desc, t["x"], order, t["rows"])
        A.twell_tokens_combine(desc, t["z"], order, t["weights"], t["y"])
        out = dict(offsets=order.offsets, pair_row=order.pair_row, rows=t["rows"], y=t["y"])
        if c["train"]:
            A.twell_tokens_combine_bwd(desc, t["z"], order, t["weights"], t["dy"], t["drows"], t["dweights"])
            A.twell_tokens_combine(desc, t["dxs"], order, None, t["dx"])
            out.update(drows=t["drows"], dweights=t["dweights"], dx=t["dx"])
        return out
    if c["op"] == "norm":
        A.twell_layernorm_fwd(t["desc"], t["x"], t["w"], t["b"], t["y"], t.get("stats"))
        if not c["train"]:
            return dict(y=t["y"])
        A.twell_layernorm_bwd(t["desc"], t["x"], t["w"], t["stats"], t["dy"], t["dx"], t["dw"], t["db"], t["ws"])
        return dict(y=t["y"], stats=t["stats"], dx=t["dx"], dw=t["dw"], db=t["db"])
    desc, offsets = t["desc"], t["offsets"] if c["E"] > 1 else None
    if c["train"]:
        A.twell_fp8_weights_pack(desc, t["w"], t["planes"], t["planes_t"])
    A.twell_fp8_linear_fwd(desc, t["planes"], t["x"], t["y"], t["ws"], offsets=offsets)
    if not c["train"]:
        return dict(y=t["y"])
    A.twell_fp8_linear_bwd(desc, t["planes_t"], t["x"], t["dy"], t["dx"], t["dw"], t["ws"], offsets=offsets)
    return dict(y=t["y"], dx=t["dx"], dw=t["dw"])


# ----------------------------------------------------------------------------- 64 bits
def _to_e4m3(v, most):
    """v in 64 bits, rounded to e4m3 with the scale of a block whose largest magnitude is ``most``."""
    e = torch.floor(torch.log2(most.clamp(min=2.0 ** -140) / 448)) - 1  # from below, whatever the logarithm's rounding
    for _ in range(3):
        e = torch.where(torch.exp2(e) * 448 < most, e + 1, e)
    s = torch.exp2(e.clamp(min=-126))
    u = v / s
    x = torch.frexp(u.abs()).exponent - 1  # 2^x <= |u| < 2^(x + 1): three bits of fraction, the last step from 2^-6 down
    step = torch.ldexp(torch.ones_like(u), x.clamp(min=-6) - 3)
    return torch.round(u / step) * step * s


def _exact_weights(w):
    w = w.double()
    out = torch.empty_like(w)
    for a in range(0, w.shape[0], BLOCK):
        for b in range(0, w.shape[1], BLOCK):
            part = w[a : a + BLOCK, b : b + BLOCK]
            out[a : a + BLOCK, b : b + BLOCK] = _to_e4m3(part, part.abs().max())
    return out


def _exact_rows(x):
    x = x.double()
    out = torch.empty_like(x)
    for b in range(0, x.shape[1], BLOCK):
        part = x[:, b : b + BLOCK]
        out[:, b : b + BLOCK] = _to_e4m3(part, part.abs().max(1, keepdim=True).values)
    return out


def exact(case, seed):
    c, t = case, _inputs(case, seed)
    if c["op"] == "norm":
        x = t["x"].double()
        var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
        r = (var + 1e-5).rsqrt()
        h, w = (x - mean) * r, t["w"].double()
        out = dict(y=torch.addcmul(t["b"].double(), h, w))
        if c["train"]:
            dy = t["dy"].double()
            d = c["d"]
            s1, s2 = dy @ w / d, ((dy * h) @ w) / d
            out.update(stats=torch.stack([mean[:, 0], r[:, 0]], 1), dx=r * (dy * w - s1[:, None] - h * s2[:, None]),
                       dw=torch.einsum("td,td->d", dy, h), db=dy.sum(0))
        return out
    if c["op"] == "tokens":
        T, E, k, d = c["T"], c["E"], c["k"], c["d"]
        if T * k * d > 1 << 29:
            return None
        ids = t["ids"].cpu().view(-1).tolist()
        order = sorted((e, p) for p, e in enumerate(ids) if 0 <= e < E)
        pair = torch.tensor([p for _, p in order], dtype=torch.int64, device="cuda")
        n, w = len(order), t["weights"].double().view(-1)
        z = t["z"].double()[:n]
        rows, y = torch.zeros(T * k, d, dtype=torch.float64, device="cuda"), torch.zeros(
            T, d, dtype=torch.float64, device="cuda")
        rows[:n] = t["x"].double()[pair // k]
        out = dict(offsets=None, pair_row=None, rows=rows, y=y.index_add(0, pair // k, z * w[pair, None]))
        if c["train"]:
            dy = t["dy"].double()[pair // k]
            drows = torch.zeros_like(rows)
            drows[:n] = dy * w[pair, None]
            dweights = torch.zeros(T * k, dtype=torch.float64, device="cuda")
            dweights[pair] = (z * dy).sum(1)
            out.update(drows=drows, dweights=dweights.view(T, k),
                       dx=y.index_add(0, pair // k, t["dxs"].double()[:n]))
        return out
    T, E, N, K = c["T"], c["E"], c["N"], c["K"]
    off = t["offsets"].tolist()
    y = torch.zeros(T, N, dtype=torch.float64, device="cuda")
    dx = torch.zeros(T, K, dtype=torch.float64, device="cuda")
    dw = torch.zeros(E, N, K, dtype=torch.float64, device="cuda") if c["train"] else None
    qx, qdy = _exact_rows(t["x"]), _exact_rows(t["dy"]) if c["train"] else None
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        m = _exact_weights(t["w"][e])
        y[a:b] = qx[a:b] @ m.T
        if c["train"]:
            dx[a:b] = qdy[a:b] @ m
            dw[e] = t["dy"][a:b].double().T @ t["x"][a:b].double()
    return dict(y=y, dx=dx, dw=dw) if c["train"] else dict(y=y)
