"""The few-token operators of the gated feed-forward layer, as cases to time and compare.

Three operators: weights packed to 4 bits with group scales and read back ("pack"), a product with such
weights for a few tokens ("linear"), and a mixture-of-experts gated feed-forward layer for a few tokens
("moe", experts in bf16 or in 4 bits).  With ``own`` false ``run`` computes them with elementary torch
operations in 32 bits; with ``own`` true it calls the library.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # one token through the gate of the 0.5B-class layer (d_model 1024, d_ff 4096): latency is all
        dict(name="linear 1 token 0.5B gate", op="linear", T=1, N=4096, K=1024, group=128, dtype="bf16"),
        # one token through the up projection of the 2B-class layer, the finest groups
        dict(name="linear 1 token 2B up", op="linear", T=1, N=8192, K=2048, group=32, dtype="bf16"),
        # sixteen sequences decoding together through the widest layer of the benchmark (4096 -> 11008)
        dict(name="linear 16 tokens wide", op="linear", T=16, N=11008, K=4096, group=128, dtype="bf16"),
        # odd everything, fp32 activations: rows that are not aligned, a last group that is short
        dict(name="linear 7 tokens odd fp32", op="linear", T=7, N=5001, K=1999, group=64, dtype="fp32"),
        # a short prompt (or a large decoding batch) through the 2B-class down projection
        dict(name="linear 128 tokens 2B down", op="linear", T=128, N=2048, K=8192, group=128, dtype="bf16"),
        # one token, few large bf16 experts of the 0.5B-class layer
        dict(name="moe 1 token bf16", op="moe", T=1, E=8, k=2, d=1024, f=4096, bits=16, group=0, act="relu",
             renorm=True, dtype="bf16"),
        # one token, many small 4-bit experts at the 2B-class width
        dict(name="moe 1 token 4 bits", op="moe", T=1, E=64, k=8, d=2048, f=1024, bits=4, group=128, act="silu",
             renorm=True, dtype="bf16"),
        # sixteen sequences decoding together, bf16 experts
        dict(name="moe 16 tokens bf16", op="moe", T=16, E=32, k=4, d=2048, f=1024, bits=16, group=0, act="relu",
             renorm=False, dtype="bf16"),
        # a decoding batch that reaches every 4-bit expert: the largest call
        dict(name="moe 64 tokens 4 bits", op="moe", T=64, E=64, k=8, d=2048, f=1024, bits=4, group=64, act="silu",
             renorm=True, dtype="bf16"),
        # odd widths and fp32 activations
        dict(name="moe 5 tokens odd fp32", op="moe", T=5, E=7, k=3, d=1001, f=707, bits=4, group=32, act="silu",
             renorm=True, dtype="fp32"),
        # packing one trained matrix of the 2B-class layer for serving, and reading it back
        dict(name="pack 2B gate", op="pack", E=1, N=8192, K=2048, group=128, transposed=False, wtype="bf16"),
        # packing the down projections of a set of experts, which training keeps one row per neuron, in fp32
        dict(name="pack expert downs fp32", op="pack", E=6, N=1001, K=1407, group=32, transposed=True, wtype="fp32"),
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
    return max(w["bytes"], w["flops"] / 50)


def draw(rng):
    most = max(_cost(c) for c in listed() if c["op"] == "moe")
    while True:
        op = rng.choice(["linear", "linear", "moe", "moe", "pack"])
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        group = rng.choice([32, 64, 128])
        if op == "linear":
            c = dict(op=op, T=_count(rng, 1, 128), N=_spread(rng, 512, 11008), K=_spread(rng, 512, 8192), group=group,
                     dtype=dtype)
        elif op == "moe":
            E = _count(rng, 4, 64)
            bits = rng.choice([4, 16])
            c = dict(op=op, T=_count(rng, 1, 64), E=E, k=rng.randint(1, min(8, E)), d=_spread(rng, 512, 2048),
                     f=_spread(rng, 256, 4096), bits=bits, group=group if bits == 4 else 0,
                     act=rng.choice(["relu", "silu"]), renorm=rng.random() < 0.5, dtype=dtype)
            if c["E"] * c["d"] * c["f"] > 64 * 2048 * 1024:
                continue
        else:
            c = dict(op=op, E=rng.choice([1, 1, 4]), N=_spread(rng, 512, 8192), K=_spread(rng, 512, 4096), group=group,
                     transposed=rng.random() < 0.5, wtype=rng.choice(["bf16", "fp32"]))
            if c["E"] * c["N"] * c["K"] > 8192 * 2048:
                continue
        if _cost(c) <= most:
            return c


def _plane_bytes(n, k, bits, group):
    """Bytes of one packed n x k matrix: the codes, and a two-byte scale for each group of a row."""
    return n * k * bits / 8 + (2 * n * math.ceil(k / group) if group else 0)


def work(case):
    c = case
    if c["op"] == "linear":
        T, N, K, e = c["T"], c["N"], c["K"], SIZE[c["dtype"]]
        return {"bytes": _plane_bytes(N, K, 4, c["group"]) + T * (N + K) * e, "flops": 2.0 * T * N * K}
    if c["op"] == "moe":
        T, E, k, d, f, e = c["T"], c["E"], c["k"], c["d"], c["f"], SIZE[c["dtype"]]
        # the experts that T tokens reach when each picks k of E at random
        reached = E * (1 - (1 - k / E) ** T)
        one = 2 * _plane_bytes(f, d, c["bits"], c["group"]) + _plane_bytes(d, f, c["bits"], c["group"])
        return {"bytes": reached * one + E * d * e + 2 * T * d * e + 8 * T * k,
                "flops": 2.0 * T * E * d + 6.0 * T * k * d * f}
    n = c["E"] * c["N"] * c["K"]
    packed = c["E"] * _plane_bytes(c["N"], c["K"], 4, c["group"])
    return {"bytes": n * SIZE[c["wtype"]] + 2 * packed + 4 * n, "flops": 0}


# ----------------------------------------------------------------------------- inputs
def _normal(g, *shape, scale=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * scale


def _inputs(case, seed):
    """The float tensors of a case, drawn on the GPU from the seed."""
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    if c["op"] == "linear":
        dt = DTYPES[c["dtype"]]
        return dict(x=_normal(g, c["T"], c["K"]).to(dt),
                    w=_normal(g, 1, c["N"], c["K"], scale=c["K"] ** -0.5).bfloat16())
    if c["op"] == "moe":
        dt = DTYPES[c["dtype"]]
        T, E, d, f = c["T"], c["E"], c["d"], c["f"]
        return dict(x=_normal(g, T, d).to(dt), router=_normal(g, E, d, scale=2 * d ** -0.5).to(dt),
                    gate=_normal(g, E, f, d, scale=d ** -0.5).bfloat16(),
                    up=_normal(g, E, f, d, scale=d ** -0.5).bfloat16(),
                    down=_normal(g, E, f, d, scale=f ** -0.5).bfloat16())  # one row per neuron
    shape = (c["E"], c["K"], c["N"]) if c["transposed"] else (c["E"], c["N"], c["K"])
    return dict(w=_normal(g, *shape, scale=c["K"] ** -0.5).to(DTYPES[c["wtype"]]))


def _quantise(w, group):
    """Codes (int8, -7..7) and scales (bf16, one for each group of inputs) of w [E, N, K]."""
    E, N, K = w.shape
    groups = -(-K // group)
    p = torch.nn.functional.pad(w.float(), (0, groups * group - K)).view(E, N, groups, group)
    s = (p.abs().amax(-1, keepdim=True) / 7).bfloat16()
    sf = s.float()
    q = torch.where(sf > 0, (p / torch.where(sf > 0, sf, 1.0)).round().clamp(-7, 7), 0.0)
    return q.view(E, N, groups * group)[..., :K].to(torch.int8).contiguous(), s.view(E, N, groups).contiguous()


def _dequantise(q, s, group):
    return q.float() * s.float().repeat_interleave(group, -1)[..., : q.shape[-1]]


def prepare(case, seed):
    c, t = dict(case), _inputs(case, seed)
    if own:
        import activation_sparse_feedforward_amd as A

        if c["op"] == "linear":
            wd = A.WDesc(1, c["N"], c["K"], 4, c["group"])
            planes = A.alloc_weights(wd)
            A.twell_weights_pack(wd, t["w"], planes)
            return dict(c=c, x=t["x"], wd=wd, w=planes,
                        y=torch.empty(c["T"], c["N"], dtype=t["x"].dtype, device="cuda"))
        if c["op"] == "moe":
            md = A.MoeDesc(c["T"], c["d"], c["f"], c["E"], c["k"], c["dtype"], c["bits"], c["group"], c["act"],
                           c["renorm"])
            w = A.alloc_moe_weights(md)
            A.twell_weights_pack(md.in_desc, t["gate"], w.gate)
            A.twell_weights_pack(md.in_desc, t["up"], w.up)
            A.twell_weights_pack(md.out_desc, t["down"], w.down, transposed=True)
            return dict(c=c, x=t["x"], md=md, router=t["router"], w=w, out=A.alloc_moe_out(md), ws=A.alloc_moe_ws(md))
        wd = A.WDesc(c["E"], c["N"], c["K"], 4, c["group"])
        return dict(c=c, w=t["w"], wd=wd, planes=A.alloc_weights(wd),
                    back=torch.empty(c["E"], c["N"], c["K"], dtype=torch.float32, device="cuda"))
    if c["op"] == "linear":
        q, s = _quantise(t["w"], c["group"])
        return dict(c=c, x=t["x"], w=(q[0], s[0]))
    if c["op"] == "moe" and c["bits"] == 4:
        down = t["down"].transpose(1, 2).contiguous()
        return dict(c=c, x=t["x"], router=t["router"], gate=_quantise(t["gate"], c["group"]),
                    up=_quantise(t["up"], c["group"]), down=_quantise(down, c["group"]))
    if c["op"] == "moe":
        return dict(c=c, x=t["x"], router=t["router"], gate=(t["gate"],), up=(t["up"],),
                    down=(t["down"].transpose(1, 2).contiguous(),))
    return dict(c=c, w=t["w"])


# ----------------------------------------------------------------------------- one pass
def _moe_plain(c, x, router, gate, up, down):
    xf, dtype = x.float(), x.dtype
    logits = xf @ router.float().T
    # a stable sort keeps the lowest index first among equals
    ids = torch.sort(logits, dim=-1, descending=True, stable=True).indices[:, : c["k"]]
    p = torch.exp(logits - logits.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    w = p.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    T, k = ids.shape

    def values(parts, at=None):
        parts = parts if at is None else tuple(v[at] for v in parts)
        return _dequantise(*parts, c["group"]) if c["bits"] == 4 else parts[0].float()

    def act(v):
        return v.clamp(min=0) if c["act"] == "relu" else v / (1 + torch.exp(-v))

    if T * k < c["E"]:  # the chosen experts' weights alone
        at = ids.reshape(-1)
        xs = xf.repeat_interleave(k, 0).unsqueeze(-1)
        h = act(torch.matmul(values(gate, at), xs)) * torch.matmul(values(up, at), xs)
        y = (torch.matmul(values(down, at), h).view(T, k, -1) * w.unsqueeze(-1)).sum(1)
    else:  # every token through every expert, weighted by zero where it was not chosen
        h = act(torch.matmul(xf, values(gate).transpose(1, 2))) * torch.matmul(xf, values(up).transpose(1, 2))
        all_w = torch.zeros_like(logits).scatter(1, ids, w)
        y = torch.matmul(h * all_w.T.unsqueeze(-1), values(down).transpose(1, 2)).sum(0)
    return dict(y=y.to(dtype), ids=ids.to(torch.int32), weights=w)


def run(state):
    c = state["c"]
    if own:
        import activation_sparse_feedforward_amd as A

        if c["op"] == "linear":
            A.twell_linear_fwd(state["wd"], state["w"], state["x"], state["y"])
            return dict(y=state["y"])
        if c["op"] == "moe":
            o = state["out"]
            A.twell_moe_fwd(state["md"], state["x"], state["router"], state["w"], o, state["ws"])
            return dict(y=o.y, ids=o.ids, weights=o.weights)
        A.twell_weights_pack(state["wd"], state["w"], state["planes"], transposed=c["transposed"])
        A.twell_weights_unpack(state["wd"], state["planes"], state["back"])
        return dict(values=state["back"])
    if c["op"] == "linear":
        return dict(y=(state["x"].float() @ _dequantise(*state["w"], c["group"]).T).to(state["x"].dtype))
    if c["op"] == "moe":
        return _moe_plain(c, state["x"], state["router"], state["gate"], state["up"], state["down"])
    w = state["w"].transpose(1, 2) if c["transposed"] else state["w"]
    return dict(values=_dequantise(*_quantise(w, c["group"]), c["group"]))


# ----------------------------------------------------------------------------- 64 bits
def _rounded_weights(w, group):
    """What w [N, K] stands for once held in 4 bits, in 64 bits, group by group of columns."""
    w = w.double()
    out = torch.empty_like(w)
    for a in range(0, w.shape[1], group):
        part = w[:, a : a + group]
        s = (part.abs().max(1, keepdim=True).values.float() / 7).bfloat16().double()
        q = torch.round(part / s.where(s > 0, torch.ones_like(s))).clamp(-7, 7)
        out[:, a : a + group] = q * s
    return out


def exact(case, seed):
    c, t = case, _inputs(case, seed)
    if c["op"] == "linear":
        return dict(y=t["x"].double() @ _rounded_weights(t["w"][0], c["group"]).T)
    if c["op"] == "pack":
        w = t["w"].transpose(1, 2) if c["transposed"] else t["w"]
        return dict(values=torch.stack([_rounded_weights(m, c["group"]) for m in w]))
    x, E, k = t["x"].double(), c["E"], c["k"]
    logits = x @ t["router"].double().T
    p = torch.softmax(logits, -1)
    order = torch.argsort(logits, dim=-1, descending=True, stable=True)[:, :k]
    w = torch.gather(p, 1, order)
    w = w / w.sum(1, keepdim=True) if c["renorm"] else w
    y = torch.zeros_like(x)
    for e in range(E):
        row, slot = (order == e).nonzero(as_tuple=True)
        if not len(row):
            continue
        mats = [t["gate"][e], t["up"][e], t["down"][e].T]
        mats = [_rounded_weights(m, c["group"]) if c["bits"] == 4 else m.double() for m in mats]
        g, u = x[row] @ mats[0].T, x[row] @ mats[1].T
        h = (torch.relu(g) if c["act"] == "relu" else g * torch.sigmoid(g)) * u
        y[row] += w[row, slot].unsqueeze(1) * (h @ mats[2].T)
    return dict(y=y, ids=None, weights=w)
