"""GPU parity of the few-token operators at serving sizes, where a wave takes several blocks of inputs, a workgroup
its most tokens, tiles and waves, and a launch more than 64 KB of LDS, against 64 bits on the GPU.

Tolerances.  The matrix instruction cuts a sum off at 24 bits, so a chain of n of them is off by n 2^-23 of what it
holds at the most; a wave that takes all of K inputs chains 4 ceil(K / 128) instructions, times three for fp32 data.
A bf16 output adds its one rounding, 2^-8, and the hidden values of the expert layer 2^-17 (bf16 data).  Element by
element, 40 times that of the output's rms is allowed, plus the rounding.
"""
import numpy as np
import pytest
import torch

import _few_token as R
from activation_sparse_feedforward_amd import twell as T
from _helpers import check_guards, guarded, host64, say

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _chain(K, dtype):
    return 4 * -(-K // 128) * (3 if dtype == "fp32" else 1) * 2.0 ** -23


def _close(got, ref, dtype, tol):
    got, rnd = got.double(), 2.0 ** -8 if dtype == "bf16" else 0.0
    assert torch.isfinite(got).all()
    norm = ref.norm().item()
    assert (got - ref).norm().item() <= (rnd + tol) * norm, (got - ref).norm().item() / norm
    assert ((got - ref).abs() <= rnd * ref.abs() + 40 * tol * norm / ref.numel() ** 0.5).all()


def _randn(g, *shape, scale=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * scale


def _packed(w, wd, transposed=False):
    """Planes of w, and the values they stand for in 64 bits (reading back is exact, as tested elsewhere)."""
    pl = T.Weights(*(guarded(t.shape, t.dtype) for t in T.alloc_weights(wd)))
    T.twell_weights_pack(wd, w, pl, transposed=transposed)
    back = torch.empty(wd.experts, wd.rows, wd.cols, dtype=torch.float32 if wd.bits == 4 else torch.bfloat16,
                       device="cuda")
    T.twell_weights_unpack(wd, pl, back)
    return pl, back


# Rows for every CU and more, so that 4 to 64 tokens and one to four tiles share a workgroup.
@pytest.mark.parametrize("T_", [1, 7, 16, 29, 128])
@pytest.mark.parametrize("N,K,group", [(2048, 8192, 128), (5001, 1999, 64), (11008, 4100, 32), (12300, 1999, 128),
                                       (16384, 2048, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_linear_deep(T_, N, K, group, dtype):
    say(f"[gpu case] linear deep T={T_} N={N} K={K} group={group} {dtype}")
    g = torch.Generator(device="cuda").manual_seed(T_ + N + K)
    wd = T.WDesc(1, N, K, 4, group)
    pl, w = _packed(_randn(g, 1, N, K, scale=K ** -0.5).bfloat16(), wd)
    x, y = _randn(g, T_, K).to(DT[dtype]), guarded((T_, N), DT[dtype])
    T.twell_linear_fwd(wd, pl, x, y)
    torch.cuda.synchronize()
    check_guards(*pl, y)
    _close(y, x.double() @ w[0].double().T, dtype, 2e-6 + _chain(K, dtype))


def _moe(T_, E, k, d, f, bits, group, dtype, act="silu"):
    say(f"[gpu case] moe deep T={T_} E={E} k={k} d={d} f={f} bits={bits} group={group} {dtype}")
    md = T.MoeDesc(T_, d, f, E, k, dtype, bits, group, act, True)
    g = torch.Generator(device="cuda").manual_seed(T_ + E + d + f)
    x, router = _randn(g, T_, d).to(DT[dtype]), _randn(g, E, d, scale=2 * d ** -0.5).to(DT[dtype])
    gate, gv = _packed(_randn(g, E, f, d, scale=d ** -0.5).bfloat16(), md.in_desc)
    up, uv = _packed(_randn(g, E, f, d, scale=d ** -0.5).bfloat16(), md.in_desc)
    down, dv = _packed(_randn(g, E, f, d, scale=f ** -0.5).bfloat16(), md.out_desc, True)
    out = T.MoeOut(*(guarded(t.shape, t.dtype) for t in T.alloc_moe_out(md)))
    ws = guarded((T.moe_ws_bytes(md),), torch.uint8)
    T.twell_moe_fwd(md, x, router, T.MoeWeights(gate, up, down), out, ws)
    torch.cuda.synchronize()
    check_guards(*out, ws, *gate, *up, *down)
    ids, wts = R.route(host64(x), host64(router), None, k, True)
    assert np.array_equal(out.ids.cpu().numpy(), ids)
    # a logit of up to some 8, summed in fp32 by lanes of d / 64 products each, through exp and the division
    assert np.all(np.abs(host64(out.weights) - wts) <= 1e-5 * wts)
    ids, wts = torch.from_numpy(ids).cuda(), torch.from_numpy(wts).cuda()
    ref = torch.zeros(T_, d, dtype=torch.float64, device="cuda")
    for e in range(E):
        row, slot = (ids == e).nonzero(as_tuple=True)
        if len(row):
            xs = x[row].double()
            a, u = xs @ gv[e].double().T, xs @ uv[e].double().T
            h = (a.clamp(min=0) if act == "relu" else a / (1 + torch.exp(-a))) * u
            ref[row] += wts[row, slot].unsqueeze(1) * (h @ dv[e].double().T)
    hidden = 2.0 ** -17 if dtype == "bf16" else 0.0
    _close(out.y, ref, dtype, 1.2e-5 + hidden + 2 * _chain(d, dtype) + _chain(f, dtype))


@pytest.mark.parametrize("T_,E,k,d,f,bits,group,dtype", [
    (1, 8, 2, 1024, 4096, 16, 0, "bf16"),
    (3, 8, 2, 1024, 4096, 16, 0, "fp32"),
    (1, 64, 8, 2048, 1024, 4, 32, "bf16"),
    (1, 64, 8, 2048, 1024, 4, 64, "bf16"),
    (1, 64, 8, 2048, 1024, 4, 128, "bf16"),
    (64, 64, 8, 2048, 1024, 4, 32, "bf16"),
    (64, 64, 8, 2048, 1024, 4, 64, "bf16"),
    (64, 64, 8, 2048, 1024, 4, 128, "bf16"),
    (16, 32, 4, 2048, 1024, 16, 0, "bf16"),
    (5, 7, 3, 1001, 707, 4, 32, "fp32"),
    (5, 7, 3, 1001, 707, 4, 64, "fp32"),
    (5, 7, 3, 1001, 707, 4, 128, "fp32"),
    (5, 7, 3, 1001, 707, 16, 0, "fp32"),
    (6, 4, 2, 2100, 2050, 4, 64, "fp32"),
    (6, 4, 2, 2100, 2050, 16, 0, "fp32"),
    (40, 3, 2, 2100, 2050, 4, 32, "fp32"),
    (40, 3, 2, 2100, 2050, 16, 0, "fp32"),
    (40, 3, 2, 2100, 2050, 4, 128, "bf16"),
])
def test_moe_deep(T_, E, k, d, f, bits, group, dtype):
    _moe(T_, E, k, d, f, bits, group, dtype)


@pytest.mark.parametrize("T_", [5, 9, 16])
@pytest.mark.parametrize("bits,group", [(16, 0), (4, 32), (4, 64), (4, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_moe_one_kernel_for_down_and_sum(T_, bits, group, dtype):
    """At most 32 (pair, block)s: the kernel that takes all pairs of 16 outputs, with five to sixteen tokens."""
    _moe(T_, 8, 2, 72, 40, bits, group, dtype, "relu")
