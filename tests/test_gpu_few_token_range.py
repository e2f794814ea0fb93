"""4-bit weights and inputs of very different sizes: a weight of 0 takes nothing from an input, however large, and a
finite sum of finite products is finite.

Tolerances.  Every output here is one product x q s, or 128 equal ones, which fp32 sums hold to 2^-16 at the worst
(128 roundings of 2^-23): the rounding to bf16 is 2^-8, the hidden values of the expert layer with bf16 data add 2^-17
each, the few fp32 roundings of a chain 2^-21 together.
"""
import numpy as np
import pytest
import torch

from activation_sparse_feedforward_amd import twell as T
from _helpers import host64, say

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
REL = {"bf16": 2.0 ** -8 + 2.0 ** -16, "fp32": 2.0 ** -20}


def _planes(w, wd):
    pl, back = T.alloc_weights(wd), torch.empty(wd.experts, wd.rows, wd.cols, device="cuda")
    T.twell_weights_pack(wd, w, pl)
    T.twell_weights_unpack(wd, pl, back)
    return pl, host64(back)


def _small_beside_large(T_, K, dtype):
    """x with a large value at input 5 and a small one, above 0, at input 0 of the same group."""
    x = torch.randn(T_, K, generator=torch.Generator(device="cuda").manual_seed(T_), device="cuda")
    x[:, 0] = x[:, 0].abs() * 0.01 + 0.001
    x[:, 5] = 1e4
    return x.to(DT[dtype])


@pytest.mark.parametrize("T_", [1, 6, 20, 100])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_linear_weights_of_zero_take_nothing_from_large_inputs(T_, group, dtype):
    say(f"[gpu case] linear outlier T={T_} group={group} {dtype}")
    N, K = 300, 520
    x = _small_beside_large(T_, K, dtype)
    w = torch.zeros(1, N, K, device="cuda")
    w[0, :, 0] = torch.linspace(0.5, 2, N, device="cuda")
    wd = T.WDesc(1, N, K, 4, group)
    pl, v = _planes(w, wd)
    y = torch.empty(T_, N, dtype=DT[dtype], device="cuda")
    T.twell_linear_fwd(wd, pl, x, y)
    ref = host64(x)[:, :1] * v[0, :, 0]
    assert np.all(np.abs(host64(y) - ref) <= REL[dtype] * np.abs(ref))


@pytest.mark.parametrize("T_", [1, 6, 20, 100])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_linear_large_inputs_with_a_finite_sum(T_, group, dtype):
    """128 inputs of 2e35 times codes of 7: 1.8e38, within fp32."""
    say(f"[gpu case] linear range T={T_} group={group} {dtype}")
    N, K = 40, 128
    wd = T.WDesc(1, N, K, 4, group)
    pl, v = _planes(torch.full((1, N, K), 1e-3, device="cuda"), wd)
    x = torch.full((T_, K), 2e35, device="cuda").to(DT[dtype])
    y = torch.empty(T_, N, dtype=DT[dtype], device="cuda")
    T.twell_linear_fwd(wd, pl, x, y)
    ref = host64(x) @ v[0].T
    assert np.all(np.abs(host64(y) - ref) <= (REL[dtype] + 2.0 ** -16) * np.abs(ref))


def _layer(T_, d, f, group, dtype, x, gate, up, down):
    """y of one expert that every token takes with weight 1."""
    md = T.MoeDesc(T_, d, f, 2, 1, dtype, 4, group, "relu", True)
    both = [torch.cat([torch.zeros_like(m), m]) for m in (gate, up, down)]
    planes, values = zip(*(_planes(m, wd) for m, wd in zip(both, (md.in_desc, md.in_desc, md.out_desc))))
    out = T.alloc_moe_out(md)
    bias = torch.tensor([float("-inf"), 0.0], device="cuda")
    T.twell_moe_fwd(md, x, torch.zeros(2, d, dtype=x.dtype, device="cuda"), T.MoeWeights(*planes), out,
                    T.alloc_moe_ws(md), router_bias=bias)
    assert (out.ids == 1).all() and (out.weights == 1).all()
    return host64(out.y), [v[1] for v in values]


@pytest.mark.parametrize("T_", [1, 6, 20, 64])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_moe_weights_of_zero_take_nothing_from_large_values(T_, group, dtype):
    """Neuron 0 is large and the outputs read neuron 1, which reads a small input beside a large one."""
    say(f"[gpu case] moe outlier T={T_} group={group} {dtype}")
    d, f = 260, 72
    x = _small_beside_large(T_, d, dtype)
    gate, down = torch.zeros(1, f, d, device="cuda"), torch.zeros(1, d, f, device="cuda")
    gate[0, 0, 5], gate[0, 1:, 0], down[0, :, 1] = 1.0, 1.0, torch.linspace(0.5, 2, d, device="cuda")
    y, (g, u, dn) = _layer(T_, d, f, group, dtype, x, gate, gate, down)
    x0 = host64(x)[:, :1]
    ref = (x0 * g[1, 0]) * (x0 * u[1, 0]) * dn[:, 1]
    assert np.all(np.abs(y - ref) <= (REL[dtype] + 2.0 ** -16) * np.abs(ref))


@pytest.mark.parametrize("T_", [1, 6, 20, 64])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_moe_large_inputs_with_finite_sums(T_, group, dtype):
    say(f"[gpu case] moe range T={T_} group={group} {dtype}")
    d, f = 128, 20
    x = torch.full((T_, d), 2e35, device="cuda").to(DT[dtype])
    w = torch.full((1, f, d), 1e-36, device="cuda")
    y, (g, u, dn) = _layer(T_, d, f, group, dtype, x, w, w, torch.full((1, d, f), 0.25, device="cuda"))
    x64 = host64(x)
    ref = ((x64 @ g.T) * (x64 @ u.T)) @ dn.T
    assert np.all(np.abs(y - ref) <= (REL[dtype] + 3 * 2.0 ** -16) * np.abs(ref))


@pytest.mark.parametrize("T_", [1, 6, 20, 100])
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_linear_infinite_inputs_and_sums_beyond_fp32(T_, group, dtype):
    """An infinite input makes its token's outputs NaN, no other token's; finite inputs whose sum is beyond fp32 give an
    infinity."""
    say(f"[gpu case] linear infinite T={T_} group={group} {dtype}")
    N, K = 70, 130
    wd = T.WDesc(1, N, K, 4, group)
    pl, v = _planes(torch.full((1, N, K), 0.5, device="cuda"), wd)
    x = torch.ones(T_, K, device="cuda").to(DT[dtype])
    x[T_ - 1, 3] = float("-inf")
    y = torch.empty(T_, N, dtype=DT[dtype], device="cuda")
    T.twell_linear_fwd(wd, pl, x, y)
    assert torch.isnan(y[T_ - 1]).all()
    ref = host64(x[:T_ - 1]) @ v[0].T
    assert np.all(np.abs(host64(y[:T_ - 1]) - ref) <= (REL[dtype] + 2.0 ** -16) * np.abs(ref))
    x[T_ - 1] = -2e38
    T.twell_linear_fwd(wd, pl, x, y)
    assert (y[T_ - 1] == float("-inf")).all() and torch.isfinite(y[:T_ - 1]).all()
