"""The binding refuses matrices of another shape than the call's, though their bytes would do."""
import pytest
import torch

from activation_sparse_feedforward_amd import twell as T
from _helpers import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits,group", [(4, 64), (16, 0)])
def test_pack_and_unpack_refuse_other_shapes(bits, group):
    say(f"[gpu case] shapes of matrices, {bits} bits")
    E, N, K = 3, 32, 160
    wd = T.WDesc(E, N, K, bits, group)
    pl = T.alloc_weights(wd)
    w = torch.randn(E, N, K, device="cuda").bfloat16()
    t = w.transpose(1, 2).contiguous()
    other = [t, w.view(N, E, K), w.view(E * N, K), w.view(E, N * K), torch.cat([w, w]), torch.cat([w, w]).view(-1)]
    for bad in other:
        with pytest.raises(ValueError, match="shape"):
            T.twell_weights_pack(wd, bad, pl)
        with pytest.raises(ValueError, match="shape"):
            T.twell_weights_unpack(wd, pl, torch.empty_like(bad))
    with pytest.raises(ValueError, match="shape"):
        T.twell_weights_pack(wd, w, pl, transposed=True)
    # a flat buffer says nothing of rows and columns; one matrix needs no axis of experts
    T.twell_weights_pack(wd, w, pl)
    flat, flat_t, back = T.alloc_weights(wd), T.alloc_weights(wd), torch.empty(E * N * K, device="cuda").bfloat16()
    T.twell_weights_pack(wd, w.view(-1), flat)
    T.twell_weights_pack(wd, t.view(-1), flat_t, transposed=True)
    assert torch.equal(flat.codes, pl.codes) and torch.equal(flat_t.codes, pl.codes)
    T.twell_weights_unpack(wd, pl, back)
    one = T.WDesc(1, N, K, bits, group)
    single = T.alloc_weights(one)
    T.twell_weights_pack(one, w[0], single)
    assert torch.equal(single.codes, pl.codes[:single.codes.numel()])
    if bits == 16:
        assert torch.equal(back.view(E, N, K), w)


def test_moe_refuses_other_routers():
    say("[gpu case] shapes of routers")
    md = T.MoeDesc(2, 64, 32, 8, 2, "bf16", 4, 32)
    w = T.alloc_moe_weights(md)
    for desc, p in zip((md.in_desc, md.in_desc, md.out_desc), w):
        T.twell_weights_pack(desc, torch.randn(8, desc.rows, desc.cols, device="cuda"), p)
    x, router = (torch.randn(n, 64, device="cuda").bfloat16() for n in (2, 8))
    bias = torch.zeros(8, device="cuda")
    out, ws = T.alloc_moe_out(md), T.alloc_moe_ws(md)
    for bad in (router.t().contiguous(), router.view(4, 128), torch.cat([router, router])):
        with pytest.raises(ValueError, match="w_router: shape"):
            T.twell_moe_fwd(md, x, bad, w, out, ws)
    for bad in (torch.zeros(9, device="cuda"), torch.zeros(2, 8, device="cuda")):
        with pytest.raises(ValueError, match="router_bias: shape"):
            T.twell_moe_fwd(md, x, router, w, out, ws, router_bias=bad)
    T.twell_moe_fwd(md, x, router, w, out, ws, router_bias=bias)
    again = T.alloc_moe_out(md)
    T.twell_moe_fwd(md, x, router.view(-1), w, again, ws, router_bias=bias.view(1, 8))
    assert all(torch.equal(a, b) for a, b in zip(out, again))
