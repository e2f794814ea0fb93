"""The decoding example: its operators together against a 64-bit model, launched and as a replayed graph."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import _few_token as R
from activation_sparse_feedforward_amd import twell as T
from _helpers import host64, say

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "decode_few_tokens.py")


def _example():
    spec = importlib.util.spec_from_file_location("decode_few_tokens", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _values(desc, planes):
    w = torch.empty(desc.experts, desc.rows, desc.cols, dtype=torch.float32 if desc.bits == 4 else torch.bfloat16,
                    device="cuda")
    T.twell_weights_unpack(desc, planes, w)
    return host64(w)


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("batch", [1, 3, 7])
def test_decoding_step(batch, bits):
    say(f"[gpu case] decoding example batch={batch} bits={bits}")
    m = _example().Decoder(batch=batch, d_model=200, d_ff=130, experts=12, top_k=3, layers=2, vocab=500, bits=bits)
    tokens = torch.arange(batch, device="cuda") * 37
    m.step(tokens)
    launched = m.logits.clone()

    # every layer from the input that it had: its choices are those of that input
    x = m.embedding[tokens]
    for router, w, out in m.layers:
        n = m._normed(x)
        T.twell_moe_fwd(m.md, n, router, w, out, m.ws)
        ids, wts = R.route(host64(n), host64(router), None, 3, True)
        assert np.array_equal(out.ids.cpu().numpy(), ids)
        ref = R.moe(host64(n), ids, wts, _values(m.md.in_desc, w.gate), _values(m.md.in_desc, w.up),
                    _values(m.md.out_desc, w.down), "silu")
        got = host64(out.y)
        # one rounding to bf16 and, ahead of it, the hidden values' to 16 bits
        assert np.linalg.norm(got - ref) <= (2.0 ** -8 + 2.0 ** -15) * np.linalg.norm(ref)
        x = x + out.y
    ref = host64(m._normed(x)) @ _values(m.head_desc, m.head)[0].T
    assert np.linalg.norm(host64(launched) - ref) <= (2.0 ** -8 + 1e-5) * np.linalg.norm(ref)

    # replays, each after other inputs and eager work, give the launched results
    m.capture()
    for _ in range(3):
        m.step((tokens + 1) % 500)
        m.forward()
        torch.cuda.synchronize()
        m.step(tokens)
        assert torch.equal(m.logits, launched)


def test_decoding_example_runs():
    eager, graph = _example().main(["--steps", "4", "--batch", "2"])
    assert torch.equal(eager, graph) and eager.shape == (2, 4)
