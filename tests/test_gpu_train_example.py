"""The training example runs, its gradients are those of the layer in 64 bits up to the 8-bit roundings, and a step
replayed from a HIP graph is the launched one."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples"))
import train_experts  # noqa: E402
from _helpers import say  # noqa: E402
from _many_token import capture  # noqa: E402

pytestmark = pytest.mark.gpu


def test_example_runs():
    say("[gpu case] training example")
    losses = train_experts.main(["--tokens", "512", "--experts", "8", "--steps", "3"])
    assert len(losses) == 4 and all(torch.isfinite(v) for v in losses)


def _reference(layer, x, dy):
    """y and gradients of everything by autograd in 64 bits, at the layer's own choice of experts."""
    w = {n: v.double().requires_grad_() for n, v in layer.weights.items()}
    x = x.double().requires_grad_()
    d = x.shape[1]
    n = torch.nn.functional.layer_norm(x, (d,), w["norm"], w["bias"], 1e-5)
    weights = torch.softmax(n @ w["router"].T, -1).gather(1, layer.ids)
    y = x
    for e in range(layer.tokens.experts):
        row, slot = (layer.ids == e).nonzero(as_tuple=True)
        r = n[row]
        h = torch.relu(r @ w["gate"][e].T) * (r @ w["up"][e].T)
        y = y.index_add(0, row, weights[row, slot].unsqueeze(1) * (h @ w["down"][e].T))
    y.backward(dy.double())
    return y, {"x": x.grad, **{k: v.grad for k, v in w.items()}}


@pytest.mark.parametrize("tokens,d,f,experts,k", [(300, 256, 128, 8, 2), (1000, 130, 72, 5, 3)])
def test_gradients(tokens, d, f, experts, k):
    """An e4m3 value is off by up to 2^-4 of itself, 3.6 % in the mean of squares of an even spread, and a product rounds
    two operands: 5.1 %.  y, down, up and router have up to three such products behind them, whose errors add as squares:
    8.8 %, and 12.5 % if all six of the layer were.  The gate's gradient has another part: relu's derivative is wrong
    where g's error is larger than g.  For two normal values of which one is 5.1 % of the other that happens to
    atan(0.051) / pi = 1.6 % of all entries, in both directions, while half of the entries make up the gradient's norm:
    sqrt(0.016 / 0.5) = 18 %, with the errors of dh and u, 5.1 % each, 19.4 %.  It goes on into dx and the norm's
    weights, which have the residual's and the other projection's parts beside it."""
    say(f"[gpu case] training example's gradients {tokens} x {d} x {f}, {k} of {experts}")
    layer = train_experts.ExpertLayer(tokens, d, f, experts, k, seed=4)
    g = torch.Generator(device="cuda").manual_seed(5)
    x, dy = (torch.randn(tokens, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    layer.pack()
    layer.forward(x)
    layer.backward(dy)
    y, grads = _reference(layer, x, dy)
    got = {"x": layer.dx, **layer.grads}
    assert (layer.y.double() - y).norm() <= 0.15 * y.norm()
    for name, want in grads.items():
        off = float((got[name].double() - want).norm() / want.norm())
        assert off <= (0.2 if name in ("gate", "x", "norm", "bias") else 0.15), (name, off)


def test_replayed_step_is_the_launched_one():
    say("[gpu case] training example's step as a graph")
    g = torch.Generator(device="cuda").manual_seed(6)
    xs = [torch.randn(700, 256, generator=g, device="cuda").bfloat16() for _ in range(2)]
    dy = torch.randn(700, 256, generator=g, device="cuda").bfloat16()
    layer = train_experts.ExpertLayer(700, 256, 128, 8, 2, seed=7)
    now = xs[0].clone()

    def step():
        layer.pack()
        layer.forward(now)
        layer.backward(dy)

    want = []
    for x in xs:
        now.copy_(x)
        step()
        torch.cuda.synchronize()
        want.append([layer.y.clone(), layer.dx.clone(), *(v.clone() for v in layer.grads.values())])
    graph = capture(step)
    for turn in (1, 0, 1):
        now.copy_(xs[turn])
        for v in (layer.y, layer.dx, *layer.grads.values()):
            v.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        got = [layer.y, layer.dx, *layer.grads.values()]
        for i, (a, b) in enumerate(zip(got, want[turn])):
            assert torch.equal(a, b), (turn, i)
