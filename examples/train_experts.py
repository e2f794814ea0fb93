"""Training a mixture-of-experts feed-forward layer: layer norm, router, tokens sorted to their experts, 8-bit products,
the weighted sum, and back.

    y = x + combine(W_down (relu(W_gate r) * (W_up r))),  r = gather(norm(x)) sorted by expert

The layer learns to imitate another one (random weights), with plain gradient steps on fp32 weights that are packed to
8 bits anew in every step.  Router and activation are elementary torch operations.  A step can be captured into a HIP
graph: no size in it depends on where tokens go.

    python examples/train_experts.py [--tokens 4096] [--experts 16] [--steps 20]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import activation_sparse_feedforward_amd as A  # noqa: E402


class ExpertLayer:
    """One layer with its weights, their gradients and everything that a step of ``tokens`` rows keeps."""

    def __init__(self, tokens=4096, d_model=512, d_ff=256, experts=16, top_k=2, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        T, d, f, E, k, P = tokens, d_model, d_ff, experts, top_k, tokens * top_k

        def normal(*shape, scale):
            return torch.randn(*shape, generator=g, device="cuda") * scale

        def rows(n, width):
            return torch.zeros(n, width, dtype=torch.bfloat16, device="cuda")

        self.weights = dict(norm=torch.ones(d, device="cuda"), bias=torch.zeros(d, device="cuda"),
                            router=normal(E, d, scale=d ** -0.5), gate=normal(E, f, d, scale=d ** -0.5),
                            up=normal(E, f, d, scale=d ** -0.5), down=normal(E, d, f, scale=f ** -0.5))
        self.grads = {name: torch.zeros_like(w) for name, w in self.weights.items()}
        self.norm, self.tokens = A.NormDesc(T, d, "bf16"), A.TokensDesc(T, d, E, k, "bf16")
        self.matrices = dict(gate=A.Fp8Desc(E, f, d), up=A.Fp8Desc(E, f, d), down=A.Fp8Desc(E, d, f))
        self.planes = {name: (A.alloc_fp8_weights(m), A.alloc_fp8_weights(m.transposed))
                       for name, m in self.matrices.items()}
        self.order, self.sort_ws = A.alloc_tokens_order(self.tokens), A.alloc_tokens_ws(self.tokens)
        self.norm_ws = A.alloc_norm_ws(self.norm)
        self.ws = torch.empty(max(A.fp8_ws_bytes(m, P) for m in self.matrices.values()), dtype=torch.uint8, device="cuda")
        self.n, self.y, self.dn, self.dx = (rows(T, d) for _ in range(4))
        self.stats = torch.empty(T, 2, device="cuda")
        self.r, self.z, self.dz, self.dr, self.dr_up = (rows(P, d) for _ in range(5))
        self.g, self.u, self.dh = (rows(P, f) for _ in range(3))
        self.dw = torch.empty(T, k, device="cuda")

    def pack(self):
        for name, m in self.matrices.items():
            A.twell_fp8_weights_pack(m, self.weights[name], *self.planes[name])

    def _product(self, name, x, y):
        A.twell_fp8_linear_fwd(self.matrices[name], self.planes[name][0], x, y, self.ws, offsets=self.order.offsets)

    def _gradients(self, name, x, dy, dx):
        A.twell_fp8_linear_bwd(self.matrices[name], self.planes[name][1], x, dy, dx, self.grads[name], self.ws,
                               offsets=self.order.offsets)

    def forward(self, x):
        """self.y of x [tokens, d_model], from packed weights."""
        self.x = x
        A.twell_layernorm_fwd(self.norm, x, self.weights["norm"], self.weights["bias"], self.n, self.stats)
        self.p = torch.softmax(self.n.float() @ self.weights["router"].T, -1)
        w, ids = self.p.topk(self.tokens.top_k, -1)
        self.w, self.ids = w.contiguous(), ids
        A.twell_tokens_sort(self.tokens, ids.to(torch.int32), self.order, self.sort_ws)
        A.twell_tokens_gather(self.tokens, self.n, self.order, self.r)
        self._product("gate", self.r, self.g)
        self._product("up", self.r, self.u)
        self.h = torch.relu(self.g) * self.u
        self._product("down", self.h, self.z)
        A.twell_tokens_combine(self.tokens, self.z, self.order, self.w, self.y)
        self.y += x
        return self.y

    def backward(self, dy):
        """self.dx and self.grads for the gradient dy of the last forward's y."""
        A.twell_tokens_combine_bwd(self.tokens, self.z, self.order, self.w, dy, self.dz, self.dw)
        self._gradients("down", self.h, self.dz, self.dh)
        self._gradients("gate", self.r, self.dh * self.u * (self.g > 0), self.dr)
        self._gradients("up", self.r, self.dh * torch.relu(self.g), self.dr_up)
        self.dr += self.dr_up
        A.twell_tokens_combine(self.tokens, self.dr, self.order, None, self.dn)
        # softmax over all experts, of which the chosen ones' probabilities are the weights
        dp = torch.zeros_like(self.p).scatter(1, self.ids, self.dw)
        dl = self.p * (dp - (self.p * dp).sum(1, keepdim=True))
        torch.mm(dl.T, self.n.float(), out=self.grads["router"])
        self.dn += (dl @ self.weights["router"]).bfloat16()
        A.twell_layernorm_bwd(self.norm, self.x, self.weights["norm"], self.stats, self.dn, self.dx,
                              self.grads["norm"], self.grads["bias"], self.norm_ws)
        self.dx += dy
        return self.dx

    def step(self, x, target, rate):
        """One gradient step towards target; the loss before it."""
        self.pack()
        e = self.forward(x).float() - target.float()
        self.backward((e * (2 / e.numel())).bfloat16())
        for name, w in self.weights.items():
            w.sub_(self.grads[name], alpha=rate)
        return (e * e).mean()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--steps", type=int, default=20)
    args = ap.parse_args(argv)
    teacher = ExpertLayer(args.tokens, experts=args.experts, seed=1)
    layer = ExpertLayer(args.tokens, experts=args.experts, seed=2)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(args.tokens, teacher.norm.d_model, generator=g, device="cuda").bfloat16()
    teacher.pack()
    target = teacher.forward(x).clone()
    losses = [layer.step(x, target, 100.0)]
    torch.cuda.synchronize()
    t = time.perf_counter()
    losses += [layer.step(x, target, 100.0) for _ in range(args.steps)]
    torch.cuda.synchronize()
    ms = (time.perf_counter() - t) * 1e3 / args.steps
    print(f"{ms:.3f} ms a step, {args.tokens / ms * 1e3:.0f} tokens/s")
    print("loss:", " ".join(f"{float(v):.4f}" for v in losses[:: max(1, args.steps // 8)]))
    return losses


if __name__ == "__main__":
    main()
