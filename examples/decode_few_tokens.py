"""Greedy decoding of a small mixture-of-experts model: the few-token operators as a serving step uses them.

Weights are laid out once; a step is then one call per layer (router, chosen experts, weighted sum) and one 4-bit
product for the logits.  The step is captured into a HIP graph, since the launches of a single token's step cost the
host more than the kernels take.  Random weights: the tokens mean nothing, the times do.

    python examples/decode_few_tokens.py [--batch 4] [--bits 4] [--steps 64]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import activation_sparse_feedforward_amd as A  # noqa: E402


class Decoder:
    """x = embedding[token]; x += moe(x / rms(x)) for each layer; logits = head(x / rms(x))."""

    def __init__(self, batch=4, d_model=1024, d_ff=512, experts=32, top_k=4, layers=4, vocab=8192, bits=4, group=64,
                 seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, scale):
            return (torch.randn(*shape, generator=g, device="cuda") * scale).bfloat16()

        self.batch, self.d_model = batch, d_model
        self.embedding = normal(vocab, d_model, scale=1.0)
        self.md = A.MoeDesc(batch, d_model, d_ff, experts, top_k, "bf16", bits, group if bits == 4 else 0, "silu", True)
        self.layers = []
        for _ in range(layers):
            w = A.alloc_moe_weights(self.md)
            A.twell_weights_pack(self.md.in_desc, normal(experts, d_ff, d_model, scale=d_model ** -0.5), w.gate)
            A.twell_weights_pack(self.md.in_desc, normal(experts, d_ff, d_model, scale=d_model ** -0.5), w.up)
            # w_down is kept with one row per neuron, the transposed form of its d_model x d_ff matrix
            A.twell_weights_pack(self.md.out_desc, normal(experts, d_ff, d_model, scale=d_ff ** -0.5), w.down,
                                 transposed=True)
            self.layers.append((normal(experts, d_model, scale=2 * d_model ** -0.5), w, A.alloc_moe_out(self.md)))
        self.ws = A.alloc_moe_ws(self.md)  # the layers run one after another and share it
        self.head_desc = A.WDesc(1, vocab, d_model, 4, group)
        self.head = A.alloc_weights(self.head_desc)
        A.twell_weights_pack(self.head_desc, normal(1, vocab, d_model, scale=d_model ** -0.5), self.head)
        self.x = torch.empty(batch, d_model, dtype=torch.bfloat16, device="cuda")
        self.logits = torch.empty(batch, vocab, dtype=torch.bfloat16, device="cuda")
        self.graph = None

    def _normed(self, x):
        return torch.nn.functional.rms_norm(x, (self.d_model,))

    def forward(self):
        """self.x [batch, d_model] to self.logits, on the current stream."""
        x = self.x
        for router, w, out in self.layers:
            A.twell_moe_fwd(self.md, self._normed(x), router, w, out, self.ws)
            x = x + out.y
        A.twell_linear_fwd(self.head_desc, self.head, self._normed(x), self.logits)

    def capture(self):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.forward()
        torch.cuda.current_stream().wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.forward()

    def step(self, tokens):
        """The next token of each sequence."""
        torch.index_select(self.embedding, 0, tokens, out=self.x)
        self.graph.replay() if self.graph else self.forward()
        return self.logits.argmax(-1)

    def generate(self, tokens, steps):
        got = []
        for _ in range(steps):
            tokens = self.step(tokens)
            got.append(tokens)
        return torch.stack(got, 1)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--bits", type=int, default=4, choices=(4, 16), help="of the experts' weights")
    ap.add_argument("--steps", type=int, default=64)
    args = ap.parse_args(argv)
    model = Decoder(batch=args.batch, bits=args.bits)
    start = torch.arange(args.batch, device="cuda")

    def timed(label):
        model.generate(start, 4)
        torch.cuda.synchronize()
        t = time.perf_counter()
        got = model.generate(start, args.steps)
        torch.cuda.synchronize()
        ms = (time.perf_counter() - t) * 1e3 / args.steps
        print(f"{label}: {ms:.3f} ms a step, {args.batch / ms * 1e3:.0f} tokens/s")
        return got

    eager = timed("launched")
    model.capture()
    graph = timed("replayed")
    print("same tokens:", bool((eager == graph).all()))
    print("first sequence:", graph[0, :12].tolist())
    return eager, graph


if __name__ == "__main__":
    main()
