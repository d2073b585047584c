"""An MoE block as it is served: tokens are routed to experts, and the experts run in e4m3 with block scales.

    python examples/moe_fp8.py                          # 8 experts of 4096 x 14336, top-2
    python examples/moe_fp8.py --experts 64 --dim 2048 --ff 1000 --top-k 6 --score sigmoid --groups 8

The tokens come out of a projection in e4m3 (``PopQLinear``). The router's logits are a plain float32 product, as the choice
of experts hangs on their order, which 8-bit operands would change; ``PopRouter`` chooses experts and weights, with
a bias that evens out their load (moved after every batch against the counts, as a trainer would); ``PopQMoE`` runs the
chosen experts. A prompt is followed by decode steps of a few tokens, the last of them replayed as a CUDA graph.
"""
from __future__ import annotations

import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def weights(g, n, k):
    """A random bf16 matrix of N(0, 0.02^2)."""
    import torch
    return (torch.randn((n, k), generator=g, device="cuda") * 0.02).to(torch.bfloat16)


class Gate:
    """A token's logit for each expert, in float32."""

    def __init__(self, w):
        self.w = w.float().t().contiguous()

    def forward(self, x):
        return x.float() @ self.w


class Block:
    """Router and experts with random weights."""

    def __init__(self, experts, dim, ff, top_k, score="softmax", groups=1, max_tokens=4096, seed=0):
        import torch

        import online_structured_ffn_gb300 as pop
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def some(n, k):
            return [weights(g, n, k) for _ in range(experts)]

        self.gate = Gate(weights(g, experts, dim))
        self.router = pop.PopRouter(experts, top_k, score=score, n_groups=groups, top_groups=max(1, groups // 2),
                                    group_sum=2 if score == "sigmoid" and groups > 1 else 1)
        self.bias = torch.zeros((experts,), device="cuda") if score == "sigmoid" else None
        self.counts = torch.zeros((experts,), dtype=torch.int32, device="cuda")
        self.ffn = pop.PopQMoE(some(ff, dim), some(ff, dim), some(dim, ff), top_k=top_k, max_tokens=max_tokens)

    def forward(self, x, balance=0.0):
        """x: bf16 [T, dim]. Returns (y bf16 [T, dim], experts, weights)."""
        experts, weights = self.router.route(self.gate.forward(x), bias=self.bias, counts=self.counts)
        if balance and self.bias is not None:  # experts with more than their share become less attractive
            self.bias -= balance * (self.counts.float() - self.counts.float().mean()).sign()
        return self.ffn.forward(x, experts, weights), experts, weights

    def check(self):
        self.ffn.check()


def main(argv=None):
    import torch

    import online_structured_ffn_gb300 as pop
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--experts", type=int, default=8)
    p.add_argument("--dim", type=int, default=4096)
    p.add_argument("--ff", type=int, default=14336)
    p.add_argument("--top-k", type=int, default=2)
    p.add_argument("--score", choices=["softmax", "sigmoid"], default="softmax")
    p.add_argument("--groups", type=int, default=1)
    p.add_argument("--prompt", type=int, default=4096)
    p.add_argument("--batch", type=int, default=32)
    p.add_argument("--steps", type=int, default=20)
    a = p.parse_args(argv)
    block = Block(a.experts, a.dim, a.ff, a.top_k, a.score, a.groups, max_tokens=max(a.prompt, a.batch))
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    before = pop.PopQLinear(weights(g, a.dim, a.dim), max_tokens=max(a.prompt, a.batch))

    def step(x, balance=0.0):
        return block.forward(before.forward(x), balance)

    def tokens(n):
        return torch.randn((n, a.dim), generator=g, device="cuda").to(torch.bfloat16)

    def timed(name, n, f):
        f()
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        for _ in range(a.steps):
            f()
        end.record()
        torch.cuda.synchronize()
        print(f"{name}: {n} tokens in {start.elapsed_time(end) / a.steps * 1e3:.1f} us")

    x = tokens(a.prompt)
    timed("prompt", a.prompt, lambda: step(x, balance=0.001))
    load = block.counts.float()
    print(f"experts' load: mean {load.mean():.0f}, most {load.max():.0f}, least {load.min():.0f}")
    x1 = tokens(a.batch)
    timed("decode step", a.batch, lambda: step(x1))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        y, _, _ = step(x1)
    timed("decode step as a graph", a.batch, graph.replay)
    before.check()
    block.check()
    return y


if __name__ == "__main__":
    main()
