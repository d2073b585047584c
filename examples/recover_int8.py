"""A gated MLP that is pruned, trained to do what it did before, and served in 8-bit integers.

    python examples/recover_int8.py                     # 4096 x 11008, 30 % of the channels gone
    python examples/recover_int8.py --dim 256 --ff 1024 --tokens 128 --steps 20

``PopFFN`` ranks the channels of a dense layer over a prompt; the pruned third state's are taken out of the matrices for
good. ``PopGatedFFN`` trains what is left against the dense layer's outputs (``Gated`` is it as a function with
gradients for autograd; weights are kept in float32 and rounded for each step). ``PopI8FFN`` then quantises the trained matrices, a
scale per channel, and serves a prompt and decode steps, the last of them as a CUDA graph.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


class Gated(torch.autograd.Function):
    """``PopGatedFFN`` with gradients of x and the three matrices: Gated.apply(x, Wg, W1, W2, ffn). The gradient that comes in is
    rounded to bf16."""

    @staticmethod
    def forward(ctx, x, Wg, W1, W2, ffn):
        if not any(ctx.needs_input_grad):
            return ffn.forward(x, Wg, W1, W2)
        y, saved = ffn.forward(x, Wg, W1, W2, save=True)
        ctx.save_for_backward(x, Wg, W1, W2, saved)
        ctx.ffn = ffn
        return y

    @staticmethod
    def backward(ctx, dy):
        x, Wg, W1, W2, saved = ctx.saved_tensors
        dy = dy.to(torch.bfloat16).contiguous()  # (of float32 outputs it is float32)
        return (*ctx.ffn.backward(dy, x, Wg, W1, W2, saved, need=ctx.needs_input_grad[:4]), None)


def kept_channels(Wg, W1, W2, prompt, rate):
    """The channels that pruning at `rate` leaves (retained or candidates), a multiple of 8 of them, in order."""
    import numpy as np

    import online_structured_ffn_gb300 as pop
    layer = pop.PopFFN(Wg, W1, W2, r=rate, gamma=0.0, max_prefill_tokens=prompt.shape[0])
    layer.prefill_partition(prompt)
    layer.check()
    R, C, P = layer.partition()
    layer.close()
    keep = np.sort(np.concatenate([R, C]))
    return torch.as_tensor(keep[:len(keep) // 8 * 8].astype("int64"), device=Wg.device)


def train(weights, batches, targets, lr):
    """Gradient steps on float32 copies of `weights`, one for each batch. Returns (bf16 matrices, losses)."""
    import online_structured_ffn_gb300 as pop
    N, D = weights[0].shape
    ffn = pop.PopGatedFFN(D, N, max_tokens=batches[0].shape[0])
    master = [w.float() for w in weights]
    losses = []
    for x, want in zip(batches, targets):
        leaves = [w.to(torch.bfloat16).requires_grad_() for w in master]
        y = Gated.apply(x, *leaves, ffn)
        loss = (y.float() - want.float()).square().mean() / want.float().square().mean()
        loss.backward()
        for w, leaf in zip(master, leaves):
            g = leaf.grad.float()
            w -= lr * w.norm() / g.norm().clamp(min=1e-30) * g
        losses.append(loss.detach())
    ffn.check()
    ffn.close()
    return [w.to(torch.bfloat16) for w in master], losses


def main(argv=None):
    import online_structured_ffn_gb300 as pop
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--dim", type=int, default=4096)
    p.add_argument("--ff", type=int, default=11008)
    p.add_argument("--rate", type=float, default=0.3)
    p.add_argument("--tokens", type=int, default=2048)
    p.add_argument("--batch", type=int, default=16)
    p.add_argument("--steps", type=int, default=50)
    p.add_argument("--lr", type=float, default=2e-3)
    a = p.parse_args(argv)
    g = torch.Generator(device="cuda")
    g.manual_seed(0)

    def rand(n, k, s=1.0):
        return (torch.randn((n, k), generator=g, device="cuda") * s).to(torch.bfloat16)

    dense = [rand(a.ff, a.dim, a.dim ** -0.5), rand(a.ff, a.dim, a.dim ** -0.5), rand(a.dim, a.ff, a.ff ** -0.5)]
    whole = pop.PopGatedFFN(a.dim, a.ff, max_tokens=a.tokens)
    keep = kept_channels(*dense, rand(a.tokens, a.dim), a.rate)
    small = [dense[0][keep].contiguous(), dense[1][keep].contiguous(), dense[2][:, keep].contiguous()]
    batches = [rand(a.tokens, a.dim) for _ in range(a.steps)]
    trained, losses = train(small, batches, [whole.forward(x, *dense) for x in batches], a.lr)
    print(f"{a.ff} channels, {len(keep)} kept; error of the outputs: first step {float(losses[0]):.4f}, last {float(losses[-1]):.4f}")

    served = pop.PopI8FFN(*trained, max_tokens=a.tokens)
    x = rand(a.tokens, a.dim)
    want = whole.forward(x, *dense).float()
    print(f"in 8-bit integers: {float((served.forward(x).float() - want).square().mean() / want.square().mean()):.4f}")

    def timed(name, n, f):
        f()
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        for _ in range(20):
            f()
        end.record()
        torch.cuda.synchronize()
        print(f"{name}: {n} tokens in {start.elapsed_time(end) / 20 * 1e3:.1f} us")

    timed("prompt", a.tokens, lambda: served.forward(x))
    x1 = rand(a.batch, a.dim)
    timed("decode step", a.batch, lambda: served.forward(x1))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        y = served.forward(x1)
    timed("decode step as a graph", a.batch, graph.replay)
    whole.check()
    served.check()
    return y, losses


if __name__ == "__main__":
    main()
