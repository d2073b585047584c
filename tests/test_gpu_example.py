"""The example MoE block: it runs, and its output is that of its parts."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    import torch

    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    spec = importlib.util.spec_from_file_location("moe_fp8", os.path.join(ROOT, "examples", "moe_fp8.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("args", [["--experts", "8"], ["--experts", "16", "--score", "sigmoid", "--groups", "4", "--top-k", "3"]])
def test_example_runs(example, args, capsys):
    y = example.main(args + ["--dim", "256", "--ff", "200", "--prompt", "300", "--batch", "8", "--steps", "2"])
    out = capsys.readouterr().out
    assert "prompt: 300 tokens" in out and "as a graph: 8 tokens" in out
    assert bool(y.float().isfinite().all()) and float(y.float().abs().max()) > 0


def test_block_is_its_parts(example):
    import torch

    import online_structured_ffn_gb300 as pop
    block = example.Block(8, 256, 200, 2, max_tokens=64)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x = torch.randn((40, 256), generator=g, device="cuda").to(torch.bfloat16)
    y, e, w = block.forward(x)
    logits = block.gate.forward(x)
    assert torch.equal(torch.topk(logits, 2, dim=1)[0], torch.gather(logits, 1, e.long()))
    assert torch.allclose(w, torch.softmax(torch.gather(logits, 1, e.long()), dim=1), atol=1e-6)
    assert torch.equal(block.counts.long(), torch.bincount(e.reshape(-1).long(), minlength=8))
    # each token's two experts one at a time, weighted and added: the same to bf16's rounding of the parts
    only = pop.PopRouter(8, 1)
    parts = torch.zeros((40, 256), device="cuda")
    none = torch.full((40, 1), -1, dtype=torch.int32, device="cuda")
    for j in range(2):
        slots = torch.cat([e[:, j:j + 1], none], dim=1).contiguous()
        parts += block.ffn.forward(x, slots, torch.cat([w[:, j:j + 1], torch.zeros_like(w[:, :1])], dim=1).contiguous()).float()
    err = (parts - y.float()).norm() / y.float().norm()
    assert float(err) < 2.0 ** -7
    assert only.route(logits)[0].shape == (40, 1)
    block.check()
