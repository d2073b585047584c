"""Calls after one that the CUDA runtime refused: they are answered for themselves."""
import pytest

from test_gpu_quant import env  # noqa: F401

pytestmark = pytest.mark.gpu


def refused(env):
    """An experts' handle for 2^20 tokens through 16 slots of 65,536 channels each: its workspace would be 1 TB."""
    pop, torch, dev = env
    w, w2 = torch.zeros((65536, 8), dtype=torch.bfloat16, device=dev), torch.zeros((8, 65536), dtype=torch.bfloat16, device=dev)
    with pytest.raises(pop.PopError) as e:
        pop.PopQMoE([w], [w], [w2], top_k=16, max_tokens=1 << 20)
    assert e.value.status == pop.POP_ERR_OOM


def test_calls_after_an_allocation_that_failed(env):
    pop, torch, dev = env
    refused(env)
    e, w = pop.PopRouter(8, 2).route(torch.arange(8.0, device=dev)[None])
    assert e.tolist() == [[7, 6]]
    refused(env)
    W = (448 * torch.eye(16, device=dev)).to(torch.bfloat16)  # scales of 1: everything is exact
    h = pop.PopQLinear(W, max_tokens=2, out_f32=True)
    assert torch.equal(h.forward(W[:1]), 448 * W[:1].float())
    refused(env)
    m = pop.PopQMoE([W], [W], [W], top_k=1, max_tokens=2)
    refused(env)
    zero, one = torch.zeros((1, 1), dtype=torch.int32, device=dev), torch.ones((1, 1), device=dev)
    assert m.forward(W[:1], zero, one).shape == (1, 16)
    q, s = pop.quantize_rows(W)
    assert float(q[0, 0].float() * s[0, 0]) == 448
    h.check()
    m.check()


def test_the_pruned_layer_after_an_allocation_that_failed(env):
    pop, torch, dev = env
    refused(env)
    g = torch.Generator(device=dev)
    g.manual_seed(0)
    w = [(torch.randn(shape, generator=g, device=dev) * 0.05).to(torch.bfloat16) for shape in ((256, 128), (256, 128), (128, 256))]
    f = pop.PopFFN(*w, r=0.3, gamma=0.1, max_batch=1, max_prefill_tokens=8)
    f.close()
