"""The example that prunes, trains and quantises a layer: it runs, its gradients are the operator's and the formula's, and what it
serves is what its parts give."""
import importlib.util
import os

import pytest

from test_gpu_gated import env, make, near, reference  # noqa: F401
from test_gpu_int8 import steps

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example(env):  # noqa: F811
    spec = importlib.util.spec_from_file_location("recover_int8", os.path.join(ROOT, "examples", "recover_int8.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("args", [["--tokens", "128", "--batch", "3"], ["--tokens", "300", "--batch", "40", "--rate", "0.5"]])
def test_example_runs(example, args, capsys):
    import torch
    y, losses = example.main(["--dim", "256", "--ff", "1024", "--steps", "3"] + args)
    out = capsys.readouterr().out
    assert "kept" in out and "in 8-bit integers" in out and "as a graph" in out
    assert bool(torch.isfinite(y.float()).all()) and all(float(v) > 0 for v in losses)


@pytest.mark.parametrize("M,D,N", [(5, 64, 136), (150, 264, 520)])
def test_gradients_through_autograd(env, example, M, D, N):  # noqa: F811
    pop, torch, dev = env
    t = make(env, 1, M, D, N)
    f = pop.PopGatedFFN(D, N, max_tokens=M)
    leaves = [t[n].clone().requires_grad_() for n in ("x", "Wg", "W1", "W2")]
    y = example.Gated.apply(*leaves, f)
    y.backward(t["dy"])
    want = reference(t)
    near(y.detach(), want["y"], "y")
    for name, leaf in zip(("dx", "dWg", "dW1", "dW2"), leaves):
        near(leaf.grad, want[name], name)
    # a leaf that needs none, and the step captured into a graph of its own while these leaves live
    frozen = [leaves[0].detach(), leaves[1].detach().requires_grad_(), leaves[2].detach(), leaves[3].detach().requires_grad_()]
    for _ in range(2):
        example.Gated.apply(*frozen, f).backward(t["dy"])
    assert frozen[0].grad is None and frozen[2].grad is None
    near(frozen[1].grad / 2, want["dWg"], "dWg")
    f.close()


def test_a_trained_layer_served_in_integers(env, example):  # noqa: F811
    """One after the other as they are used: forward, backward, an update, quantising, the integer layer, and its first product by
    itself."""
    pop, torch, dev = env
    M, D, N = 70, 136, 264
    t = make(env, 2, M, D, N)
    w = [t[n] for n in ("Wg", "W1", "W2")]
    batches = [make(env, 3 + i, M, D, N)["x"] for i in range(3)]
    trained, losses = example.train(w, batches, [0.5 * t["dy"]] * 3, 1e-3)
    assert len(losses) == 3 and all(not torch.equal(a, b) for a, b in zip(trained, w))
    inside, given = pop.PopI8FFN(*trained, max_tokens=M), pop.PopI8FFN(*(pop.quantize_rows_i8(m) for m in trained), max_tokens=M)
    x = t["x"]
    assert torch.equal(inside.forward(x), given.forward(x))
    gate = pop.PopI8Linear(trained[0], max_tokens=M, out_f32=True)
    (xq, xs), (q, s) = steps(x), steps(trained[0])
    exact = xs.double()[:, None] * s.double() * (xq.double() @ q.double().t())
    got = gate.forward(x).double()
    assert float((got - exact).abs().max()) <= 4 * 2.0 ** -24 * float(exact.abs().max())
    for h in (inside, given, gate):
        h.check()
        h.close()
