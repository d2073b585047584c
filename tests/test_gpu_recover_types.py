"""The example's function with gradients on handles whose outputs and gradients are float32: autograd hands it a float32 dy
then, and takes gradients of a leaf in the leaf's own type. Where no gradient is wanted nothing is kept."""
import pytest

from test_gpu_gated import env, make, near, reference  # noqa: F401
from test_gpu_recover import example  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("grad_f32", [False, True])
@pytest.mark.parametrize("M,D,N", [(5, 64, 136), (150, 264, 520)])
def test_gradients_through_autograd_of_float32_outputs(env, example, M, D, N, grad_f32):  # noqa: F811
    pop, torch, dev = env
    t = make(env, 60, M, D, N)
    f = pop.PopGatedFFN(D, N, max_tokens=M, out_f32=True, grad_f32=grad_f32)
    leaves = [t[n].clone().requires_grad_() for n in ("x", "Wg", "W1", "W2")]
    y = example.Gated.apply(*leaves, f)
    assert y.dtype == torch.float32
    y.backward(t["dy"].float())  # (exact in bf16: the reference has the same dy)
    want = reference(t)
    near(y.detach(), want["y"], "y")
    for name, leaf in zip(("dx", "dWg", "dW1", "dW2"), leaves):
        assert leaf.grad.dtype == torch.bfloat16
        near(leaf.grad, want[name], name)
    # one that is not is rounded to bf16 first
    g = torch.Generator(device=dev)
    g.manual_seed(61)
    dy = torch.randn((M, D), generator=g, device=dev)
    got = torch.autograd.grad(example.Gated.apply(*leaves, f), leaves, dy)
    again = torch.autograd.grad(example.Gated.apply(*leaves, f), leaves, dy.to(torch.bfloat16).float())
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    f.check()
    f.close()


def test_nothing_is_kept_where_no_gradient_is_wanted(env, example, monkeypatch):  # noqa: F811
    pop, torch, dev = env
    M, D, N = 20, 64, 136
    t = make(env, 62, M, D, N)
    f = pop.PopGatedFFN(D, N, max_tokens=M)
    asked = []
    forward = f.forward

    def watched(*args, **kw):
        asked.append(bool(kw.get("save")))
        return forward(*args, **kw)

    monkeypatch.setattr(f, "forward", watched)
    args = [t[n] for n in ("x", "Wg", "W1", "W2")]
    y = example.Gated.apply(*args, f)
    assert asked == [False] and not y.requires_grad and torch.equal(y, forward(*args))
    z = example.Gated.apply(args[0], args[1].clone().requires_grad_(), *args[2:], f)
    assert asked == [False, True] and z.requires_grad and torch.equal(y, z)
    f.close()
