"""A gradient of the gated MLP has the same bits whichever others are asked for: its sum over the rows is split by the sizes
alone. On 152 SMs one, two and three matrices' gradients of these sizes are numbers of tiles that would be shared by different
numbers of CTAs if they were counted."""
import pytest

from test_gpu_gated import env, make, near, reference  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("grad_f32", [True, False])
@pytest.mark.parametrize("M,D,N", [(512, 512, 1024), (512, 1024, 1024), (600, 264, 1032), (1000, 264, 2056), (4096, 256, 256)])
def test_bits_do_not_depend_on_what_else_is_asked_for(env, M, D, N, grad_f32):  # noqa: F811
    pop, torch, dev = env
    t = make(env, 40, M, D, N)
    w = (t["Wg"], t["W1"], t["W2"])
    f = pop.PopGatedFFN(D, N, max_tokens=M, grad_f32=grad_f32)
    y, saved = f.forward(t["x"], *w, save=True)
    every = f.backward(t["dy"], t["x"], *w, saved)
    want = reference(t)
    for name, got in zip(("dx", "dWg", "dW1", "dW2"), every):
        near(got, want[name], name)
    zeros = [torch.zeros_like(g) for g in every[1:]]
    for mask in range(1, 16):
        need = [bool(mask >> i & 1) for i in range(4)]
        some = f.backward(t["dy"], t["x"], *w, saved, need=need)
        for name, n, a, b in zip(("dx", "dWg", "dW1", "dW2"), need, some, every):
            assert torch.equal(a, b) if n else a is None, f"{name} of {need}"
        # added to zeros: the same sums
        for z in zeros:
            z.zero_()
        some = f.backward(t["dy"], t["x"], *w, saved, need=need, grads=zeros, accumulate=True)
        for name, n, a, b in zip(("dWg", "dW1", "dW2"), need[1:], some[1:], every[1:]):
            assert torch.equal(a, b) if n else a is None, f"{name} of {need}, added"
    f.check()
    f.close()
