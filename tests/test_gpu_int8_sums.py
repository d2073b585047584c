"""Sums of many integers, bit for bit.

Integers that are multiples of 8 from 8 to 120 have products that are multiples of 64. Up to 65536 of them sum to less than 2^30,
so every partial sum, in whatever order, is a multiple of 64 below 2^30: 24 bits, exact in fp32, although the sums are far
past 2^24. Integers from 1 to 15 sum to less than 2^24 as they are. All are of one sign, and differ from row to row and channel to
channel: a product that is left out, taken twice or taken from another row shows, as does a sum rounded to fewer bits.
"""
import pytest

from test_gpu_int8 import env, integers  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("step,top", [(8, 15), (1, 15)])
@pytest.mark.parametrize("M", [1, 2, 16, 17, 100, 130, 300])
@pytest.mark.parametrize("N,K", [(3, 65536), (300, 65536), (1300, 28672), (264, 65528)])
def test_long_sums_of_one_sign_are_exact(env, M, N, K, step, top):  # noqa: F811
    pop, torch, dev = env
    assert K * (step * top) ** 2 < 2 ** 24 * step * step
    W, x = (step * integers(env, s, rows, K, 1, top) for s, rows in ((50, N), (51, M)))
    h = pop.PopI8Linear(W, torch.full((N,), 0.5, device=dev), max_tokens=M, out_f32=True)
    y = h.forward_q(x, torch.full((M,), 4.0, device=dev))
    h.check()
    want = 2 * (x.double() @ W.double().t())
    assert float(want.max()) > 2 ** 26 or step == 1
    assert torch.equal(y.double(), want)
    h.close()
