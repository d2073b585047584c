"""Waits of the 8-bit products that run out: with a limit of 1 ns every wait that is not over within its first tries
does (which needs more than a few k-blocks: with one or two of them none is that long). The kernels record it and return, well within the seconds that each of their other waits may take, and the check
reports it once."""
import time

import pytest

from test_gpu_quant import check_product, choose, env, f64, layer, matrix, rows, spread_matrix, spread_rows  # noqa: F401

pytestmark = pytest.mark.gpu


def give_up(env, handle, call):
    """Runs `call` with the shortest limit until a wait runs out; the limit is the default again after it."""
    pop, torch, dev = env
    flush = torch.empty((64 << 20,), device=dev)
    for _ in range(20):
        flush.zero_()  # the matrix comes from memory, and the first waits last microseconds
        torch.cuda.synchronize()
        handle.set_wait_limit(1)
        t0 = time.monotonic()
        call()
        handle.set_wait_limit(2_000_000_000)
        try:
            handle.check()
        except pop.PopError as e:
            assert e.status == pop.POP_ERR_TIMEOUT
            assert time.monotonic() - t0 < 6  # a second or so for what is on its way, of each product
            handle.check()  # cleared
            return
    pytest.fail("no wait ran out")


@pytest.mark.parametrize("M,N,K", [(1, 4096, 16384), (16, 11008, 4096), (40, 8192, 8192), (300, 2048, 16384)])
def test_product_of_few_rows_gives_up(env, M, N, K):
    pop, torch, dev = env
    h = pop.PopQLinear((rows(env, 1, N, K, "f32") * 0.05).to(torch.bfloat16), max_tokens=M, out_f32=True)
    x = rows(env, 2, M, K)
    give_up(env, h, lambda: h.forward(x))
    h.close()


@pytest.mark.parametrize("T,E,k,D,N", [(1, 4, 2, 4096, 4096), (40, 8, 2, 2048, 2048), (2048, 2, 2, 2048, 4096)])
def test_experts_give_up(env, T, E, k, D, N):
    """Thin products, and wide gated ones (4096 slots over two experts)."""
    pop, torch, dev = env
    ws = [[(rows(env, 10 * i + e, n, m, "f32") * 0.05).to(torch.bfloat16) for e in range(E)]
          for i, (n, m) in enumerate(((N, D), (N, D), (D, N)))]
    m = pop.PopQMoE(*ws, top_k=k, max_tokens=T, out_f32=True)
    x = rows(env, 3, T, D) * 0.3
    e, w = choose(env, 4, T, E, k)
    give_up(env, m, lambda: m.forward(x, e, w))
    m.close()


def test_a_limit_of_nothing_is_refused(env):
    pop, torch, dev = env
    h = pop.PopQLinear(torch.zeros((8, 8), dtype=torch.bfloat16, device=dev), max_tokens=1)
    with pytest.raises(pop.PopError) as e:
        h.set_wait_limit(0)
    assert e.value.status == pop.POP_ERR_INVALID_ARG


@pytest.mark.parametrize("M,N,K", [(2560, 2048, 9728), (2560, 2304, 4096)])
def test_product_of_many_rows_gives_up(env, M, N, K):
    """The wide plain product. 80 tiles over 76 pairs: of 76 k-blocks, so that a pair's whole tile, where its eight
    epilogue warps do not meet, is followed by a run of the four that are split, where they do; and 90 whole ones of 32."""
    pop, torch, dev = env
    h = pop.PopQLinear((rows(env, 5, N, K, "f32") * 0.05).to(torch.bfloat16), max_tokens=M, out_f32=True)
    x = rows(env, 6, M, K)
    for _ in range(3):
        give_up(env, h, lambda: h.forward(x))
    h.close()
