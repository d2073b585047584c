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


def good_again(env, handle, call, x, limits):
    """Calls under limits at which all, some or none of a tile's sharers give up, each followed by the check and by good calls.
    Two inputs in turn: the parts that an earlier call left would not show with one."""
    pop, torch, dev = env
    other = (x.roll(1, 1) * 0.5).contiguous()
    want, want_other = call(x), call(other)
    ran_out = 0
    for ns in limits:
        for _ in range(2):
            handle.set_wait_limit(ns)
            call(other)
            handle.set_wait_limit(2_000_000_000)
            try:
                handle.check()
            except pop.PopError as e:
                assert e.status == pop.POP_ERR_TIMEOUT
                ran_out += 1
            for a, b in ((x, want), (other, want_other), (x, want)):
                assert torch.equal(call(a), b), f"after a limit of {ns} ns"
            handle.check()
    assert ran_out > 0


@pytest.mark.parametrize("M,N,K", [(1, 11008, 4096), (16, 11008, 4096), (40, 2000, 8192), (300, 520, 8192),  # thin, tiles shared
                                   (2560, 2048, 9728), (1100, 200, 10248)])  # wide: four of 80 tiles split, all five
def test_products_after_a_wait_that_ran_out(env, M, N, K):
    pop, torch, dev = env
    h = pop.PopQLinear((rows(env, 7, N, K, "f32") * 0.05).to(torch.bfloat16), max_tokens=M, out_f32=True)
    good_again(env, h, h.forward, rows(env, 8, M, K), (1, 600, 1000, 1300, 1600, 2000, 2500, 3000, 3500))
    h.close()


@pytest.mark.parametrize("T,E,k,D,N,limits", [(40, 8, 2, 2048, 1000, (1, 600, 1000, 1500, 2000, 2500, 3500)),
                                              (2600, 1, 1, 10248, 1032, (1, 3000))])  # wide, its gated tiles whole and split
def test_experts_after_a_wait_that_ran_out(env, T, E, k, D, N, limits):
    pop, torch, dev = env
    ws = [[(rows(env, 20 * i + e, n, m, "f32") * 0.05).to(torch.bfloat16) for e in range(E)]
          for i, (n, m) in enumerate(((N, D), (N, D), (D, N)))]
    m = pop.PopQMoE(*ws, top_k=k, max_tokens=T, out_f32=True)
    e, w = choose(env, 10, T, E, k)
    good_again(env, m, lambda x: m.forward(x, e, w), rows(env, 9, T, D) * 0.3, limits)
    m.close()
