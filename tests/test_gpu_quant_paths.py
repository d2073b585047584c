"""The 8-bit products where their kernels split and share work: long k over few tiles (parts of a tile summed by the
last of its blocks), several row tiles, the change from one kernel to the other, calls one after another without
a wait. Tolerances are those of test_gpu_quant.py, by the same derivation."""
import numpy as np
import pytest

from test_gpu_quant import (U, ceil, check_experts, check_product, choose, env, f64, layer, matrix,  # noqa: F401
                            ref_experts, ref_rows, rows, spread_matrix, spread_rows)

pytestmark = pytest.mark.gpu


def product_ref(x, ws):
    q, s = ref_rows(f64(x))
    return spread_rows(q, ((s * 448).astype(np.float32) / np.float32(448)).astype(np.float64))


@pytest.mark.parametrize("M,N,K", [(1100, 200, 10248),   # wide: five tiles of 81 k-blocks over all pairs
                                   (1280, 1000, 12000),  # wide: twenty tiles split, some into three
                                   (1, 130, 20000), (3, 128, 28672), (20, 257, 9000), (50, 200, 16392),  # thin, few tiles
                                   (130, 300, 9608), (500, 140, 4104), (1024, 136, 264),  # thin, several row tiles
                                   (2100, 1300, 136)])   # wide, more tiles than pairs, one or two k-blocks
def test_split_products(env, M, N, K):
    pop, torch, dev = env
    wq, ws = matrix(env, 3, N, K)
    x = rows(env, 4, M, K)
    h = pop.PopQLinear(wq, ws, max_tokens=M, out_f32=True)
    y = h.forward(x)
    wd = spread_matrix(f64(wq), ws.double().cpu().numpy())
    check_product(y, product_ref(x, ws), wd, ceil(K, 128), "f32", f"{M}x{N}x{K}")
    for _ in range(3):
        assert torch.equal(h.forward(x), y)
    h.check()


@pytest.mark.parametrize("T,E,k,D,N", [(1100, 1, 1, 12000, 136),  # wide gate/up split over k
                                       (1200, 2, 2, 520, 10248),  # wide down split over k
                                       (400, 2, 1, 264, 136), (30, 2, 1, 9000, 200), (600, 40, 2, 136, 264)])
def test_split_experts(env, T, E, k, D, N):
    pop, torch, dev = env
    packs, dense = layer(env, 5, E, D, N)
    x = rows(env, 6, T, D) * 0.3
    e, w = choose(env, 7, T, E, k)
    m = pop.PopQMoE(*packs, top_k=k, max_tokens=T, out_f32=True)
    y = m.forward(x, e, w)
    check_experts(y, ref_experts(f64(x), e.cpu().numpy(), w.double().cpu().numpy(), *dense), "f32", (T, E, k, D, N))
    assert torch.equal(m.forward(x, e, w), y)
    m.check()


def test_calls_one_after_another(env):
    """Calls of many lengths, two handles in turn, nothing waited for in between: each result is that of a call alone."""
    pop, torch, dev = env
    N, K = 520, 2056
    hs = [pop.PopQLinear(*matrix(env, 10 + i, N, K), max_tokens=1300, out_f32=True) for i in range(2)]
    xs = [rows(env, 20 + i, m, K) for i, m in enumerate((1, 1300, 16, 70, 17, 600, 33, 1100, 2))]
    alone = []
    for h in hs:
        for x in xs:
            alone.append(h.forward(x))
            torch.cuda.synchronize()
    for _ in range(3):
        got = [h.forward(x) for h in hs for x in xs]
        assert all(torch.equal(a, b) for a, b in zip(got, alone))
        got = [h.forward(x) for x in xs for h in hs]
        assert all(torch.equal(a, alone[i]) for a, i in zip(got, [j * len(xs) + i for i in range(len(xs)) for j in range(2)]))
    for h in hs:
        h.check()


def test_layers_one_after_another(env):
    """Two layers that feed each other, decode steps and prompts mixed, against the same calls one by one."""
    pop, torch, dev = env
    E, D, N = 4, 256, 264
    layers = [pop.PopQMoE(*layer(env, 30 + i, E, D, N)[0], top_k=2, max_tokens=700) for i in range(2)]
    steps = [(t, rows(env, t, t, D), *choose(env, t + 1, t, E, 2)) for t in (1, 700, 3, 40, 333, 16, 2)]

    def chain(wait):
        out = []
        for _, x, e, w in steps:
            for m in layers:
                x = m.forward(x, e, w)
                if wait:
                    torch.cuda.synchronize()
            out.append(x)
        return out

    want = chain(True)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(chain(False), want))
    for m in layers:
        m.check()


def test_streams_in_turn(env):
    """One handle on two streams that wait for each other."""
    pop, torch, dev = env
    h = pop.PopQLinear(*matrix(env, 40, 300, 1032), max_tokens=200, out_f32=True)
    xs = [rows(env, 41 + i, m, 1032) for i, m in enumerate((5, 150, 30, 200))]
    want = [h.forward(x) for x in xs]
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for i, x in enumerate(xs * 3):
        s, other = (a, b) if i % 2 == 0 else (b, a)
        s.wait_stream(other)
        got.append(h.forward(x, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i % len(xs)]) for i, y in enumerate(got))


def test_routing_feeds_experts_in_a_graph(env):
    """The router's outputs as the experts' inputs, captured and replayed with other logits."""
    pop, torch, dev = env
    E, D, N, T = 8, 256, 136, 64
    m = pop.PopQMoE(*layer(env, 50, E, D, N)[0], top_k=2, max_tokens=T)
    r = pop.PopRouter(E, 2)
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    logits = [torch.randn((T, E), generator=g, device=dev) for _ in range(3)]
    logits[2][5] = float("-inf")  # a token without an expert
    x = rows(env, 51, T, D)
    want = [m.forward(x, *r.route(l)) for l in logits]
    assert bool((want[2][5] == 0).all())
    src, out = logits[0].clone(), torch.empty_like(want[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.forward(x, *r.route(src), y=out)
    for l, y in zip(logits, want):
        src.copy_(l)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, y)
    m.check()
