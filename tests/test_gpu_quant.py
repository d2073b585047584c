"""Quantised rows, products and experts (include/pop_quant.h) against their definitions in 64 bits.

Tolerances, from the arithmetic:
- quantised values and scales: the definition is a chain of single fp32 operations, so both are exact.
- products: with u = 2^-23 for an addition (a tensor core's adder may truncate), a block's sum of 128
  exact products is off by at most 128 u of the sum of magnitudes, and scaling and adding KB blocks by
  (KB + 3) u more: |error| <= (KB + 131) u * sum |x w|, plus half a unit of y's type
  (relative 2^-8 for bf16's 8 significant bits, 2^-24 for fp32).
- experts: gate and up are off by some 2^-18 of their size each, so SiLU(g) u by less than 2^-16; a rounding
  interval of e4m3 is at least 2^-4 of the value, so less than 2^-12 of the intermediate values round the
  other way, by at most 2^-3 of themselves: relative 2-norm of y's error <= 2^-3 * 2^-6 = 2^-9, and another
  2^-9 for bf16 outputs. A single row may take four times that.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -23


@pytest.fixture(scope="module")
def env():
    import torch

    import __graft_entry__
    __graft_entry__.build()
    import online_structured_ffn_gb300 as pop
    torch.cuda.set_device(0)
    return pop, torch, torch.device("cuda", 0)


def ceil(a, b):
    return -(-a // b)


def gen(env, seed):
    _, torch, dev = env
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return g


def rows(env, seed, M, K, dtype="bf16"):
    _, torch, dev = env
    g = gen(env, seed)
    x = torch.randn((M, K), generator=g, device=dev) * torch.exp(torch.randn((K,), generator=g, device=dev))
    return x.to(torch.bfloat16) if dtype == "bf16" else x


def e4m3(v):
    """Nearest e4m3 number, ties to even, of float64 values up to 448 in magnitude."""
    m, e = np.frexp(v)
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.rint(v / step) * step


def ref_rows(x):
    """float64 [M, K]: e4m3 values, scales."""
    M, K = x.shape
    q, s = np.zeros_like(x), np.zeros((M, ceil(K, 128)))
    for b in range(s.shape[1]):
        part = x[:, 128 * b:128 * b + 128]
        a = np.maximum(np.abs(part).max(axis=1), 2.0 ** -64)
        q[:, 128 * b:128 * b + 128] = e4m3(part * 448 / a[:, None])
        s[:, b] = a / 448
    return q, s


def ref_matrix(w):
    N, K = w.shape
    q, s = np.zeros_like(w), np.zeros((ceil(N, 128), ceil(K, 128)))
    for i in range(s.shape[0]):
        for b in range(s.shape[1]):
            part = w[128 * i:128 * i + 128, 128 * b:128 * b + 128]
            a = max(np.abs(part).max(), 2.0 ** -64)
            q[128 * i:128 * i + 128, 128 * b:128 * b + 128] = e4m3(part * 448 / a)
            s[i, b] = a / 448
    return q, s


def spread_rows(q, s):
    return q * np.repeat(s, 128, axis=1)[:, :q.shape[1]]


def spread_matrix(q, s):
    return q * np.repeat(np.repeat(s, 128, axis=0)[:q.shape[0]], 128, axis=1)[:, :q.shape[1]]


def f64(t):
    return t.float().double().cpu().numpy() if t.dtype != np.float64 else t


def matrix(env, seed, N, K):
    """(e4m3 [N, K], scales) on the device."""
    _, torch, dev = env
    w = rows(env, seed, N, K, "f32") * 0.05
    q, s = ref_matrix(w.double().cpu().numpy())
    return (torch.from_numpy(q).float().to(dev).to(torch.float8_e4m3fn),
            torch.from_numpy(s.astype(np.float32)).to(dev))


def check_product(y, xd, wd, KB, out, what):
    ref = xd @ wd.T
    mag = np.abs(xd) @ np.abs(wd).T
    tol = (KB + 131) * U * mag + (2.0 ** -8 if out == "bf16" else 2.0 ** -24) * np.abs(ref) + 1e-30
    err = np.abs(f64(y) - ref)
    bad = ~(err <= tol * (1 + 2.0 ** -8))
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside, worst {np.nanmax(err / tol)} of the bound"


# ------------------------------------------------------------------------------------ rows

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K", [(1, 8), (1, 128), (3, 136), (7, 1000), (64, 1024), (130, 4096), (1, 28672), (1000, 264)])
def test_rows(env, M, K, dtype):
    pop, torch, dev = env
    x = rows(env, M + K, M, K, dtype)
    q, s = pop.quantize_rows(x)
    rq, rs = ref_rows(x.double().cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), (rs * 448).astype(np.float32) / np.float32(448))
    differ = f64(q) != rq
    if dtype == "bf16":
        assert not differ.any()
    else:  # 0.875 x is rounded: one value in a million may lie on the other side of a tie
        assert differ.mean() <= 1e-5


def test_rows_special_values(env):
    pop, torch, dev = env
    inf, nan, big = float("inf"), float("nan"), 3.3e38
    x = torch.zeros((7, 256), dtype=torch.float32, device=dev)
    x[1, 5] = 1e-30
    x[2, 130] = -big
    x[3, 7] = inf
    x[4, 200] = nan
    x[5, :] = 448.0
    x[6, 0], x[6, 1], x[6, 2] = 448.0, 17.0, 19.0  # ties between 16 and 18, 18 and 20
    q, s = pop.quantize_rows(x)
    q, s = q.float().cpu().numpy(), s.cpu().numpy()
    assert np.all(q[0] == 0) and np.all(s[0] == np.float32(2.0 ** -64) / np.float32(448))
    assert q[1, 5] == 0  # far below the smallest scale's step
    assert q[2, 130] == -448 and s[2, 1] == np.float32(big) / np.float32(448) and np.all(q[2, :130] == 0)
    assert np.isinf(s[3, 0]) and np.isnan(q[3, 7]) and np.all(q[3, 128:] == 0)
    assert np.isnan(s[4, 1]) and np.isfinite(s[4, 0])
    assert np.all(q[5] == 448) and s[5, 0] == 1
    assert list(q[6, :3]) == [448, 16, 20]


def test_rows_strided_and_empty(env):
    pop, torch, dev = env
    x = rows(env, 3, 40, 520)
    q, s = pop.quantize_rows(x[3:20:2, 8:400])
    q2, s2 = pop.quantize_rows(x[3:20:2, 8:400].contiguous())
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)
    q, s = pop.quantize_rows(x[:0])
    assert q.shape == (0, 520) and s.shape == (0, 5)


# ------------------------------------------------------------------------------------ products

@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 8), (1, 128, 128), (1, 1000, 520), (2, 257, 1024), (5, 4096, 4096), (15, 384, 2048),
                                   (16, 640, 1032), (17, 129, 136), (33, 2000, 776), (63, 130, 128), (64, 512, 512), (65, 300, 1160),
                                   (127, 256, 384), (128, 256, 4096), (129, 511, 1000), (300, 1025, 2056), (700, 777, 640)])
def test_product(env, M, N, K, out):
    pop, torch, dev = env
    wq, ws = matrix(env, N + K, N, K)
    x = rows(env, M + 7, M, K)
    h = pop.PopQLinear(wq, ws, max_tokens=M, out_f32=out == "f32")
    y = h.forward(x)
    rq, rs = ref_rows(f64(x))
    rs = (rs * 448).astype(np.float32) / np.float32(448)
    wd = spread_matrix(f64(wq), ws.double().cpu().numpy())
    check_product(y, spread_rows(rq, rs.astype(np.float64)), wd, ceil(K, 128), out, f"{M}x{N}x{K}")
    q, s = pop.quantize_rows(x)
    y2 = h.forward_q(q, s)
    assert torch.equal(y, y2), "quantised on the way and before"
    h.check()
    h.close()


def test_product_of_a_bf16_matrix(env):
    pop, torch, dev = env
    W = (rows(env, 5, 300, 392, "f32") * 0.05).to(torch.bfloat16)
    x = rows(env, 6, 9, 392)
    q, s = ref_matrix(f64(W))
    wq = torch.from_numpy(q).float().to(dev).to(torch.float8_e4m3fn)
    ws = torch.from_numpy((s * 448).astype(np.float32) / np.float32(448)).to(dev)
    a, b = pop.PopQLinear(W, max_tokens=16), pop.PopQLinear(wq, ws, max_tokens=16)
    assert torch.equal(a.forward(x), b.forward(x))


@pytest.mark.parametrize("M,cap", [(37, 16), (300, 128), (129, 128), (5, 1), (200, 64)])
def test_product_in_chunks_is_the_same(env, M, cap):
    pop, torch, dev = env
    wq, ws = matrix(env, 11, 520, 776)
    x = rows(env, 12, M, 776)
    q, s = pop.quantize_rows(x)
    h = pop.PopQLinear(wq, ws, max_tokens=cap, out_f32=True)
    wd = spread_matrix(f64(wq), ws.double().cpu().numpy())
    check_product(h.forward(x), spread_rows(f64(q), s.double().cpu().numpy()), wd, 7, "f32", "chunks")
    h.check()


@pytest.mark.parametrize("M", [1, 40, 200])
def test_product_of_strided_rows(env, M):
    pop, torch, dev = env
    N, K = 333, 264
    wq, ws = matrix(env, 21, N, K)
    wide = rows(env, 22, M, K + 64)
    h = pop.PopQLinear(wq, ws, max_tokens=256, out_f32=False)
    x = wide[:, 16:16 + K]
    y = torch.full((M, N + 11), 7.0, dtype=torch.bfloat16, device=dev)
    h.forward(x, y[:, 3:3 + N])
    assert torch.equal(y[:, 3:3 + N], h.forward(x.contiguous()))
    assert bool((y[:, :3] == 7).all()) and bool((y[:, 3 + N:] == 7).all()), "written outside the output"
    q, s = pop.quantize_rows(x)
    qw, sw = torch.zeros((M, K + 24), dtype=torch.uint8, device=dev), torch.zeros((M, 9), device=dev)
    qw[:, 8:8 + K], sw[:, 2:5] = q.view(torch.uint8), s
    assert torch.equal(h.forward_q(qw.view(torch.float8_e4m3fn)[:, 8:8 + K], sw[:, 2:5]), h.forward_q(q, s))


@pytest.mark.parametrize("M", [4, 40, 200])
def test_rows_that_are_not_finite_stay_apart(env, M):
    pop, torch, dev = env
    wq, ws = matrix(env, 31, 260, 520)
    x = rows(env, 32, M, 520)
    h = pop.PopQLinear(wq, ws, max_tokens=M)
    good = h.forward(x)
    x[1, 300], x[3, 5] = float("nan"), float("inf")
    y = h.forward(x)
    assert bool(torch.isnan(y[1]).all()) and bool(torch.isnan(y[3]).all())
    rest = [i for i in range(M) if i not in (1, 3)]
    assert torch.equal(y[rest], good[rest])


@pytest.mark.parametrize("M", [1, 16, 100, 300])
def test_product_repeats_its_bits_on_any_stream_and_in_a_graph(env, M):
    pop, torch, dev = env
    wq, ws = matrix(env, 41, 2000, 4096)
    x = rows(env, 42, M, 4096)
    h = pop.PopQLinear(wq, ws, max_tokens=M, out_f32=True)
    y = h.forward(x)
    for _ in range(5):
        assert torch.equal(h.forward(x), y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    z = h.forward(x, stream=side)
    side.synchronize()
    assert torch.equal(z, y)
    out = torch.zeros_like(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h.forward(x, out)
    x2 = rows(env, 43, M, 4096)
    want = h.forward(x2)
    x.copy_(x2)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    h.check()


# ------------------------------------------------------------------------------------ experts

def ref_experts(x, experts, weights, wg, w1, w2):
    """float64: x [T, D]; matrices as lists of float64 [N, D], [N, D], [D, N]."""
    xd = spread_rows(*ref_rows(x))
    y = np.zeros_like(x)
    for e in range(len(wg)):
        for j in range(experts.shape[1]):
            t = np.nonzero(experts[:, j] == e)[0]
            if len(t):
                g, u = xd[t] @ wg[e].T, xd[t] @ w1[e].T
                h = spread_rows(*ref_rows(g / (1 + np.exp(-g)) * u))
                y[t] += (h @ w2[e].T) * weights[t, j][:, None]
    return y


def layer(env, seed, E, D, N):
    _, torch, dev = env
    packs, dense = [], []
    for i, (n, k) in enumerate(((N, D), (N, D), (D, N))):
        ms = [matrix(env, seed + 100 * e + i, n, k) for e in range(E)]
        packs.append(([m[0] for m in ms], [m[1] for m in ms]))
        dense.append([spread_matrix(f64(q), s.double().cpu().numpy()) for q, s in ms])
    return packs, dense


def check_experts(y, ref, out, what):
    y, tol = f64(y), 2.0 ** -9 * (2 if out == "bf16" else 1)
    assert np.isfinite(y).all(), what
    norm = np.linalg.norm(ref, axis=1)
    err = np.linalg.norm(y - ref, axis=1)
    assert np.linalg.norm(err) <= tol * np.linalg.norm(norm) + 1e-30, (what, np.linalg.norm(err) / np.linalg.norm(norm))
    assert np.all(err <= 4 * tol * norm + 1e-30), (what, np.max(err / np.maximum(norm, 1e-30)))


def choose(env, seed, T, E, k, dropped=0.0):
    _, torch, dev = env
    g = gen(env, seed)
    v, e = torch.topk(torch.randn((T, E), generator=g, device=dev), k, dim=1)
    e = e.to(torch.int32)
    if dropped:
        e[torch.rand((T, k), generator=g, device=dev) < dropped] = -1
    return e.contiguous(), torch.softmax(v, dim=1)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("T,E,k,D,N,dropped", [(1, 1, 1, 128, 128, 0), (1, 8, 2, 256, 520, 0), (3, 4, 1, 8, 8, 0), (16, 3, 3, 136, 264, 0),
                                               (33, 8, 2, 512, 1000, 0.2), (40, 64, 6, 384, 200, 0.1), (7, 256, 8, 128, 136, 0),
                                               (200, 2, 1, 256, 384, 0), (333, 3, 2, 520, 1160, 0.1), (150, 1, 1, 1024, 640, 0),
                                               (64, 16, 1, 264, 256, 0.9), (700, 5, 2, 256, 136, 0)])
def test_experts(env, T, E, k, D, N, dropped, out):
    pop, torch, dev = env
    packs, dense = layer(env, T + E, E, D, N)
    x = rows(env, T, T, D) * 0.3
    experts, weights = choose(env, T + 1, T, E, k, dropped)
    m = pop.PopQMoE(*packs, top_k=k, max_tokens=T, out_f32=out == "f32")
    y = m.forward(x, experts, weights)
    m.check()
    check_experts(y, ref_experts(f64(x), experts.cpu().numpy(), weights.double().cpu().numpy(), *dense), out, (T, E, k, D, N))
    assert torch.equal(y, m.forward(x, experts, weights)), "the same call gives the same bits"
    m.close()


@pytest.mark.parametrize("T", [2, 50, 400])
def test_experts_uneven(env, T):
    """All tokens to one expert; every slot empty; one expert in both slots; in chunks; strided; other stream."""
    pop, torch, dev = env
    E, D, N = 4, 256, 392
    packs, dense = layer(env, 9, E, D, N)
    x = rows(env, 10, T, D) * 0.3
    weights = torch.full((T, 2), 0.5, device=dev)
    m = pop.PopQMoE(*packs, top_k=2, max_tokens=T, out_f32=True)

    def ref(e):
        return ref_experts(f64(x), e.cpu().numpy(), weights.double().cpu().numpy(), *dense)

    for slots in ((2, -1), (3, 3), (0, 3)):
        e = torch.tensor([slots], dtype=torch.int32, device=dev).repeat(T, 1)
        check_experts(m.forward(x, e, weights), ref(e), "f32", slots)
    none = torch.full((T, 2), -1, dtype=torch.int32, device=dev)
    assert bool((m.forward(x, none, weights) == 0).all())
    e, _ = choose(env, 5, T, E, 2)
    want = m.forward(x, e, weights)
    check_experts(want, ref(e), "f32", "mixed")
    part = pop.PopQMoE(*packs, top_k=2, max_tokens=max(1, T // 3), out_f32=True)
    check_experts(part.forward(x, e, weights), ref(e), "f32", "chunks")
    wide = torch.zeros((T, D + 40), dtype=torch.bfloat16, device=dev)
    wide[:, 8:8 + D] = x
    y = torch.full((T, D + 8), 3.0, device=dev)
    m.forward(wide[:, 8:8 + D], e, weights, y[:, 4:4 + D])
    assert torch.equal(y[:, 4:4 + D], want) and bool((y[:, :4] == 3).all()) and bool((y[:, 4 + D:] == 3).all())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    z = m.forward(x, e, weights, stream=side)
    side.synchronize()
    assert torch.equal(z, want)
    m.check()
    part.check()


def test_experts_report_an_index_out_of_range(env):
    pop, torch, dev = env
    packs, dense = layer(env, 1, 2, 128, 128)
    m = pop.PopQMoE(*packs, top_k=2, max_tokens=8, out_f32=True)
    x = rows(env, 2, 8, 128)
    w = torch.full((8, 2), 0.5, device=dev)
    e = torch.tensor([[0, 1]] * 8, dtype=torch.int32, device=dev)
    e[3, 1] = 2
    y = m.forward(x, e, w)
    with pytest.raises(pop.PopError) as err:
        m.check()
    assert err.value.status == pop.POP_ERR_DEVICE
    e[3, 1] = -1
    assert torch.equal(y, m.forward(x, e, w))
    m.check()


def test_experts_of_bf16_matrices_and_a_token_that_is_not_finite(env):
    pop, torch, dev = env
    E, D, N, T = 2, 136, 264, 20
    ws = [[(rows(env, 70 + 10 * i + e, *shape, "f32") * 0.05).to(torch.bfloat16) for e in range(E)]
          for i, shape in enumerate(((N, D), (N, D), (D, N)))]
    dense = [[spread_matrix(*ref_matrix(f64(w))) for w in group] for group in ws]
    m = pop.PopQMoE(*ws, top_k=1, max_tokens=T)
    x = rows(env, 77, T, D) * 0.3
    e, w = choose(env, 78, T, E, 1)
    y = m.forward(x, e, w)
    check_experts(y, ref_experts(f64(x), e.cpu().numpy(), w.double().cpu().numpy(), *dense), "bf16", "bf16 matrices")
    x[4, 0] = float("nan")
    z = m.forward(x, e, w)
    rest = [t for t in range(T) if t != 4]
    assert bool(torch.isnan(z[4]).all()) and torch.equal(z[rest], y[rest])


def test_experts_zero_tokens_and_graph(env):
    pop, torch, dev = env
    packs, _ = layer(env, 3, 4, 256, 256)
    m = pop.PopQMoE(*packs, top_k=2, max_tokens=32)
    x = rows(env, 4, 32, 256)
    e, w = choose(env, 6, 32, 4, 2)
    assert m.forward(x[:0], e[:0], w[:0]).shape == (0, 256)
    m.forward(x, e, w)
    out = torch.zeros((32, 256), dtype=torch.bfloat16, device=dev)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.forward(x, e, w, out)
    e2, w2 = choose(env, 7, 32, 4, 2)
    want = m.forward(x, e2, w2)
    e.copy_(e2)
    w.copy_(w2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    m.check()
