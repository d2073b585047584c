"""The wide 8-bit products (many rows to a matrix) and the kernel that groups many slots by expert, on every path that a call
can take: both output types, whole and split tiles, outputs and rows at odd places, rows that are in e4m3 already, values
that are not finite beside values that are, rows that end in a pair's first or second block, graphs and streams.
Tolerances are those of test_gpu_quant.py, by the same derivation."""
import numpy as np
import pytest

from test_gpu_quant import (U, ceil, check_experts, choose, env, f64, layer, matrix, ref_experts, ref_rows, rows,  # noqa: F401
                            spread_matrix, spread_rows)

pytestmark = pytest.mark.gpu


def plan(env, M, N, K):
    """(whole tiles, split tiles) of a wide product: 256 x 256 tiles over pairs of SMs, of which those of a last round
    that is long and nearly empty are split over k."""
    _, torch, dev = env
    pairs = torch.cuda.get_device_properties(dev).multi_processor_count // 2
    tiles, KB = ceil(M, 256) * ceil(ceil(N, 128), 2), ceil(K, 128)
    rest = tiles % pairs
    split = rest if KB * (pairs - rest) >= 72 * pairs else 0
    return tiles - split, split


def kernels(torch, call):
    """Names of the kernels that a call launches; none where the profiler has no access to the GPU."""
    from torch.profiler import ProfilerActivity, profile
    for _ in range(2):  # (a process's first profile holds nothing)
        with profile(activities=[ProfilerActivity.CPU, ProfilerActivity.CUDA]) as p:
            call()
            torch.cuda.synchronize()
    return " ".join(e.name for e in p.events() if "k_" in e.name)


def quantised(env, x):
    """float64 [M, K]: the definition's values of bf16 rows, on the device."""
    _, torch, dev = env
    q, s = ref_rows(f64(x))
    s = ((s * 448).astype(np.float32) / np.float32(448)).astype(np.float64)
    return torch.from_numpy(spread_rows(q, s)).to(dev)


def check_wide(env, y, xd, wd, K, out, what):
    _, torch, dev = env
    ref, mag = xd @ wd.T, xd.abs() @ wd.abs().T
    tol = (ceil(K, 128) + 131) * U * mag + (2.0 ** -8 if out == "bf16" else 2.0 ** -24) * ref.abs() + 1e-30
    over = (y.double() - ref).abs() / (tol * (1 + 2.0 ** -8))
    assert bool((over <= 1).all()), f"{what}: {int((~(over <= 1)).sum())} of {over.numel()} outside, worst {float(over.max())} of the bound"


def wide_matrix(env, seed, N, K):
    """(e4m3 [N, K], scales, float64 [N, K] on the device)."""
    _, torch, dev = env
    wq, ws = matrix(env, seed, N, K)
    return wq, ws, torch.from_numpy(spread_matrix(f64(wq), ws.double().cpu().numpy())).to(dev)


# (M, N, K), whole and split tiles. All have more than 1024 rows, which the thin kernel does not take.
CASES = [((1025, 1, 8), (5, 0)), ((1100, 300, 264), (10, 0)), ((1300, 129, 1000), (6, 0)), ((2049, 640, 520), (27, 0)),
         ((5000, 1300, 136), (114 + 6, 0)),  # more tiles than pairs, one or two k-blocks
         ((1280, 1000, 12600), (0, 20)),     # split, into four or five each
         ((1100, 200, 10248), (0, 5)), ((1281, 1700, 20600), (0, 42)),
         ((2560, 2048, 9728), (76, 4)),      # a whole tile each, then four split
         ((2817, 1700, 10360), (76, 8))]      # ... the last ones with one row


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("size,tiles", CASES, ids=["x".join(map(str, c[0])) for c in CASES])
def test_wide_product(env, size, tiles, out):
    pop, torch, dev = env
    M, N, K = size
    if torch.cuda.get_device_properties(dev).multi_processor_count == 152:
        assert plan(env, M, N, K) == tiles
    wq, ws, wd = wide_matrix(env, 3, N, K)
    x = rows(env, 4, M, K)
    h = pop.PopQLinear(wq, ws, max_tokens=M, out_f32=out == "f32")
    y = h.forward(x)
    check_wide(env, y, quantised(env, x), wd, K, out, f"{M}x{N}x{K}")
    q, s = pop.quantize_rows(x)
    for _ in range(2):
        assert torch.equal(h.forward(x), y) and torch.equal(h.forward_q(q, s), y)
    h.check()


def test_these_calls_are_wide(env):
    pop, torch, dev = env
    h = pop.PopQLinear(*matrix(env, 1, 300, 264), max_tokens=1100)
    x = rows(env, 2, 1100, 264)
    names = kernels(torch, lambda: h.forward(x))
    if not names:
        pytest.skip("the profiler reports no kernels here")
    assert "k_qgemm_wide" in names and "k_qgemm_thin" not in names
    assert "k_qgemm_wide" not in kernels(torch, lambda: h.forward(x[:900]))
    m = pop.PopQMoE(*layer(env, 5, 2, 136, 264)[0], top_k=2, max_tokens=1100)
    e, w = choose(env, 6, 1100, 2, 2)
    x = rows(env, 7, 1100, 136)
    names = kernels(torch, lambda: m.forward(x, e, w))
    assert "k_plan" in names and "k_qgemm_wide" in names and "k_qgemm_thin" not in names


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K,left,right", [(1100, 333, 264, 3, 8), (1400, 512, 520, 1, 0), (1400, 512, 520, 8, 8), (1030, 200, 392, 0, 1)])
def test_wide_product_of_strided_rows_and_outputs(env, M, N, K, left, right, out):
    pop, torch, dev = env
    wq, ws, wd = wide_matrix(env, 11, N, K)
    around = rows(env, 12, M, K + 64)
    x = around[:, 16:16 + K]
    h = pop.PopQLinear(wq, ws, max_tokens=M, out_f32=out == "f32")
    want = h.forward(x.contiguous())
    check_wide(env, want, quantised(env, x), wd, K, out, "contiguous")
    y = torch.full((M, left + N + right), 7.0, dtype=h.out_dtype(), device=dev)
    h.forward(x, y[:, left:left + N])
    assert torch.equal(y[:, left:left + N], want)
    assert bool((y[:, :left] == 7).all()) and bool((y[:, left + N:] == 7).all()), "written outside the output"
    q, s = pop.quantize_rows(x)
    qw, sw = torch.zeros((M, K + 24), dtype=torch.uint8, device=dev), torch.zeros((M, ceil(K, 128) + 3), device=dev)
    qw[:, 8:8 + K], sw[:, 2:2 + ceil(K, 128)] = q.view(torch.uint8), s
    z = h.forward_q(qw.view(torch.float8_e4m3fn)[:, 8:8 + K], sw[:, 2:2 + ceil(K, 128)])
    assert torch.equal(z, want)
    h.check()


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(1290, 260, 520), (1153, 2100, 1032), (1100, 200, 10248)])
def test_wide_rows_that_are_not_finite_stay_apart(env, M, N, K, out):
    """... also where a last block has no rows and multiplies what an earlier tile has left in its place."""
    pop, torch, dev = env
    wq, ws, _ = wide_matrix(env, 31, N, K)
    x = rows(env, 32, M, K)
    h = pop.PopQLinear(wq, ws, max_tokens=M, out_f32=out == "f32")
    good = h.forward(x)
    assert bool(torch.isfinite(good).all())
    odd = torch.tensor([0, 127, 128, 300, 700, 1023, M - 1], device=dev)
    x[odd, 300], x[300, 5], x[700, K - 1] = float("nan"), float("inf"), float("-inf")
    y = h.forward(x)
    assert bool(torch.isnan(y[odd]).all())
    rest = torch.ones((M,), dtype=torch.bool, device=dev)
    rest[odd] = False
    assert torch.equal(y[rest], good[rest])
    q, s = pop.quantize_rows(x)
    z = h.forward_q(q, s)
    assert bool(torch.isnan(z[odd]).all()) and torch.equal(z[rest], good[rest])
    h.check()


@pytest.mark.parametrize("M,N,K", [(1100, 300, 1032), (1280, 1000, 12600), (2560, 2048, 9728)])
def test_wide_product_on_any_stream_and_in_a_graph(env, M, N, K):
    pop, torch, dev = env
    wq, ws, _ = wide_matrix(env, 41, N, K)
    x = rows(env, 42, M, K)
    h = pop.PopQLinear(wq, ws, max_tokens=M)
    y = h.forward(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    z = h.forward(x, stream=side)
    side.synchronize()
    assert torch.equal(z, y)
    out = torch.zeros_like(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h.forward(x, out)
    x2 = rows(env, 43, M, K)
    want = h.forward(x2)
    x.copy_(x2)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    h.check()


def test_wide_chunks(env):
    """Chunks of more rows than the thin kernel takes, and a last one of fewer."""
    pop, torch, dev = env
    wq, ws, wd = wide_matrix(env, 51, 300, 520)
    x = rows(env, 52, 2700, 520)
    h = pop.PopQLinear(wq, ws, max_tokens=1200)
    check_wide(env, h.forward(x), quantised(env, x), wd, 520, "bf16", "chunks")
    h.check()


# ------------------------------------------------------------------------------------ experts

@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("T,E,k,D,N,dropped", [
    (700, 64, 4, 136, 136, 0.0), (400, 256, 8, 128, 136, 0.3), (1100, 33, 2, 264, 136, 0.1), (150, 200, 16, 136, 128, 0.05),  # plan, thin
    (2048, 3, 1, 136, 136, 0.0), (2049, 3, 1, 136, 136, 0.0),  # without and with a plan
    (1300, 2, 2, 264, 392, 0.1), (1100, 1, 1, 520, 136, 0.0), (2600, 4, 2, 136, 264, 0.2),  # wide
    (1025, 1, 4, 136, 264, 0.5)])  # wide, one expert in several of a token's slots
def test_many_slots(env, T, E, k, D, N, dropped, out):
    pop, torch, dev = env
    packs, dense = layer(env, 3 * T + E, E, D, N)
    x = rows(env, T, T, D) * 0.3
    if k <= E:
        experts, weights = choose(env, T + 1, T, E, k, dropped)
    else:
        experts, weights = torch.zeros((T, k), dtype=torch.int32, device=dev), torch.full((T, k), 1.0 / k, device=dev)
        experts[::3, 1] = -1
    m = pop.PopQMoE(*packs, top_k=k, max_tokens=T, out_f32=out == "f32")
    y = m.forward(x, experts, weights)
    m.check()
    check_experts(y, ref_experts(f64(x), experts.cpu().numpy(), weights.double().cpu().numpy(), *dense), out, (T, E, k, D, N))
    assert torch.equal(y, m.forward(x, experts, weights))
    # weights of empty slots are not looked at
    w2 = weights.masked_fill(experts < 0, float("nan")).contiguous()
    assert torch.equal(y, m.forward(x, experts, w2))
    m.close()


def test_many_slots_report_an_index_out_of_range(env):
    pop, torch, dev = env
    T, E, k = 700, 40, 4
    m = pop.PopQMoE(*layer(env, 61, E, 128, 128)[0], top_k=k, max_tokens=T, out_f32=True)
    x = rows(env, 62, T, 128)
    e, w = choose(env, 63, T, E, k)
    for at, bad in (((0, 0), E), ((699, 3), -2), ((350, 1), 2 ** 31 - 1), ((123, 2), -2 ** 31), ((31, 0), 255)):
        e2 = e.clone()
        e2[at] = bad
        y = m.forward(x, e2, w)
        with pytest.raises(pop.PopError) as err:
            m.check()
        assert err.value.status == pop.POP_ERR_DEVICE
        e2[at] = -1
        assert torch.equal(y, m.forward(x, e2, w))
        m.check()


@pytest.mark.parametrize("counts", [(2, 1298), (1300, 0), (1024, 276), (1, 1299), (257, 1043)])
def test_wide_experts_of_uneven_load(env, counts):
    """Two experts with few, none or most of the tokens; the same tokens in another order; a token that is not finite."""
    pop, torch, dev = env
    D, N, T = 136, 264, sum(counts)
    packs, dense = layer(env, 71, 2, D, N)
    m = pop.PopQMoE(*packs, top_k=1, max_tokens=2 * T, out_f32=True)  # (2 T: in which all are wide)
    x = (rows(env, 72, T, D) * 0.3).repeat(2, 1)
    e = torch.cat([torch.full((c,), i, dtype=torch.int32, device=dev) for i, c in enumerate(counts)] * 2)[:, None].contiguous()
    w = torch.ones((2 * T, 1), device=dev)
    y = m.forward(x, e, w)
    check_experts(y[:T], ref_experts(f64(x[:T]), e[:T].cpu().numpy(), np.ones((T, 1)), *dense), "f32", counts)
    assert torch.equal(y[:T], y[T:])
    g = torch.randperm(2 * T, generator=torch.Generator().manual_seed(1)).to(dev)
    assert torch.equal(m.forward(x[g].contiguous(), e[g].contiguous(), w), y[g])
    bad = [0, T - 1, T + 5]
    x[bad, 7] = float("nan")
    z = m.forward(x, e, w)
    rest = torch.ones((2 * T,), dtype=torch.bool, device=dev)
    rest[bad] = False
    assert bool(torch.isnan(z[bad]).all()) and torch.equal(z[rest], y[rest])
    m.check()


def test_many_slots_in_a_graph_strided_and_in_chunks(env):
    pop, torch, dev = env
    E, D, N, T = 2, 264, 136, 1500
    packs, dense = layer(env, 81, E, D, N)
    m = pop.PopQMoE(*packs, top_k=2, max_tokens=T)
    around = torch.zeros((T, D + 24), dtype=torch.bfloat16, device=dev)
    around[:, 8:8 + D] = rows(env, 82, T, D) * 0.3
    x = around[:, 8:8 + D]
    e, w = choose(env, 83, T, E, 2, 0.1)
    y = torch.full((T, D + 16), 3.0, dtype=torch.bfloat16, device=dev)
    m.forward(x, e, w, y[:, 8:8 + D])
    want = m.forward(x.contiguous(), e, w)
    assert torch.equal(y[:, 8:8 + D], want) and bool((y[:, :8] == 3).all()) and bool((y[:, 8 + D:] == 3).all())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.forward(x, e, w, y[:, 8:8 + D])
    e2, w2 = choose(env, 84, T, E, 2, 0.3)
    want = m.forward(x, e2, w2)
    e.copy_(e2)
    w.copy_(w2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y[:, 8:8 + D], want)
    m.check()
    part = pop.PopQMoE(*packs, top_k=2, max_tokens=1100, out_f32=True)  # 1100 wide, 400 thin
    ref = ref_experts(f64(x), e2.cpu().numpy(), w2.double().cpu().numpy(), *dense)
    check_experts(part.forward(x, e2, w2), ref, "f32", "chunks")
    part.check()


# ------------------------------------------------------------------------------------ rows

def test_rows_longer_than_any_matrix(env):
    """More than 32 blocks of a row a CTA, many CTAs a row."""
    pop, torch, dev = env
    x = rows(env, 91, 2, 1_000_008)
    q, s = pop.quantize_rows(x)
    rq, rs = ref_rows(f64(x))
    assert np.array_equal(f64(q), rq)
    assert np.array_equal(s.cpu().numpy(), (rs * 448).astype(np.float32) / np.float32(448))
