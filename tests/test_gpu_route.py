"""Routing on the GPU (include/pop_route.h) against its definition in 64 bits.

Chosen experts must be the definition's, ties included, wherever its choice values are apart in fp32:
without a bias the softmax order is that of the logits, which is exact. Sigmoid and biased values round,
so where two of them lie within 2^-20 of their size (each is a few fp32 operations, every one off by at most
2^-22), either order is right. Weights are a score over a sum of at most 256 scores: 2^-24 * 20 relative.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch

    import __graft_entry__
    __graft_entry__.build()
    import online_structured_ffn_gb300 as pop
    torch.cuda.set_device(0)
    return pop, torch, torch.device("cuda", 0)


def scores(l, kind):
    with np.errstate(all="ignore"):
        live = ~np.isnan(l) & (l != -np.inf)
        l = np.where(live, np.minimum(l, np.finfo(np.float32).max), -np.inf)
        if kind == "sigmoid":
            return np.where(live, 1 / (1 + np.exp(-l)), 0.0), live, l
        top = np.max(l, initial=-np.inf)
        e = np.where(live, np.exp(l - (top if live.any() else 0.0)), 0.0)
        return e / (e.sum() or 1.0), live, l


def ref_token(l, kind, bias, G, top_groups, group_sum):
    """(scores, choice values with -inf for what cannot be chosen, group values, group cut) of one token."""
    s, live, l = scores(l, kind)
    c = s + bias if bias is not None else (s if kind == "sigmoid" else l)
    c = np.where(live & ~np.isnan(c), c, -np.inf)
    per = len(l) // G
    v = np.full(G, -np.inf)
    for g in range(G):
        best = np.sort(c[g * per:(g + 1) * per])[::-1][:group_sum]
        best = best[best > -np.inf]
        if len(best):
            v[g] = best.sum()
    return s, c, v


def check(env, L, experts, weights, k, kind, bias, G, top_groups, group_sum, renorm, scale):
    ex, w = experts.cpu().numpy(), weights.double().cpu().numpy()
    E = L.shape[1]
    per = E // G
    rounds = kind == "sigmoid" or bias is not None
    band = 2.0 ** -20 if rounds else 0.0
    for t in range(L.shape[0]):
        s, c, v = ref_token(L[t], kind, bias, G, top_groups, group_sum)
        order = np.argsort(-v, kind="stable")
        keep = np.zeros(G, bool)
        keep[order[:top_groups]] = True
        got = ex[t][ex[t] >= 0]
        if G > 1 and top_groups < G and v[order[top_groups]] > -np.inf:
            a, b = v[order[top_groups - 1]], v[order[top_groups]]
            if rounds and a - b <= band * max(abs(a), abs(b), 1e-3) and a != b:
                continue  # two groups too near to tell apart in fp32
        c = np.where(np.repeat(keep, per), c, -np.inf)
        want = np.argsort(-c, kind="stable")[:k]
        want = want[c[want] > -np.inf]
        assert len(got) == len(want) and list(ex[t]) == list(got) + [-1] * (k - len(got)), (t, ex[t], want)
        if not np.array_equal(got, want):
            assert rounds, (t, got, want)
            assert len(set(got)) == len(got)
            near = band * np.maximum(np.abs(c[want]), 1e-3)
            assert np.all(np.abs(c[got] - c[want]) <= near), (t, got, want)
        chosen = s[got]
        if renorm:
            chosen = chosen / chosen.sum() if chosen.sum() > 0 else chosen * 0
        assert np.all(np.abs(w[t][:len(got)] - chosen * scale) <= 20 * 2.0 ** -24 * chosen * abs(scale) + 1e-37), (t, w[t], chosen)
        assert np.all(w[t][len(got):] == 0)


def logits(env, seed, T, E, dtype, masked=0.0, grid=None):
    _, torch, dev = env
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    l = torch.randn((T, E), generator=g, device=dev) * 2
    if grid:
        l = torch.round(l * grid) / grid  # many exact ties
    if masked:
        l = l.masked_fill(torch.rand((T, E), generator=g, device=dev) < masked, float("-inf"))
    return l.to(torch.bfloat16) if dtype == "bf16" else l


CASES = [  # T, E, k, kind, bias, groups, top_groups, group_sum, renorm, scale, masked, grid
    (1, 1, 1, "softmax", False, 1, 1, 1, True, 1.0, 0, None),
    (1, 8, 2, "softmax", False, 1, 1, 1, True, 1.0, 0, None),
    (33, 8, 2, "softmax", False, 1, 1, 1, False, 1.0, 0, 2),
    (257, 7, 7, "softmax", False, 1, 1, 1, True, 1.0, 0.3, None),
    (100, 33, 5, "softmax", True, 1, 1, 1, True, 2.0, 0.1, None),
    (65, 64, 6, "softmax", False, 8, 3, 1, False, 16.0, 0, 4),
    (129, 100, 16, "softmax", False, 4, 2, 1, True, 1.0, 0.8, None),
    (50, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5, 0, None),
    (50, 256, 8, "sigmoid", False, 8, 4, 1, True, 1.0, 0.9, 8),
    (31, 128, 1, "sigmoid", False, 1, 1, 1, False, 1.0, 0.97, None),
    (40, 12, 3, "sigmoid", True, 6, 2, 2, False, 1.0, 0.5, None),
    (20, 256, 16, "sigmoid", True, 256, 40, 1, True, 1.0, 0, None),
    (20, 240, 12, "softmax", True, 3, 2, 2, True, 1.0, 0.2, None),
    (1000, 16, 4, "softmax", False, 1, 1, 1, True, 1.0, 0, 1),
    (300, 5, 2, "sigmoid", False, 5, 3, 1, True, 1.0, 0.4, None),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}x{c[1]}k{c[2]}{c[3]}g{c[5]}")
def test_route(env, case, dtype):
    pop, torch, dev = env
    T, E, k, kind, biased, G, tg, gs, renorm, scale, masked, grid = case
    l = logits(env, T + E, T, E, dtype, masked, grid)
    bias = logits(env, 5, 1, E, "f32")[0] * 0.1 if biased else None
    r = pop.PopRouter(E, k, score=kind, n_groups=G, top_groups=tg, group_sum=gs, renorm=renorm, scale=scale)
    counts = torch.full((E,), -7, dtype=torch.int32, device=dev)
    experts, weights = r.route(l, bias=bias, counts=counts)
    b = None if bias is None else bias.double().cpu().numpy()
    check(env, l.double().cpu().numpy(), experts, weights, k, kind, b, G, tg, gs, renorm, scale)
    chosen = experts[experts >= 0].long()
    assert torch.equal(counts.long(), torch.bincount(chosen, minlength=E))
    again = r.route(l, bias=bias)
    assert torch.equal(again[0], experts) and torch.equal(again[1], weights)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_special_values(env, kind):
    pop, torch, dev = env
    inf, nan, low = float("inf"), float("nan"), float(np.finfo(np.float32).min)
    l = torch.tensor([[-inf] * 6, [nan] * 6, [low] * 6, [inf, 0, inf, 1, nan, -inf], [0.0, -0.0, 0.0, -0.0, 0.0, -0.0],
                      [-inf, nan, 3.0, -inf, -inf, low], [1e30, 1e30, -1e30, 0, 0, 0]], device=dev)
    r = pop.PopRouter(6, 3, score=kind, renorm=True)
    e, w = r.route(l)
    e, w = e.cpu().numpy(), w.cpu().numpy()
    assert np.isfinite(w).all()
    assert list(e[0]) == [-1] * 3 and list(e[1]) == [-1] * 3 and np.all(w[:2] == 0)
    assert list(e[2]) == [0, 1, 2]
    assert np.allclose(w[2], 1 / 3 if kind == "softmax" else 0)  # sigmoid of the lowest value is 0: no sum to divide by
    assert list(e[3]) == [0, 2, 3]
    assert list(e[4]) == [0, 1, 2] and np.allclose(w[4], 1 / 3)
    assert list(e[5]) == [2, 5, -1] and w[5][0] == 1 and np.all(w[5][1:] == 0)
    assert list(e[6][:2]) == [0, 1] and np.allclose(w[6][:2], 0.5 if kind == "softmax" else 0.4)


def test_bias_closes_and_opens_experts(env):
    pop, torch, dev = env
    l = torch.zeros((5, 4), device=dev)
    bias = torch.tensor([float("-inf"), 0.0, float("nan"), 1.0], device=dev)
    e, w = pop.PopRouter(4, 3, score="sigmoid", renorm=False).route(l, bias=bias)
    assert e.tolist() == [[3, 1, -1]] * 5 and w.tolist() == [[0.5, 0.5, 0.0]] * 5


@pytest.mark.parametrize("E,k", [(8, 2), (100, 6), (256, 8)])
def test_strided_streams_graph_and_empty(env, E, k):
    pop, torch, dev = env
    wide = logits(env, 9, 70, E + 5, "bf16")
    r = pop.PopRouter(E, k)
    want = r.route(wide[:, 3:3 + E].contiguous())
    got = r.route(wide[:, 3:3 + E])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = r.route(wide[:, 3:3 + E], stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    e, w = r.route(wide[:0, :E])
    assert e.shape == (0, k) and w.shape == (0, k)
    src = wide[:, 3:3 + E].contiguous()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = r.route(src)
    src.copy_(wide[:, :E])
    graph.replay()
    torch.cuda.synchronize()
    again = r.route(src)
    assert torch.equal(out[0], again[0]) and torch.equal(out[1], again[1])


def test_many_tokens(env):
    pop, torch, dev = env
    l = logits(env, 2, 70001, 64, "f32")
    e, w = pop.PopRouter(64, 4).route(l)
    v, i = torch.topk(l, 4, dim=1)
    assert torch.equal(torch.gather(l, 1, e.long()), v)
    p = torch.softmax(v.double(), dim=1)
    assert float((w.double() - p).abs().max()) <= 20 * 2.0 ** -24
