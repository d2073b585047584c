"""The trainable gated MLP against its formulas in 64 bits, value by value.

The bounds count the roundings that include/pop_gated.h names. A value rounded to bf16 is off by at most 2^-8 of itself; a
sum of K products on the tensor cores in fp32 by at most K 2^-23 of the sum of the products' magnitudes (each of K additions
rounds or cuts off at 2^-23 of what has been summed); the activation and its slope, made of a few fp32 operations, an
exponential and a division that are good to a few 2^-23, by at most 2^-19 (1 + |g|) of their size; gate and up values that
were kept are cut off at 2^-15 of themselves at most, which moves SiLU(g) and its slope (whose own slopes are at most 1.1
and 0.5) by at most 2^-14 (1 + |g|).
"""
import pytest

pytestmark = pytest.mark.gpu

R16, ACC = 2.0 ** -8, 2.0 ** -23


@pytest.fixture(scope="module")
def env():
    import torch
    import online_structured_ffn_gb300 as pop
    return pop, torch, torch.device("cuda", 0)


def make(env, seed, M, D, N, ldx=None, scale=1.0):
    pop, torch, dev = env
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def r(rows, cols, s, ld=None):
        t = torch.randn((rows, ld or cols), generator=g, device=dev) * s
        return t.to(torch.bfloat16)[:, :cols]

    w = 1.5 / D ** 0.5
    return dict(x=r(M, D, scale, ldx), dy=r(M, D, 1.0, ldx), Wg=r(N, D, w), W1=r(N, D, w), W2=r(D, N, 1.0 / N ** 0.5))


def reference(t):
    """Values and how far a call's may be from them, before the rounding to their own type."""
    import torch
    x, dy, Wg, W1, W2 = (t[n].double() for n in ("x", "dy", "Wg", "W1", "W2"))
    M, D, N = x.shape[0], x.shape[1], Wg.shape[0]
    g, u, dh = x @ Wg.t(), x @ W1.t(), dy @ W2
    eg, eu, eh = (D * ACC * (a.abs() @ b.abs()) for a, b in ((x, Wg.t()), (x, W1.t()), (dy, W2)))
    p = torch.sigmoid(g)
    act, slope = g * p, p * (1 + g * (1 - p))
    wide = 1 + g.abs()
    h = act * u
    e_act = 1.1 * eg + 2.0 ** -19 * wide * act.abs()
    e_h = R16 * h.abs() + 1.01 * (e_act * u.abs() + (act.abs() + e_act) * eu)
    k_act = e_act + 2.0 ** -14 * wide * act.abs()
    k_slope = 0.5 * eg + (2.0 ** -14 + 2.0 ** -19) * wide
    k_u = eu + 2.0 ** -15 * u.abs()
    dg, du = dh * u * slope, dh * act
    e_dg = R16 * dg.abs() + 1.01 * (eh * (u * slope).abs() + (dh.abs() + eh) * (k_u * slope.abs() + (u.abs() + k_u) * k_slope))
    e_du = R16 * du.abs() + 1.01 * (eh * act.abs() + (dh.abs() + eh) * k_act)

    def product(a, ea, b, k):
        return a @ b, 1.01 * (ea @ b.abs()) + 1.01 * k * ACC * (a.abs() @ b.abs())

    none = torch.zeros_like(dy)
    dx = [product(dg, e_dg, Wg, 2 * N), product(du, e_du, W1, 2 * N)]
    dW2 = product(dy.t(), none.t(), h, M)
    return dict(y=product(h, e_h, W2.t(), N), dx=(dx[0][0] + dx[1][0], dx[0][1] + dx[1][1]),
                dWg=product(dg.t(), e_dg.t(), x, M), dW1=product(du.t(), e_du.t(), x, M),
                dW2=(dW2[0], dW2[1] + 1.01 * (dy.abs().t() @ e_h)))


def near(got, want, what, old=None):
    import torch
    value, off = want
    value = value if old is None else value + old.double()
    off = off + (R16 if got.dtype == torch.bfloat16 else ACC) * (value.abs() + off) + 1e-37
    worst = ((got.double() - value).abs() / off).max()
    assert torch.isfinite(got).all() and float(worst) <= 1, f"{what}: {float(worst):.2f} of its bound"


SIZES = [(1, 8, 8), (1, 256, 1024), (2, 64, 136), (3, 520, 72), (31, 128, 128), (33, 136, 264), (128, 64, 256), (129, 200, 392),
         (256, 256, 512), (257, 264, 520), (300, 1000, 2736), (640, 72, 1288), (1025, 136, 264)]


@pytest.mark.parametrize("out_f32,grad_f32", [(False, False), (True, True)])
@pytest.mark.parametrize("M,D,N", SIZES)
def test_forward_and_backward(env, M, D, N, out_f32, grad_f32):
    pop, torch, dev = env
    t = make(env, M + D + N, M, D, N)
    f = pop.PopGatedFFN(D, N, max_tokens=M, out_f32=out_f32, grad_f32=grad_f32)
    w = (t["Wg"], t["W1"], t["W2"])
    y, saved = f.forward(t["x"], *w, save=True)
    assert torch.equal(f.forward(t["x"], *w), y)
    grads = f.backward(t["dy"], t["x"], *w, saved)
    f.check()
    want = reference(t)
    assert y.dtype == (torch.float32 if out_f32 else torch.bfloat16)
    near(y, want["y"], "y")
    for name, got in zip(("dx", "dWg", "dW1", "dW2"), grads):
        near(got, want[name], name)
    for a, b in zip(grads, f.backward(t["dy"], t["x"], *w, saved)):
        assert torch.equal(a, b)
    f.close()


@pytest.mark.parametrize("grad_f32", [False, True])
def test_gradients_are_added_to_what_is_there(env, grad_f32):
    pop, torch, dev = env
    M, D, N = 70, 136, 328
    t = make(env, 1, M, D, N)
    w = (t["Wg"], t["W1"], t["W2"])
    f = pop.PopGatedFFN(D, N, max_tokens=M, grad_f32=grad_f32)
    y, saved = f.forward(t["x"], *w, save=True)
    into = [torch.randn_like(m, dtype=f.grad_dtype()) for m in w]
    old = [m.clone() for m in into]
    got = f.backward(t["dy"], t["x"], *w, saved, grads=into, accumulate=True)
    assert all(a.data_ptr() == b.data_ptr() for a, b in zip(got[1:], into))
    want = reference(t)
    for name, a, o in zip(("dWg", "dW1", "dW2"), into, old):
        near(a, want[name], name, o)
    f.backward(t["dy"], t["x"], *w, saved, grads=into)
    for name, a in zip(("dWg", "dW1", "dW2"), into):
        near(a, want[name], name)
    f.close()


def test_what_is_not_needed_is_left_out(env):
    pop, torch, dev = env
    M, D, N = 40, 128, 264
    t = make(env, 2, M, D, N)
    w = (t["Wg"], t["W1"], t["W2"])
    f = pop.PopGatedFFN(D, N, max_tokens=64)
    y, saved = f.forward(t["x"], *w, save=True)
    every = f.backward(t["dy"], t["x"], *w, saved)
    for mask in range(16):
        need = [bool(mask >> i & 1) for i in range(4)]
        some = f.backward(t["dy"], t["x"], *w, saved, need=need)
        for n, a, b in zip(need, some, every):
            assert torch.equal(a, b) if n else a is None
    f.close()


def test_rows_apart_and_neighbours_untouched(env):
    pop, torch, dev = env
    M, D, N = 37, 72, 200
    t = make(env, 3, M, D, N, ldx=96)
    w = (t["Wg"], t["W1"], t["W2"])
    f = pop.PopGatedFFN(D, N, max_tokens=M)
    assert t["x"].stride(0) == 96
    under = torch.full((M + 1, 88), 7.0, dtype=torch.bfloat16, device=dev)
    y, saved = f.forward(t["x"], *w, y=under[:M, 8:80], save=True)
    grads = f.backward(t["dy"], t["x"], *w, saved)
    want = reference(t)
    near(y, want["y"], "y")
    for name, got in zip(("dx", "dWg", "dW1", "dW2"), grads):
        near(got, want[name], name)
    assert (under[M] == 7).all() and (under[:, :8] == 7).all() and (under[:, 80:] == 7).all()
    f.close()


def test_no_rows(env):
    pop, torch, dev = env
    D, N = 64, 128
    t = make(env, 4, 1, D, N)
    w = (t["Wg"], t["W1"], t["W2"])
    f = pop.PopGatedFFN(D, N, max_tokens=8)
    x = t["x"][:0]
    y, saved = f.forward(x, *w, save=True)
    assert y.shape == (0, D) and saved.numel() == 0
    dx, *grads = f.backward(x, x, *w, saved)
    assert dx.shape == (0, D) and all((g == 0).all() for g in grads)
    into = [torch.ones_like(g) for g in grads]
    f.backward(x, x, *w, saved, grads=into, accumulate=True)
    assert all((g == 1).all() for g in into)
    f.close()


def test_rows_that_are_not_finite(env):
    """They give nothing finite themselves; the other rows have what they have without them, and so do the gradients of the
    matrices where such a row's dy is 0 ... which 0 * NaN is not: those are NaN."""
    pop, torch, dev = env
    M, D, N = 40, 128, 264
    t = make(env, 5, M, D, N)
    w = (t["Wg"], t["W1"], t["W2"])
    f = pop.PopGatedFFN(D, N, max_tokens=M)
    y0, s0 = f.forward(t["x"], *w, save=True)
    g0 = f.backward(t["dy"], t["x"], *w, s0)
    x = t["x"].clone()
    x[3, 5], x[17, 0] = float("nan"), float("inf")
    y, s = f.forward(x, *w, save=True)
    grads = f.backward(t["dy"], x, *w, s)
    rest = [i for i in range(M) if i not in (3, 17)]
    assert y[3].isnan().all() and y[17].isnan().any() and torch.equal(y[rest], y0[rest])
    assert grads[0][3].isnan().all() and torch.equal(grads[0][rest], g0[0][rest])
    assert all(g.isnan().any() for g in grads[1:])
    f.close()


def test_large_gates(env):
    """Gates far out on either side: SiLU is g or 0 there, its slope 1 or 0, and nothing overflows on the way."""
    pop, torch, dev = env
    M, D, N = 8, 64, 64
    t = make(env, 6, M, D, N, scale=300.0)
    w = (t["Wg"], t["W1"], t["W2"])
    f = pop.PopGatedFFN(D, N, max_tokens=M, out_f32=True, grad_f32=True)
    y, saved = f.forward(t["x"], *w, save=True)
    want = reference(t)
    near(y, want["y"], "y")
    for name, got in zip(("dx", "dWg", "dW1", "dW2"), f.backward(t["dy"], t["x"], *w, saved)):
        near(got, want[name], name)
    f.close()


def test_gradients_against_differences(env):
    """The loss sum(dy y) in 64 bits at x and the matrices moved either way along a direction: its change is the gradients'
    product with the direction, to what differences of that step leave (third derivatives, about 1e-6 here) and the
    gradients' own bounds."""
    pop, torch, dev = env
    M, D, N = 24, 64, 136
    t = make(env, 7, M, D, N)
    f = pop.PopGatedFFN(D, N, max_tokens=M, out_f32=True, grad_f32=True)
    w = (t["Wg"], t["W1"], t["W2"])
    y, saved = f.forward(t["x"], *w, save=True)
    grads = f.backward(t["dy"], t["x"], *w, saved)
    want = reference(t)
    at = [t[n].double() for n in ("x", "Wg", "W1", "W2")]

    def loss(x, Wg, W1, W2):
        g = x @ Wg.t()
        return float((t["dy"].double() * ((g * torch.sigmoid(g) * (x @ W1.t())) @ W2.t())).sum())

    for i, name in enumerate(("dx", "dWg", "dW1", "dW2")):
        v = torch.randn(at[i].shape, dtype=torch.float64, device=dev)
        step = 1e-4 / float(v.norm())
        sides = [loss(*(a + s * step * v if j == i else a for j, a in enumerate(at))) for s in (1, -1)]
        change = (sides[0] - sides[1]) / (2 * step)
        off = float((want[name][1] * v.abs()).sum()) + ACC * float((grads[i].double() * v).abs().sum())
        assert abs(change - float((grads[i].double() * v).sum())) <= off + 1e-5 * float(v.norm()) * float(grads[i].norm())
    f.close()


def test_replayed_graph_and_another_stream(env):
    """A captured step reads what its inputs hold when it is replayed, and two graphs of one handle share its workspace in
    turn."""
    pop, torch, dev = env
    M, D, N = 100, 128, 392
    f = pop.PopGatedFFN(D, N, max_tokens=128)

    def step(t):
        y, saved = f.forward(t["x"], t["Wg"], t["W1"], t["W2"], save=True)
        return (y, *f.backward(t["dy"], t["x"], t["Wg"], t["W1"], t["W2"], saved))

    ts = [make(env, 8 + i, m, D, N) for i, m in enumerate((M, 31))]
    for t in ts:
        step(t)
    graphs, outs = [], []
    for t in ts:
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(t))
        graphs.append(g)
    for seed in (20, 30):
        for i, t in enumerate(ts):
            for name, new in make(env, seed + i, t["x"].shape[0], D, N).items():
                t[name].copy_(new)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        got = [[o.clone() for o in out] for out in outs]
        side = torch.cuda.Stream()
        for i, t in enumerate(ts):
            with torch.cuda.stream(side):
                again = step(t)
            side.synchronize()
            for a, b in zip(got[i], again):
                assert torch.equal(a, b)
    f.check()
    f.close()


def test_a_wait_that_runs_out_is_reported(env):
    """With a limit of 1 ns every wait that is not over at once does; the kernels return and the handle is good again."""
    pop, torch, dev = env
    M, D, N = 512, 4096, 2048
    t = make(env, 9, M, D, N)
    w = (t["Wg"], t["W1"], t["W2"])
    f = pop.PopGatedFFN(D, N, max_tokens=M)
    y0, saved = f.forward(t["x"], *w, save=True)
    g0 = f.backward(t["dy"], t["x"], *w, saved)
    flush = torch.empty((64 << 20,), device=dev)
    for call in (lambda: f.forward(t["x"], *w), lambda: f.backward(t["dy"], t["x"], *w, saved)):
        for _ in range(20):
            flush.zero_()
            torch.cuda.synchronize()
            f.set_wait_limit(1)
            call()
            f.set_wait_limit(2_000_000_000)
            try:
                f.check()
            except pop.PopError as e:
                assert e.status == pop.POP_ERR_TIMEOUT
                break
        else:
            pytest.fail("no wait ran out")
        f.check()
        assert torch.equal(f.forward(t["x"], *w), y0)
        for a, b in zip(f.backward(t["dy"], t["x"], *w, saved), g0):
            assert torch.equal(a, b)
        f.check()
    f.close()


@pytest.mark.parametrize("M,D,N", [(1, 4096, 5504), (9, 8200, 264), (200, 2048, 9736), (777, 2048, 5496), (2560, 128, 264), (20, 72, 19464)])
def test_tiles_shared_by_several_ctas(env, M, D, N):
    """Few tiles of long sums, and last rounds that are cut: every product of a step."""
    pop, torch, dev = env
    t = make(env, 11, M, D, N)
    w = (t["Wg"], t["W1"], t["W2"])
    f = pop.PopGatedFFN(D, N, max_tokens=M)
    y, saved = f.forward(t["x"], *w, save=True)
    assert torch.equal(f.forward(t["x"], *w), y)
    grads = f.backward(t["dy"], t["x"], *w, saved)
    f.check()
    want = reference(t)
    near(y, want["y"], "y")
    for name, got in zip(("dx", "dWg", "dW1", "dW2"), grads):
        near(got, want[name], name)
    for _ in range(3):
        for a, b in zip(grads, f.backward(t["dy"], t["x"], *w, saved)):
            assert torch.equal(a, b)
    f.close()


@pytest.mark.parametrize("M,D,N", [(40, 2048, 2736), (600, 4096, 1000)])
def test_calls_after_a_wait_that_ran_out(env, M, D, N):
    """At limits at which all, some or none of a shared tile's CTAs give up, what they leave is cleared by the check."""
    pop, torch, dev = env
    ts = [make(env, 12 + i, M, D, N) for i in range(2)]
    f = pop.PopGatedFFN(D, N, max_tokens=M)

    def step(t):
        w = (t["Wg"], t["W1"], t["W2"])
        y, saved = f.forward(t["x"], *w, save=True)
        return (y, *f.backward(t["dy"], t["x"], *w, saved))

    want = [step(t) for t in ts]
    ran_out = 0
    for ns in (1, 600, 1000, 1500, 2000, 2500, 3500):
        f.set_wait_limit(ns)
        step(ts[1])
        f.set_wait_limit(2_000_000_000)
        try:
            f.check()
        except pop.PopError as e:
            assert e.status == pop.POP_ERR_TIMEOUT
            ran_out += 1
        for i in (0, 1, 0):
            for a, b in zip(step(ts[i]), want[i]):
                assert torch.equal(a, b), f"after a limit of {ns} ns"
        f.check()
    assert ran_out > 0
    f.close()


@pytest.mark.parametrize("M,D,N", [(300, 136, 2736), (300, 136, 5496), (520, 136, 2000), (520, 136, 2736), (520, 4096, 264), (777, 4096, 264),
                                   (1030, 136, 2736), (1030, 2048, 264), (1290, 136, 1032), (1290, 136, 2000), (1540, 136, 1032),
                                   (2048, 136, 1032), (2048, 2048, 264), (3100, 136, 264), (3100, 520, 264), (3100, 1000, 264),
                                   (3100, 136, 520), (3100, 2048, 264)])
def test_tiles_of_every_width(env, M, D, N):
    """On 152 SMs these take tiles of each width from 128 to 256 columns, in each product that has a choice."""
    pop, torch, dev = env
    t = make(env, 13, M, D, N)
    w = (t["Wg"], t["W1"], t["W2"])
    f = pop.PopGatedFFN(D, N, max_tokens=M, out_f32=M % 2 == 1)
    y, saved = f.forward(t["x"], *w, save=True)
    grads = f.backward(t["dy"], t["x"], *w, saved)
    f.check()
    want = reference(t)
    near(y, want["y"], "y")
    for name, got in zip(("dx", "dWg", "dW1", "dW2"), grads):
        near(got, want[name], name)
    f.close()


@pytest.mark.parametrize("M", [31, 32, 33, 63, 64, 65])
def test_few_rows_of_long_sums(env, M):
    """Boxes of each height, and rings of each length, gone round several times."""
    pop, torch, dev = env
    t = make(env, 14, M, 1288, 1544)
    w = (t["Wg"], t["W1"], t["W2"])
    f = pop.PopGatedFFN(1288, 1544, max_tokens=M)
    y, saved = f.forward(t["x"], *w, save=True)
    grads = f.backward(t["dy"], t["x"], *w, saved)
    f.check()
    want = reference(t)
    near(y, want["y"], "y")
    for name, got in zip(("dx", "dWg", "dW1", "dW2"), grads):
        near(got, want[name], name)
    f.close()


@pytest.mark.parametrize("M,D,N", [(150, 4040, 4200), (200, 5000, 2056), (300, 2056, 3208)])
def test_tiles_shared_by_three_pairs(env, M, D, N):
    """On 152 SMs these are, in the products forward and of x and the hidden values backward."""
    pop, torch, dev = env
    t = make(env, 15, M, D, N)
    w = (t["Wg"], t["W1"], t["W2"])
    f = pop.PopGatedFFN(D, N, max_tokens=M, out_f32=True)
    y, saved = f.forward(t["x"], *w, save=True)
    grads = f.backward(t["dy"], t["x"], *w, saved)
    f.check()
    want = reference(t)
    near(y, want["y"], "y")
    for name, got in zip(("dx", "dWg", "dW1", "dW2"), grads):
        near(got, want[name], name)
    f.close()


@pytest.mark.parametrize("M", [100, 129, 300])
def test_rows_apart_subsets_and_rows_that_are_not_finite_of_more_rows(env, M):
    pop, torch, dev = env
    D, N = 136, 392
    t = make(env, 16, M, D, N, ldx=152)
    w = (t["Wg"], t["W1"], t["W2"])
    f = pop.PopGatedFFN(D, N, max_tokens=M)
    wide = torch.full((M + 1, D + 16), 7.0, dtype=torch.bfloat16, device=dev)
    apart = torch.zeros((M, D + 24), dtype=torch.bfloat16, device=dev)
    apart[:, 8:8 + D] = t["dy"]
    dy = apart[:, 8:8 + D]
    y, saved = f.forward(t["x"], *w, y=wide[:M, 8:8 + D], save=True)
    every = f.backward(dy, t["x"], *w, saved)
    want = reference(t)
    near(y, want["y"], "y")
    for name, got in zip(("dx", "dWg", "dW1", "dW2"), every):
        near(got, want[name], name)
    assert (wide[M] == 7).all() and (wide[:, :8] == 7).all() and (wide[:, 8 + D:] == 7).all()
    for mask in (1, 2, 4, 8, 9, 14):
        need = [bool(mask >> i & 1) for i in range(4)]
        for n, a, b in zip(need, f.backward(dy, t["x"], *w, saved, need=need), every):
            assert torch.equal(a, b) if n else a is None
    into = [torch.randn_like(m) for m in w]
    old = [g.clone() for g in into]
    f.backward(dy, t["x"], *w, saved, grads=into, accumulate=True)
    for name, got, o in zip(("dWg", "dW1", "dW2"), into, old):
        near(got, want[name], name, old=o)
    x = t["x"].clone()
    x[3, 5], x[M - 1, 0] = float("nan"), float("inf")
    rest = [i for i in range(M) if i not in (3, M - 1)]
    y2, s2 = f.forward(x, *w, save=True)
    grads = f.backward(dy, x, *w, s2)
    assert y2[3].isnan().all() and torch.equal(y2[rest], y[rest])
    assert grads[0][3].isnan().all() and torch.equal(grads[0][rest], every[0][rest])
    assert all(g.isnan().any() for g in grads[1:])
    f.check()
    f.close()
