"""Rows, products and the gated MLP in 8-bit integers against their formulas in 64 bits.

Quantising is checked for equality with the header's steps in fp32. A product's integers are summed exactly in fp32 while no
partial sum passes 2^24; its value is then off by the roundings of s_x s_w, of the product with the sum, and of the output's
type. Beyond 2^24 each of K additions rounds or cuts off at 2^-23 of what has been summed.
"""
import pytest

pytestmark = pytest.mark.gpu

R16, R32, ACC = 2.0 ** -8, 2.0 ** -24, 2.0 ** -23


@pytest.fixture(scope="module")
def env():
    import torch
    import online_structured_ffn_gb300 as pop
    return pop, torch, torch.device("cuda", 0)


def gen(env, seed):
    g = env[1].Generator(device=env[2])
    g.manual_seed(seed)
    return g


def normal(env, seed, rows, cols, dtype="bf16", ld=None, scale=1.0):
    pop, torch, dev = env
    x = torch.randn((rows, ld or cols), generator=gen(env, seed), device=dev) * scale
    return (x.to(torch.bfloat16) if dtype == "bf16" else x)[:, :cols]


def integers(env, seed, rows, cols, lo=-127, hi=127):
    pop, torch, dev = env
    return torch.randint(lo, hi + 1, (rows, cols), generator=gen(env, seed), device=dev, dtype=torch.int32).to(torch.int8)


def steps(x):
    """The header's formula, in fp32."""
    import torch
    x = x.float()
    a = x.abs().amax(dim=1).clamp(min=2.0 ** -64)
    return torch.round(x * (127.0 / 128.0) / a[:, None] * 128.0).to(torch.int8), a / torch.full_like(a, 127.0)


def near(got, value, off, what):
    import torch
    off = off + (R16 if got.dtype == torch.bfloat16 else R32) * (value.abs() + off) + 1e-37
    worst = float(((got.double() - value).abs() / off).max())
    assert torch.isfinite(got).all() and worst <= 1, f"{what}: {worst:.2f} of its bound"


# ------------------------------------------------------------------ rows

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K", [(1, 8), (1, 1024), (3, 16), (7, 72), (65, 1032), (33, 4096), (9, 8192), (5, 8200), (2, 32768), (2, 65536),
                                 (1, 200008), (1001, 520)])
def test_rows(env, M, K, dtype):
    pop, torch, dev = env
    x = normal(env, M + K, M, K, dtype)
    q, s = pop.quantize_rows_i8(x)
    want_q, want_s = steps(x)
    assert torch.equal(q, want_q) and torch.equal(s, want_s)


def test_rows_apart_and_special(env):
    pop, torch, dev = env
    x = normal(env, 1, 9, 200, "f32", ld=256)
    assert torch.equal(pop.quantize_rows_i8(x)[0], steps(x)[0])
    # halves, which go to the even integer; zeros; magnitudes at either end
    t = torch.zeros((6, 64), device=dev)
    t[0, :8] = torch.tensor([127.0, 0.5, 1.5, -0.5, -1.5, 2.5, 126.5, -126.5], device=dev)
    t[2] = 2.0 ** -126
    t[3, :3] = torch.tensor([3.3e38, -3.3e38, 1e38], device=dev)
    t[4, 0] = -(2.0 ** -64)
    t[5] = 1e-30
    q, s = pop.quantize_rows_i8(t)
    assert q[0, :8].tolist() == [127, 0, 2, 0, -2, 2, 126, -126] and float(s[0]) == 1
    assert (q[1] == 0).all() and (q[2] == 0).all() and q[3, :3].tolist() == [127, -127, 38] and int(q[4, 0]) == -127
    assert torch.isfinite(s).all()
    for dtype in (torch.float32, torch.bfloat16):
        b = torch.ones((4, 1040), device=dev, dtype=dtype)
        b[1, 1039], b[2, 3] = float("nan"), float("-inf")
        q, s = pop.quantize_rows_i8(b)
        assert s.isnan().tolist() == [False, True, True, False] and (q[1:3] == 0).all() and (q[0] == 127).all() and (q[3] == 127).all()
    q, s = pop.quantize_rows_i8(x[:0])
    assert q.shape == (0, 200) and s.shape == (0,)


# ------------------------------------------------------------------ products

PRODUCTS = [(1, 1, 8), (1, 256, 1024), (1, 4096, 4104), (2, 100, 72), (5, 129, 136), (16, 1000, 2048), (17, 255, 520), (33, 513, 264),
            (64, 384, 1032), (65, 1001, 640), (127, 8, 4096), (128, 256, 256), (129, 264, 328), (257, 77, 8200), (300, 2000, 1000),
            (1025, 300, 136), (2500, 136, 72)]


@pytest.mark.parametrize("out_f32", [False, True])
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_product(env, M, N, K, out_f32):
    pop, torch, dev = env
    W = normal(env, N, N, K, scale=0.05)
    wq, ws = steps(W)
    h = pop.PopI8Linear(wq, ws, max_tokens=M, out_f32=out_f32)
    x = normal(env, M, M, K)
    xq, xs = steps(x)
    value = xs.double()[:, None] * ws.double() * (xq.double() @ wq.double().t())
    assert float((xq.double().abs() @ wq.double().abs().t()).max()) < 2 ** 24 or K > 2048
    off = 2 * R32 * value.abs() + (K * ACC if K > 2048 else 0) * 2.0 ** -6 * value.abs().max()
    y = h.forward(x)
    assert y.dtype == (torch.float32 if out_f32 else torch.bfloat16)
    near(y, value, off, "y")
    assert torch.equal(h.forward_q(xq, xs), y)
    h2 = pop.PopI8Linear(W, max_tokens=M, out_f32=out_f32)  # quantised here
    assert torch.equal(h2.forward(x), y)
    h.check()
    h.close()
    h2.close()


@pytest.mark.parametrize("M,N,K", [(1, 300, 1032), (8, 136, 1024), (40, 200, 1000), (130, 128, 1032), (600, 300, 1016)])
def test_sums_of_integers_are_exact(env, M, N, K):
    """Up to 1032 products of up to 127 * 128 stay below 2^24: every bit is right, with scales that are powers of two."""
    pop, torch, dev = env
    wq, xq = integers(env, 1, N, K, -128), integers(env, 2, M, K)
    wq[0] = -128
    xq[0] = 127
    h = pop.PopI8Linear(wq, torch.full((N,), 0.5, device=dev), max_tokens=M, out_f32=True)
    y = h.forward_q(xq, torch.full((M,), 4.0, device=dev))
    want = 2 * (xq.double() @ wq.double().t())
    assert torch.equal(y.double(), want) and float(y[0, 0]) == 2 * K * 127 * -128
    h.close()


def test_long_sums_of_one_sign(env):
    pop, torch, dev = env
    K = 65536
    wq, xq = torch.full((3, K), 127, dtype=torch.int8, device=dev), torch.full((2, K), 125, dtype=torch.int8, device=dev)
    one = torch.ones((3,), device=dev)
    h = pop.PopI8Linear(wq, one, max_tokens=2, out_f32=True)
    y = h.forward_q(xq, one[:2])
    value = torch.full((2, 3), 127.0 * 125 * K, dtype=torch.float64, device=dev)
    near(y, value, K * ACC * value, "y")
    h.close()


def test_rows_apart_odd_outputs_and_neighbours(env):
    """y at any alignment of its elements, its rows apart, and what lies around it untouched."""
    pop, torch, dev = env
    for M in (3, 40, 200):
        for N in (77, 136):
            for f32 in (False, True):
                W = normal(env, N, N, 264)
                h = pop.PopI8Linear(W, max_tokens=M, out_f32=f32)
                x = normal(env, M, M, 264, ld=280)
                want = h.forward(x.contiguous())
                for start, ld in ((1, N + 3), (8, N + 16), (0, N)):
                    under = torch.full((M + 1, ld + start), 7.0, dtype=h.out_dtype(), device=dev)
                    view = under[:M, start:start + N]
                    got = h.forward(x, y=view)
                    assert torch.equal(got, want) and got.data_ptr() == view.data_ptr()
                    assert (under[M] == 7).all() and (under[:, :start] == 7).all() and (under[:, start + N:] == 7).all()
                h.close()


def test_calls_longer_than_the_workspace(env):
    pop, torch, dev = env
    W = normal(env, 1, 200, 264)
    x = normal(env, 2, 300, 264)
    small, large = pop.PopI8Linear(W, max_tokens=70), pop.PopI8Linear(W, max_tokens=300)
    assert torch.equal(small.forward(x), large.forward(x))
    q, s = pop.quantize_rows_i8(x)
    assert torch.equal(small.forward_q(q, s), large.forward(x))
    assert small.forward(x[:0]).shape == (0, 200)
    small.close()
    large.close()


def test_rows_that_are_not_finite(env):
    pop, torch, dev = env
    for M in (4, 200):
        W = normal(env, 1, 136, 264)
        h = pop.PopI8Linear(W, max_tokens=M)
        f = pop.PopI8FFN(W, W, normal(env, 2, 264, 136), max_tokens=M)
        x = normal(env, 3, M, 264)
        y0, z0 = h.forward(x), f.forward(x)
        x[1, 7], x[2, 0] = float("inf"), float("nan")
        y, z = h.forward(x), f.forward(x)
        rest = [i for i in range(M) if i not in (1, 2)]
        assert y[1:3].isnan().all() and torch.equal(y[rest], y0[rest])
        assert z[1:3].isnan().all() and torch.equal(z[rest], z0[rest])
        h.close()
        f.close()


# ------------------------------------------------------------------ the gated MLP

@pytest.mark.parametrize("out_f32", [False, True])
@pytest.mark.parametrize("M,D,N", [(1, 8, 8), (1, 256, 1024), (2, 2048, 264), (7, 136, 72), (16, 264, 2000), (33, 128, 520), (64, 1024, 1032),
                                   (100, 72, 4104), (129, 264, 392), (300, 1000, 2736), (1030, 136, 264)])
def test_ffn(env, M, D, N, out_f32):
    """A hidden value whose quotient lies near a half may go to either side: the bound has the step of each that is as near as
    the errors of h and of its row's largest value make possible (SiLU's operations good to 2^-19 (1 + |g|))."""
    pop, torch, dev = env
    ws = [steps(normal(env, i, *shape, scale=1.2 / shape[1] ** 0.5)) for i, shape in enumerate(((N, D), (N, D), (D, N)))]
    f = pop.PopI8FFN(*ws, max_tokens=M, out_f32=out_f32)
    x = normal(env, 5, M, D)
    xq, xs = (t.double() for t in steps(x))
    (gq, gs), (uq, us), (dq, ds) = ((q.double(), s.double()) for q, s in ws)
    g, u = xs[:, None] * gs * (xq @ gq.t()), xs[:, None] * us * (xq @ uq.t())
    h = g * torch.sigmoid(g) * u
    rel = 2.0 ** -18 * (1 + g.abs().amax(dim=1, keepdim=True))
    s = h.abs().amax(dim=1, keepdim=True).clamp(min=2.0 ** -64) / 127
    t = h / s
    half = (t.abs() - t.abs().floor() - 0.5).abs() <= 2 * rel * t.abs() + 2.0 ** -20
    value = ds * s * (torch.round(t) @ dq.t())  # whole numbers are summed: a sum of 0 is 0
    off = ds * ((half * s) @ dq.abs().t()) + (rel + 4 * R32) * value.abs()
    off += (N * ACC if N > 1032 else 0) * 2.0 ** -6 * value.abs().max()
    y = f.forward(x)
    assert y.dtype == (torch.float32 if out_f32 else torch.bfloat16)
    near(y, value, off, "y")
    for _ in range(2):
        assert torch.equal(f.forward(x), y)
    f.check()
    f.close()


def test_ffn_of_other_forms(env):
    pop, torch, dev = env
    D, N = 136, 264
    ms = [normal(env, i, *shape, scale=0.1) for i, shape in enumerate(((N, D), (N, D), (D, N)))]
    x = normal(env, 5, 150, D, ld=160)
    whole = pop.PopI8FFN(*(steps(m) for m in ms), max_tokens=150)
    y = whole.forward(x)
    inside, chunks = pop.PopI8FFN(*ms, max_tokens=150), pop.PopI8FFN(*ms, max_tokens=64)
    assert torch.equal(inside.forward(x), y) and torch.equal(chunks.forward(x), y)
    under = torch.full((151, 160), 7.0, dtype=torch.bfloat16, device=dev)
    assert torch.equal(whole.forward(x, y=under[:150, 8:8 + D]), y)
    assert (under[150] == 7).all() and (under[:, :8] == 7).all() and (under[:, 8 + D:] == 7).all()
    assert whole.forward(x[:0]).shape == (0, D)
    for f in (whole, inside, chunks):
        f.close()


# ------------------------------------------------------------------ graphs, streams, waits

@pytest.mark.parametrize("M", [1, 20, 200])
def test_replayed_graphs_and_another_stream(env, M):
    pop, torch, dev = env
    D, N = 264, 520
    ms = [normal(env, i, *shape, scale=0.1) for i, shape in enumerate(((N, D), (N, D), (D, N)))]
    f, h = pop.PopI8FFN(*ms, max_tokens=M), pop.PopI8Linear(ms[0], max_tokens=M)
    xs = [normal(env, 5 + i, M, D) for i in range(2)]

    def call(x):
        return f.forward(x), h.forward(x), *pop.quantize_rows_i8(x)

    for x in xs:
        call(x)
    graphs, outs = [], []
    for x in xs:
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(x))
        graphs.append(g)
    for seed in (20, 30):
        for i, x in enumerate(xs):
            x.copy_(normal(env, seed + i, M, D))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        got = [[o.clone() for o in out] for out in outs]
        side = torch.cuda.Stream()
        for i, x in enumerate(xs):
            with torch.cuda.stream(side):
                again = call(x)
            side.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got[i], again))
            torch.cuda.synchronize()
            third = (f.forward(x, stream=side), h.forward(x, stream=side), *pop.quantize_rows_i8(x, stream=side))
            side.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got[i], third))
    f.close()
    h.close()


@pytest.mark.parametrize("M,D,N", [(1, 8192, 16384), (64, 8192, 8192), (400, 4096, 2048)])
def test_calls_after_a_wait_that_ran_out(env, M, D, N):
    pop, torch, dev = env
    ms = [normal(env, i, *shape, scale=0.02) for i, shape in enumerate(((N, D), (N, D), (D, N)))]
    f, h = pop.PopI8FFN(*ms, max_tokens=M), pop.PopI8Linear(ms[0], max_tokens=M)
    xs = [normal(env, 5 + i, M, D) for i in range(2)]
    flush = torch.empty((64 << 20,), device=dev)
    for o in (f, h):
        want = [o.forward(x) for x in xs]
        ran_out = 0
        for ns in 10 * (1,) + (600, 1000, 1500, 2000, 2500, 3500):
            flush.zero_()
            torch.cuda.synchronize()
            o.set_wait_limit(ns)
            o.forward(xs[1])
            o.set_wait_limit(2_000_000_000)
            try:
                o.check()
            except pop.PopError as e:
                assert e.status == pop.POP_ERR_TIMEOUT
                ran_out += 1
            for i in (0, 1, 0):
                assert torch.equal(o.forward(xs[i]), want[i]), f"after a limit of {ns} ns"
            o.check()
        assert ran_out > 0
        o.close()


@pytest.mark.parametrize("M,D,N", [(1, 1000, 2736), (8, 1024, 2048), (3, 4096, 11008)])
def test_rows_quantised_on_the_way_after_short_limits(env, M, D, N):
    """The same where the rows are converted inside the products and the hidden rows' largest values come from the tiles. (Waits
    this short mostly end within their first tries: none need run out.)"""
    pop, torch, dev = env
    ms = [normal(env, i, *shape, scale=0.02) for i, shape in enumerate(((N, D), (N, D), (D, N)))]
    f, h = pop.PopI8FFN(*ms, max_tokens=M), pop.PopI8Linear(ms[0], max_tokens=M)
    xs = [normal(env, 5 + i, M, D) for i in range(2)]
    q, s = pop.quantize_rows_i8(xs[0])
    flush = torch.empty((64 << 20,), device=dev)
    for o, calls in ((f, (f.forward,)), (h, (h.forward, lambda x: h.forward_q(*pop.quantize_rows_i8(x))))):
        for call in calls:
            want = [call(x) for x in xs]
            for ns in (1, 1, 500, 1000, 2000):
                flush.zero_()
                torch.cuda.synchronize()
                o.set_wait_limit(ns)
                call(xs[1])
                o.set_wait_limit(2_000_000_000)
                try:
                    o.check()
                except pop.PopError as e:
                    assert e.status == pop.POP_ERR_TIMEOUT
                for i in (0, 1, 0):
                    assert torch.equal(call(xs[i]), want[i]), f"after a limit of {ns} ns"
                o.check()
        o.close()
    assert torch.equal(q, steps(xs[0])[0])


@pytest.mark.parametrize("M", [1, 20, 64, 100])
@pytest.mark.parametrize("N", [264, 2000, 2400, 3080, 4200, 4800, 9600, 9800, 20000])
def test_tiles_shared_by_one_to_eight(env, M, N):
    """Short sums and longer ones: on 152 SMs clusters of every number of CTAs, one and two on an SM."""
    pop, torch, dev = env
    for K in (200, 2056):
        W, x = integers(env, N, N, K, -9, 9), integers(env, N + 1, M, K, -9, 9)
        sx, sw = torch.rand((M,), device=dev) + 0.5, torch.rand((N,), device=dev) + 0.5
        h = pop.PopI8Linear(W, sw, max_tokens=M, out_f32=True)
        y = h.forward_q(x, sx)
        h.check()
        # the sums are whole numbers below 2^24, and exact: what is left is two products' roundings
        value = (x.double() @ W.double().t()) * sx.double()[:, None] * sw.double()
        assert bool(((y.double() - value).abs() <= value.abs() * (2 * 2.0 ** -24) * (1 + 2.0 ** -20)).all())
        h.close()
