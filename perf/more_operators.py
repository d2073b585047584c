"""The cases on which the trainable gated MLP and the 8-bit integer operators are measured.

Five operators: the gated MLP on user-held weights (``gated``: forward), the same with what its backward
pass gives (``train``), quantising rows to 8-bit integers with a scale per token (``rows8``), the matrix
product in 8-bit integers with a scale per token and per channel (``linear8``) and the gated MLP made of
such products (``ffn8``). ``run`` computes each in plain torch operations, or, with ``own`` set, through
the framework's entry points.
"""
import math

import torch

own = False

Q_MAX = 127.0
AMAX_MIN = 2.0 ** -64


# ---------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one token through the 7B layer with weights that are being trained (a sample drawn between two steps)
        dict(name="gated_token", op="gated", M=1, D=4096, N=11008),
        # a 2048-token prompt through the same layer, nothing kept for a backward pass
        dict(name="gated_prompt", op="gated", M=2048, D=4096, N=11008),
        # a training step of the tiny configuration, where launches are all
        dict(name="train_tiny", op="train", M=64, D=256, N=1024),
        # a ragged batch through a middling layer
        dict(name="train_ragged", op="train", M=777, D=2048, N=5496),
        # a training step of the 7B layer on 4096 tokens
        dict(name="train_large", op="train", M=4096, D=4096, N=11008),
        # the activations of a 4096-token prefill chunk
        dict(name="rows8_prefill", op="rows8", M=4096, K=4096, dtype="bf16"),
        # a ragged number of rows of the 7B layer's intermediate width, in float32
        dict(name="rows8_ragged", op="rows8", M=1001, K=11008, dtype="f32"),
        # one token through one projection of the 7B layer
        dict(name="linear8_token", op="linear8", M=1, N=11008, K=4096, dtype="bf16", out="bf16"),
        # a batch of 16 through the 70B layer's down projection
        dict(name="linear8_batch", op="linear8", M=16, N=8192, K=28672, dtype="bf16", out="f32"),
        # a ragged prompt through the 70B layer's up projection, its rows quantised before
        dict(name="linear8_prompt", op="linear8", M=4001, N=28672, K=8192, dtype="int8", out="bf16"),
        # a decode step of 32 sequences through the 7B layer
        dict(name="ffn8_decode", op="ffn8", M=32, D=4096, N=11008),
        # a ragged prompt through it
        dict(name="ffn8_prompt", op="ffn8", M=1000, D=4096, N=11008),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gated", "train", "rows8", "linear8", "ffn8"])
    if op == "rows8":
        M = _log_uniform(rng, 1, 8192)
        return dict(op=op, M=M, K=8 * _log_uniform(rng, 8, max(8, min(28672, (4096 * 4096) // M) // 8)),
                    dtype=rng.choice(["bf16", "f32"]))
    if op == "linear8":
        M = _log_uniform(rng, 1, 4001)
        K = 8 * _log_uniform(rng, 32, 28672 // 8)
        N = _log_uniform(rng, 256, min(28672, 8192 * 28672 // K))
        return dict(op=op, M=M, N=N, K=K, dtype=rng.choice(["bf16", "int8"]), out=rng.choice(["bf16", "f32"]))
    M = _log_uniform(rng, 1, 4096)
    D = 8 * _log_uniform(rng, 32, 4096 // 8)
    return dict(op=op, M=M, D=D, N=8 * _log_uniform(rng, 64, 11008 // 8))


# --------------------------------------------------------------------------------------- inputs

def _dev():
    return torch.device("cuda", torch.cuda.current_device())


def _normal(g, rows, width, scale=1.0):
    return torch.randn((rows, width), generator=g, device=g.device) * scale


def _activations(g, rows, width):
    """N(0, 1) times a factor of each column's own: a few columns stand out, as in trained layers."""
    c = torch.exp(0.5 * torch.randn((width,), generator=g, device=g.device))
    return torch.randn((rows, width), generator=g, device=g.device) * c


def _weight8(g, n, k):
    """A matrix [n, k] of N(0, 0.02^2) in 8-bit integers and a float32 scale per row."""
    return _quantize(_normal(g, n, k, 0.02))


def prepare(case, seed):
    dev = _dev()
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = dict(case)
    M = case["M"]
    if case["op"] == "rows8":
        x = _activations(g, M, case["K"])
        s["x"] = x.to(torch.bfloat16) if case["dtype"] == "bf16" else x
    elif case["op"] == "linear8":
        s["wq"], s["ws"] = _weight8(g, case["N"], case["K"])
        s["x"] = _activations(g, M, case["K"]).to(torch.bfloat16)
        if case["dtype"] == "int8":
            s["xq"], s["xs"] = _quantize(s["x"].float())
        if own:
            import online_structured_ffn_gb300 as pop
            s["linear"] = pop.PopI8Linear(s["wq"], s["ws"], max_tokens=M, out_f32=case["out"] == "f32")
    else:
        D, N = case["D"], case["N"]
        s["x"] = _activations(g, M, D).to(torch.bfloat16)
        if case["op"] == "ffn8":
            s["wg"], s["w1"], s["w2"] = _weight8(g, N, D), _weight8(g, N, D), _weight8(g, D, N)
            if own:
                import online_structured_ffn_gb300 as pop
                s["ffn"] = pop.PopI8FFN(s["wg"], s["w1"], s["w2"], max_tokens=M)
        else:
            s["wg"], s["w1"], s["w2"] = (_normal(g, *shape, 0.02).to(torch.bfloat16)
                                         for shape in ((N, D), (N, D), (D, N)))
            if case["op"] == "train":
                s["dy"] = _normal(g, M, D, 1e-3).to(torch.bfloat16)
            if own:
                import online_structured_ffn_gb300 as pop
                s["ffn"] = pop.PopGatedFFN(D, N, max_tokens=M)
    return s


# ------------------------------------------------------------------------------ the plain forms

def _quantize(x):
    """x float32 [M, K]: (int8 [M, K], scales [M]). A row's value is rint(128 * ((127/128 * x) / amax)): for bf16
    inputs 127/128 * x is exact, so the one rounded division leaves ties where they are."""
    a = x.abs().amax(dim=1).clamp(min=AMAX_MIN)
    q = torch.round(x * (127.0 / 128.0) / a[:, None] * 128.0)
    return q.to(torch.int8), a / torch.full_like(a, Q_MAX)


def _product8(xq, xs, wq, ws):
    return xq.float() @ wq.float().t() * xs[:, None] * ws


def _gate(g):
    return 1.0 / (1.0 + torch.exp(-g))


def _forward(s):
    x, wg, w1, w2 = (s[n].float() for n in ("x", "wg", "w1", "w2"))
    g, u = x @ wg.t(), x @ w1.t()
    h = g * _gate(g) * u
    return x, wg, w1, w2, g, u, h, h @ w2.t()


def _train_plain(s):
    x, wg, w1, w2, g, u, h, y = _forward(s)
    dy = s["dy"].float()
    dh = dy @ w2
    p = _gate(g)
    dg = dh * u * p * (1.0 + g * (1.0 - p))
    du = dh * g * p
    return [t.to(torch.bfloat16) for t in (y, dg @ wg + du @ w1, dg.t() @ x, du.t() @ x, dy.t() @ h)]


def _ffn8_plain(s):
    xq, xs = _quantize(s["x"].float())
    g, u = _product8(xq, xs, *s["wg"]), _product8(xq, xs, *s["w1"])
    return _product8(*_quantize(g * _gate(g) * u), *s["w2"]).to(torch.bfloat16)


def run(state):
    s = state
    if own:
        import online_structured_ffn_gb300 as pop
        if s["op"] == "rows8":
            return pop.quantize_rows_i8(s["x"])
        if s["op"] == "linear8":
            return s["linear"].forward_q(s["xq"], s["xs"]) if s["dtype"] == "int8" else s["linear"].forward(s["x"])
        if s["op"] == "ffn8":
            return s["ffn"].forward(s["x"])
        if s["op"] == "gated":
            return s["ffn"].forward(s["x"], s["wg"], s["w1"], s["w2"])
        y, saved = s["ffn"].forward(s["x"], s["wg"], s["w1"], s["w2"], save=True)
        return [y, *s["ffn"].backward(s["dy"], s["x"], s["wg"], s["w1"], s["w2"], saved)]
    if s["op"] == "rows8":
        return _quantize(s["x"].float())
    if s["op"] == "linear8":
        xq, xs = (s["xq"], s["xs"]) if s["dtype"] == "int8" else _quantize(s["x"].float())
        return _product8(xq, xs, s["wq"], s["ws"]).to(torch.bfloat16 if s["out"] == "bf16" else torch.float32)
    if s["op"] == "ffn8":
        return _ffn8_plain(s)
    return _forward(s)[-1].to(torch.bfloat16) if s["op"] == "gated" else _train_plain(s)


# ----------------------------------------------------------------------------------------- work

def work(case):
    M = case["M"]
    if case["op"] == "rows8":
        K = case["K"]
        return {"bytes": M * K * ((2 if case["dtype"] == "bf16" else 4) + 1) + 4 * M, "flops": 4 * M * K}
    if case["op"] == "linear8":
        N, K = case["N"], case["K"]
        x = M * K * 2 if case["dtype"] == "bf16" else M * (K + 4)
        return {"bytes": N * (K + 4) + x + M * N * (2 if case["out"] == "bf16" else 4), "flops": 2 * M * N * K}
    D, N = case["D"], case["N"]
    if case["op"] == "ffn8":
        return {"bytes": 3 * N * D + 8 * N + 4 * D + 4 * M * D, "flops": 6 * M * N * D}
    if case["op"] == "gated":
        return {"bytes": 6 * N * D + 4 * M * D, "flops": 6 * M * N * D}
    return {"bytes": 12 * N * D + 8 * M * D, "flops": 18 * M * N * D}


# ------------------------------------------------------------------- the definitions in 64 bits

def _exact_rows(x):
    most = x.abs().max(dim=1).values.clamp(min=AMAX_MIN)
    return torch.round(x * 127 / most[:, None]), most / 127


def _exact_product(q, scale, w):
    """Rows q of whole numbers with their scales, times a matrix of such rows; some rows of the matrix at a time."""
    parts = [q @ w[0][lo:lo + 4096].double().t() for lo in range(0, w[0].shape[0], 4096)]
    return torch.cat(parts, dim=1) * (scale[:, None] * w[1].double()[None, :])


def exact(case, seed):
    global own
    was, own = own, False  # the inputs alone
    try:
        s = prepare(case, seed)
    finally:
        own = was
    x = s["x"].double()
    if case["op"] == "rows8":
        return None, _exact_rows(x)[1]
    if case["op"] == "linear8":
        q, scale = (s["xq"].double(), s["xs"].double()) if case["dtype"] == "int8" else _exact_rows(x)
        return _exact_product(q, scale, (s["wq"], s["ws"]))
    if case["op"] == "ffn8":
        rows = _exact_rows(x)
        gate = _exact_product(*rows, s["wg"])
        return _exact_product(*_exact_rows(torch.nn.functional.silu(gate) * _exact_product(*rows, s["w1"])), s["w2"])
    wg, w1, w2 = (s[n].double() for n in ("wg", "w1", "w2"))
    gate, up = torch.mm(x, wg.t()), torch.mm(x, w1.t())
    act = torch.nn.functional.silu(gate)
    if case["op"] == "gated":
        return torch.mm(act * up, w2.t())
    dy = s["dy"].double()
    back = torch.mm(dy, w2)
    # the derivative of g sigma(g): sigma(g) + g sigma(g) sigma(-g)
    slope = torch.sigmoid(gate) + act * torch.sigmoid(-gate)
    d_gate, d_up = back * up * slope, back * act
    return [torch.mm(act * up, w2.t()), torch.mm(d_gate, wg) + torch.mm(d_up, w1), torch.mm(d_gate.t(), x),
            torch.mm(d_up.t(), x), torch.mm(dy.t(), act * up)]
