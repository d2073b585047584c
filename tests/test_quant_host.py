"""Refusals of the routing and 8-bit calls, found on the host before anything reaches a GPU."""
import ctypes

import pytest

FAKE = 4096  # an aligned address that is never used: every call below is refused


@pytest.fixture(scope="module")
def pop():
    import __graft_entry__
    __graft_entry__.build()
    import online_structured_ffn_gb300 as pop
    return pop


ROUTE = dict(n_experts=16, top_k=2, score=0, n_groups=1, top_groups=1, group_sum=1, renorm=1, scale=1.0)


def route(pop, T=4, logits=FAKE, bf16=0, ld=16, bias=None, experts=FAKE, weights=FAKE, counts=None, **cfg):
    c = pop.pop_route_config(**{**ROUTE, **cfg})
    return pop.load_library().pop_route(ctypes.byref(c), logits, bf16, ld, bias, T, experts, weights, counts, None)


@pytest.mark.parametrize("bad", [
    dict(n_experts=0), dict(n_experts=257), dict(top_k=0), dict(top_k=17, n_experts=32), dict(top_k=17), dict(score=2),
    dict(n_groups=3), dict(n_groups=0), dict(top_groups=0), dict(n_groups=4, top_groups=5), dict(group_sum=0),
    dict(group_sum=3), dict(group_sum=2), dict(n_groups=8, top_groups=1, top_k=3), dict(renorm=2),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(T=-1), dict(T=1 << 28), dict(logits=None),
    dict(experts=None), dict(weights=None), dict(ld=15), dict(bf16=2), dict(logits=FAKE + 2), dict(logits=FAKE + 1, bf16=1),
    dict(experts=FAKE + 2), dict(weights=FAKE + 1), dict(bias=FAKE + 2), dict(counts=FAKE + 3)])
def test_route_refuses(pop, bad):
    assert route(pop, **bad) == pop.POP_ERR_INVALID_ARG
    assert pop.load_library().pop_route_last_error().startswith(b"pop_route: ")


def test_route_of_nothing(pop):
    assert route(pop, T=0, logits=None, experts=None, weights=None) == pop.POP_OK
    assert pop.load_library().pop_route(None, FAKE, 0, 16, None, 4, FAKE, FAKE, None, None) == pop.POP_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(x=None), dict(q=None), dict(s=None), dict(K=0), dict(K=12), dict(M=-1), dict(ldx=120),
                                 dict(ldx=132), dict(f32=1, ldx=130), dict(ldq=120), dict(ldq=130), dict(x=FAKE + 8),
                                 dict(q=FAKE + 4), dict(s=FAKE + 2), dict(f32=2)])
def test_quantize_refuses(pop, bad):
    a = {**dict(x=FAKE, f32=0, ldx=128, M=4, K=128, q=FAKE, ldq=128, s=FAKE), **bad}
    st = pop.load_library().pop_quantize_rows(a["x"], a["f32"], a["ldx"], a["M"], a["K"], a["q"], a["ldq"], a["s"], None)
    assert st == pop.POP_ERR_INVALID_ARG
    assert pop.load_library().pop_quant_last_error().startswith(b"pop_quantize_rows: ")


def test_quantize_of_nothing(pop):
    assert pop.load_library().pop_quantize_rows(None, 0, 128, 0, 128, None, 128, None, None) == pop.POP_OK


@pytest.mark.parametrize("bad", [dict(N=0), dict(N=65537), dict(K=0), dict(K=12), dict(K=65544), dict(max_tokens=0),
                                 dict(max_tokens=(1 << 20) + 1), dict(out_f32=2)])
def test_linear_create_refuses(pop, bad):
    lib, out = pop.load_library(), ctypes.c_void_p(1)
    c = pop.pop_qlinear_config(**{**dict(N=64, K=64, max_tokens=4, out_f32=0), **bad})
    assert lib.pop_qlinear_create(ctypes.byref(c), FAKE, FAKE, None, ctypes.byref(out)) == pop.POP_ERR_INVALID_ARG
    assert out.value is None


def test_null_and_misaligned_handles(pop):
    lib, out = pop.load_library(), ctypes.c_void_p(1)
    bad = pop.POP_ERR_INVALID_ARG
    c = pop.pop_qlinear_config(N=64, K=64, max_tokens=4, out_f32=0)
    assert lib.pop_qlinear_create(ctypes.byref(c), None, None, None, ctypes.byref(out)) == bad and out.value is None
    assert lib.pop_qlinear_create(ctypes.byref(c), FAKE + 8, None, None, ctypes.byref(out)) == bad
    assert lib.pop_qlinear_create(ctypes.byref(c), FAKE, FAKE + 2, None, ctypes.byref(out)) == bad
    assert lib.pop_qlinear_create(None, FAKE, None, None, ctypes.byref(out)) == bad
    assert lib.pop_qlinear_create(ctypes.byref(c), FAKE, None, None, None) == bad
    assert lib.pop_qlinear_forward(None, FAKE, 64, 1, FAKE, 64, None) == bad
    assert lib.pop_qlinear_forward_quantized(None, FAKE, 64, FAKE, 1, 1, FAKE, 64, None) == bad
    assert lib.pop_qlinear_check(None) == bad and lib.pop_qmoe_check(None) == bad
    assert lib.pop_qmoe_forward(None, FAKE, 64, FAKE, FAKE, 1, FAKE, 64, None) == bad
    assert b"NULL" in lib.pop_quant_last_error()
    lib.pop_qlinear_destroy(None)
    lib.pop_qmoe_destroy(None)


def test_experts_create_refuses(pop):
    lib, out = pop.load_library(), ctypes.c_void_p(1)
    good = dict(n_experts=2, top_k=1, D=64, D_FF=128, max_tokens=4, out_f32=0)

    def ptrs(*v):
        return (ctypes.c_void_p * len(v))(*v)

    p = ptrs(FAKE, FAKE)

    def create(args, **cfg):
        c = pop.pop_qmoe_config(**{**good, **cfg})
        st = lib.pop_qmoe_create(ctypes.byref(c), *args, None, ctypes.byref(out))
        assert out.value is None
        return st

    bad = pop.POP_ERR_INVALID_ARG
    for cfg in (dict(n_experts=0), dict(n_experts=257), dict(top_k=0), dict(top_k=17), dict(D=12), dict(D=0), dict(D_FF=0),
                dict(D_FF=65544), dict(max_tokens=0), dict(out_f32=-1)):
        assert create((p, p, p, None, None, None), **cfg) == bad, cfg
    assert create((None, p, p, None, None, None)) == bad
    assert create((p, p, p, p, None, p)) == bad  # scales of some matrices only
    assert create((p, ptrs(FAKE, None), p, None, None, None)) == bad
    assert create((p, p, p, p, p, ptrs(None, FAKE))) == bad
    assert create((ptrs(FAKE, FAKE + 8), p, p, None, None, None)) == bad
    assert lib.pop_quant_last_error().startswith(b"pop_qmoe_create: ")


def test_binding_refuses_what_is_not_a_cuda_tensor_of_the_right_kind(pop):
    torch = pytest.importorskip("torch")
    with pytest.raises(pop.PopError):
        pop.PopRouter(8, 2, score="relu")
    r = pop.PopRouter(8, 2)
    for bad in (torch.zeros(4, 8), torch.zeros(4, 7), torch.zeros((4, 8), dtype=torch.float64), torch.zeros(8)):
        with pytest.raises(pop.PopError) as e:
            r.route(bad)
        assert e.value.status == pop.POP_ERR_INVALID_ARG
    with pytest.raises(pop.PopError):
        pop.quantize_rows(torch.zeros((4, 8), dtype=torch.bfloat16))  # on the CPU
    with pytest.raises(pop.PopError):
        pop.quantize_rows(torch.zeros(8))
    with pytest.raises(pop.PopError):
        pop.PopQLinear(torch.zeros((8, 8), dtype=torch.bfloat16))
    with pytest.raises(pop.PopError):
        pop.PopQMoE([torch.zeros((8, 8), dtype=torch.bfloat16)], [torch.zeros((8, 8))], [torch.zeros((8, 8))], top_k=1)
