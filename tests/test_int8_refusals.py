"""Refusals of the 8-bit integer calls, found on the host before anything reaches a GPU."""
import ctypes

import pytest

from test_quant_refusals import Stand, pop  # noqa: F401

FAKE = 4096  # an aligned address that is never used: every call below is refused


@pytest.mark.parametrize("bad", [dict(x=None), dict(q=None), dict(s=None), dict(K=0), dict(K=12), dict(K=(1 << 30) + 8), dict(M=-1),
                                 dict(M=(1 << 27) + 1), dict(ldx=120), dict(ldx=132), dict(f32=1, ldx=130), dict(ldq=120), dict(ldq=130),
                                 dict(x=FAKE + 8), dict(q=FAKE + 4), dict(s=FAKE + 2), dict(f32=2)])
def test_rows_refuse(pop, bad):
    a = {**dict(x=FAKE, f32=0, ldx=128, M=4, K=128, q=FAKE, ldq=128, s=FAKE), **bad}
    st = pop.load_library().pop_quantize_rows_int(a["x"], a["f32"], a["ldx"], a["M"], a["K"], a["q"], a["ldq"], a["s"], None)
    assert st == pop.POP_ERR_INVALID_ARG
    assert pop.load_library().pop_int_last_error().startswith(b"pop_quantize_rows_int: ")


def test_no_rows(pop):
    assert pop.load_library().pop_quantize_rows_int(None, 0, 128, 0, 128, None, 128, None, None) == pop.POP_OK


@pytest.mark.parametrize("bad", [dict(N=0), dict(N=65537), dict(K=0), dict(K=12), dict(K=65544), dict(max_tokens=0),
                                 dict(max_tokens=(1 << 20) + 1), dict(out_f32=2)])
def test_linear_create_refuses(pop, bad):
    lib, out = pop.load_library(), ctypes.c_void_p(1)
    c = pop.pop_ilinear_config(**{**dict(N=64, K=64, max_tokens=4, out_f32=0), **bad})
    assert lib.pop_ilinear_create(ctypes.byref(c), FAKE, FAKE, None, ctypes.byref(out)) == pop.POP_ERR_INVALID_ARG
    assert out.value is None and lib.pop_int_last_error().startswith(b"pop_ilinear_create: ")


@pytest.mark.parametrize("bad", [dict(D=0), dict(D=12), dict(D_FF=65544), dict(D_FF=4), dict(max_tokens=0), dict(out_f32=-1)])
def test_ffn_create_refuses(pop, bad):
    lib, out = pop.load_library(), ctypes.c_void_p(1)
    c = pop.pop_iffn_config(**{**dict(D=64, D_FF=64, max_tokens=4, out_f32=0), **bad})
    assert lib.pop_iffn_create(ctypes.byref(c), *[FAKE] * 6, None, ctypes.byref(out)) == pop.POP_ERR_INVALID_ARG
    assert out.value is None and lib.pop_int_last_error().startswith(b"pop_iffn_create: ")


def test_pointers_that_are_missing_or_misaligned(pop):
    lib, out = pop.load_library(), ctypes.c_void_p(1)
    c, f = pop.pop_ilinear_config(N=64, K=64, max_tokens=4), pop.pop_iffn_config(D=64, D_FF=64, max_tokens=4)
    bad = pop.POP_ERR_INVALID_ARG
    for w, s in ((None, FAKE), (FAKE + 8, FAKE), (FAKE, FAKE + 2)):
        assert lib.pop_ilinear_create(ctypes.byref(c), w, s, None, ctypes.byref(out)) == bad
    assert lib.pop_ilinear_create(None, FAKE, FAKE, None, ctypes.byref(out)) == bad
    assert lib.pop_ilinear_create(ctypes.byref(c), FAKE, FAKE, None, None) == bad
    for i in range(6):  # a missing matrix; a missing scale beside others; either off its alignment
        for change in (None, FAKE + 2):
            p = [FAKE] * 6
            p[i] = change
            assert lib.pop_iffn_create(ctypes.byref(f), *p, None, ctypes.byref(out)) == bad
    for call in (lib.pop_ilinear_forward, lib.pop_iffn_forward):
        assert call(None, FAKE, 64, 1, FAKE, 64, None) == bad
    assert lib.pop_ilinear_forward_quantized(None, FAKE, 64, FAKE, 1, FAKE, 64, None) == bad
    for call in (lib.pop_ilinear_set_wait_limit, lib.pop_iffn_set_wait_limit):
        assert call(None, 1000) == bad
    for call in (lib.pop_ilinear_check, lib.pop_iffn_check):
        assert call(None) == bad
    lib.pop_ilinear_destroy(None)
    lib.pop_iffn_destroy(None)


def test_arguments_of_other_shapes_types_and_devices(pop, monkeypatch):
    import torch
    monkeypatch.setattr(pop, "_gpus", 2, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)
    f32, bf16, i8 = torch.float32, torch.bfloat16, torch.int8

    def refused(call):
        with pytest.raises(pop.PopError) as e:
            call()
        assert e.value.status == pop.POP_ERR_INVALID_ARG

    W, S = Stand((16, 8), i8, 0), Stand((16,), f32, 0)
    refused(lambda: pop.quantize_rows_i8(Stand((4, 8), i8, 0)))
    refused(lambda: pop.quantize_rows_i8(Stand((4, 8), bf16, 1)))
    refused(lambda: pop.quantize_rows_i8(Stand((4,), bf16, 0)))
    refused(lambda: pop.PopI8Linear(W))
    refused(lambda: pop.PopI8Linear(Stand((16, 8), bf16, 0), S))
    refused(lambda: pop.PopI8Linear(W, Stand((8,), f32, 0)))
    refused(lambda: pop.PopI8Linear(W, Stand((16,), f32, 1)))
    b, d = Stand((16, 8), bf16, 0), Stand((8, 16), bf16, 0)
    refused(lambda: pop.PopI8FFN(b, b, b))
    refused(lambda: pop.PopI8FFN(b, d, d))
    refused(lambda: pop.PopI8FFN((W, S), b, d))
    refused(lambda: pop.PopI8FFN(b, b, Stand((8, 16), bf16, 1)))
    h = pop.PopI8Linear.__new__(pop.PopI8Linear)  # ones whose handles are never reached
    h.__dict__.update(N=16, K=8, cfg=pop.pop_ilinear_config(N=16, K=8, max_tokens=4, out_f32=1))
    x = Stand((4, 8), bf16, 0)
    refused(lambda: h.forward(Stand((4, 16), bf16, 0)))
    refused(lambda: h.forward(Stand((4, 8), f32, 0)))
    refused(lambda: h.forward(Stand((4, 8), bf16, 1)))
    refused(lambda: h.forward(x, y=Stand((4, 16), bf16, 0)))
    refused(lambda: h.forward(x, y=Stand((3, 16), f32, 0)))
    refused(lambda: h.forward_q(Stand((4, 8), i8, 0), Stand((3,), f32, 0)))
    refused(lambda: h.forward_q(x, Stand((4,), f32, 0)))
    f = pop.PopI8FFN.__new__(pop.PopI8FFN)
    f.__dict__.update(N=16, D=8, cfg=pop.pop_iffn_config(D=8, D_FF=16, max_tokens=4, out_f32=0))
    refused(lambda: f.forward(Stand((4, 16), bf16, 0)))
    refused(lambda: f.forward(x, y=Stand((4, 8), f32, 0)))
    refused(lambda: f.forward(x, y=Stand((4, 8), bf16, 1)))
