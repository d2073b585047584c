"""Refusals of the trainable gated MLP, found on the host before anything reaches a GPU."""
import ctypes

import pytest

from test_quant_refusals import Stand, pop  # noqa: F401

FAKE = 4096  # an aligned address that is never used: every call below is refused


@pytest.mark.parametrize("bad", [dict(D=0), dict(D=12), dict(D=65544), dict(D_FF=0), dict(D_FF=20), dict(D_FF=65544), dict(D=-8),
                                 dict(max_tokens=0), dict(max_tokens=(1 << 20) + 1), dict(out_f32=2), dict(grad_f32=-1)])
def test_create_refuses(pop, bad):
    lib, out = pop.load_library(), ctypes.c_void_p(1)
    c = pop.pop_gated_config(**{**dict(D=64, D_FF=64, max_tokens=4, out_f32=0, grad_f32=0), **bad})
    assert lib.pop_gated_create(ctypes.byref(c), ctypes.byref(out)) == pop.POP_ERR_INVALID_ARG
    assert out.value is None and lib.pop_gated_last_error().startswith(b"pop_gated_create: ")


def test_nothing_to_work_with(pop):
    lib, out = pop.load_library(), ctypes.c_void_p(1)
    c = pop.pop_gated_config(D=64, D_FF=64, max_tokens=4, out_f32=0, grad_f32=0)
    assert lib.pop_gated_create(None, ctypes.byref(out)) == pop.POP_ERR_INVALID_ARG
    assert lib.pop_gated_create(ctypes.byref(c), None) == pop.POP_ERR_INVALID_ARG
    assert lib.pop_gated_forward(None, FAKE, 64, 1, FAKE, FAKE, FAKE, FAKE, 64, None, None) == pop.POP_ERR_INVALID_ARG
    assert lib.pop_gated_backward(None, FAKE, 64, 1, FAKE, FAKE, FAKE, FAKE, FAKE, 64, FAKE, 64, FAKE, FAKE, FAKE, 0,
                                  None) == pop.POP_ERR_INVALID_ARG
    assert lib.pop_gated_set_wait_limit(None, 1) == pop.POP_ERR_INVALID_ARG
    assert lib.pop_gated_check(None) == pop.POP_ERR_INVALID_ARG
    lib.pop_gated_destroy(None)


def test_bytes_that_are_kept(pop):
    size = pop.load_library().pop_gated_saved_bytes
    assert size(64, 0) == 0 and size(12, 4) == 0 and size(64, -1) == 0 and size(64, (1 << 20) + 1) == 0
    assert size(64, 1) == 32 * 64 * 6 + 64 * 2 and size(64, 32) == 32 * 64 * 8
    assert size(65536, 1 << 20) == 8 << 36  # beyond 32 bits


def gone(pop):
    f = pop.PopGatedFFN.__new__(pop.PopGatedFFN)  # one whose handle is never reached
    f.__dict__.update(D=16, N=8, _shapes=((8, 16), (16, 8)), _kept_bytes={}, cfg=pop.pop_gated_config(D=16, D_FF=8, max_tokens=4, out_f32=0, grad_f32=0))
    return f


def test_arguments_of_other_shapes_types_and_devices(pop, monkeypatch):
    import torch
    monkeypatch.setattr(pop, "_gpus", 2, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)
    bf16, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
    f = gone(pop)
    rows = lambda r=4, c=16, t=bf16, i=0: Stand((r, c), t, i)  # noqa: E731
    good = dict(x=rows(), Wg=rows(8), W1=rows(8), W2=rows(16, 8))
    kept = Stand((32 * 8 * 6 + 4 * 8 * 2,), u8, 0)

    def refused(call, **change):
        with pytest.raises(pop.PopError) as e:
            call(change)
        assert e.value.status == pop.POP_ERR_INVALID_ARG

    for change in (dict(x=rows(c=8)), dict(x=rows(t=f32)), dict(Wg=rows(16)), dict(W1=rows(8, t=f32)), dict(W2=rows(8)),
                   dict(x=rows(i=1)), dict(W1=rows(8, i=1)), dict(y=rows(3)), dict(y=rows(t=f32)), dict(y=rows(i=1))):
        refused(lambda c: f.forward(**{**good, **c}), **change)
    back = dict(good, dy=rows(), saved=kept)
    grads = (rows(8), rows(8), rows(16, 8))
    for change in (dict(dy=rows(3)), dict(dy=rows(t=f32)), dict(saved=Stand((4,), u8, 0)), dict(saved=rows()), dict(dy=rows(i=1)),
                   dict(need=(True,)), dict(grads=grads[:2]), dict(accumulate=True), dict(accumulate=True, grads=(None, *grads[1:])),
                   dict(grads=(rows(8, t=f32), *grads[1:]), need=(False, True, True, True)),
                   dict(grads=(rows(8, i=1), *grads[1:]))):
        refused(lambda c: f.backward(**{**back, **c}), **change)
