"""More refusals of the routing and 8-bit calls on the host."""
import pytest


@pytest.fixture(scope="module")
def pop():
    import __graft_entry__
    __graft_entry__.build()
    import online_structured_ffn_gb300 as pop
    return pop


def test_wait_limit_of_no_handle(pop):
    lib = pop.load_library()
    for call in (lib.pop_qlinear_set_wait_limit, lib.pop_qmoe_set_wait_limit):
        assert call(None, 1000) == pop.POP_ERR_INVALID_ARG
        assert b"set_wait_limit" in lib.pop_quant_last_error()


def test_counts_of_no_tokens_are_checked(pop):
    """With counts there is something to write for no tokens, too."""
    import ctypes
    lib = pop.load_library()
    cfg = pop.pop_route_config(n_experts=16, top_k=2, score=0, n_groups=1, top_groups=1, group_sum=1, renorm=1, scale=1.0)
    assert lib.pop_route(ctypes.byref(cfg), None, 0, 16, None, 0, None, None, 4097, None) == pop.POP_ERR_INVALID_ARG
    assert b"counts" in lib.pop_route_last_error()
    assert lib.pop_route(ctypes.byref(cfg), None, 0, 16, None, 0, None, None, None, None) == pop.POP_OK


class Stand:
    """Stands in for a contiguous CUDA tensor of a machine with several GPUs."""
    is_cuda = True

    def __init__(self, shape, dtype, index):
        import torch
        self.shape, self.dtype, self.index = tuple(shape), dtype, index
        self.device = torch.device("cuda", index)

    def dim(self):
        return len(self.shape)

    def stride(self):
        return (self.shape[1], 1)

    def is_contiguous(self):
        return True

    def element_size(self):
        return self.dtype.itemsize

    def data_ptr(self):
        return 4096

    def get_device(self):
        return self.index

    def record_stream(self, stream):
        raise AssertionError("reached a stream")


def test_tensors_of_another_device_are_refused(pop, monkeypatch):
    """A call launches on the current device: everything it is given has to lie there."""
    import torch
    monkeypatch.setattr(pop, "_gpus", 2, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    f32, bf16, i32, fp8 = torch.float32, torch.bfloat16, torch.int32, torch.float8_e4m3fn

    def refused(call):
        with pytest.raises(pop.PopError) as e:
            call()
        assert e.value.status == pop.POP_ERR_INVALID_ARG and "cuda:1" in str(e.value)

    r = pop.PopRouter(8, 2)
    here, there = Stand((4, 8), f32, 0), Stand((4, 8), f32, 1)
    refused(lambda: r.route(there))
    refused(lambda: r.route(here, bias=Stand((8,), f32, 1)))
    refused(lambda: r.route(here, counts=Stand((8,), i32, 1)))
    refused(lambda: pop.quantize_rows(Stand((4, 8), bf16, 1)))
    refused(lambda: pop.PopQLinear(Stand((8, 8), bf16, 1)))
    refused(lambda: pop.PopQLinear(Stand((8, 8), fp8, 0), Stand((1, 1), f32, 1)))

    def gone(kind, **attributes):
        h = kind.__new__(kind)  # one whose handle is never reached
        h.__dict__.update(attributes)
        return h

    h = gone(pop.PopQLinear, N=8, K=8, cfg=pop.pop_qlinear_config(N=8, K=8, max_tokens=4, out_f32=1))
    x0, x1, xq, xs = Stand((4, 8), bf16, 0), Stand((4, 8), bf16, 1), Stand((4, 8), fp8, 0), Stand((4, 1), f32, 0)
    refused(lambda: h.forward(x1))
    refused(lambda: h.forward(x0, y=there))
    refused(lambda: h.forward_q(Stand((4, 8), fp8, 1), xs))
    refused(lambda: h.forward_q(xq, Stand((4, 1), f32, 1)))
    m = gone(pop.PopQMoE, D=8, N=8, E=2, cfg=pop.pop_qmoe_config(n_experts=2, top_k=2, D=8, D_FF=8, max_tokens=4, out_f32=1))
    e, w = Stand((4, 2), i32, 0), Stand((4, 2), f32, 0)
    refused(lambda: m.forward(x1, e, w))
    refused(lambda: m.forward(x0, Stand((4, 2), i32, 1), w))
    refused(lambda: m.forward(x0, e, Stand((4, 2), f32, 1)))
    refused(lambda: m.forward(x0, e, w, y=there))
    a, b = [Stand((8, 8), bf16, 0)] * 2, [Stand((8, 8), bf16, 0), Stand((8, 8), bf16, 1)]
    refused(lambda: pop.PopQMoE(a, b, a, top_k=1))
    # all on one device, which is not the current one; and a stream of another
    refused(lambda: pop.PopQMoE(b[1:], b[1:], b[1:], top_k=1))

    class Stream:
        device_index, cuda_stream = 1, 12345

    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)
    refused(lambda: r.route(here, stream=Stream()))


@pytest.mark.parametrize("K", [(1 << 28) - 4088, 1 << 28, (1 << 31) - 8])
def test_rows_longer_than_a_grid_are_refused(pop, K):
    lib = pop.load_library()
    assert lib.pop_quantize_rows(4096, 0, K, 1, K, 4096, K, 4096, None) == pop.POP_ERR_INVALID_ARG
    assert b"2^28" in lib.pop_quant_last_error()


def test_a_stream_that_names_no_device_is_taken_as_it_is(pop, monkeypatch):
    """Any object with a raw handle will do for the current stream."""
    import torch
    monkeypatch.setattr(pop, "_gpus", 1)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 77, raising=False)

    class Stream:
        cuda_stream = 77

    assert pop._on(Stream(), Stand((4, 8), torch.float32, 0)) == (77, None)
