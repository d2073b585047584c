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
