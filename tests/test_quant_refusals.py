"""More refusals of the routing and 8-bit calls on the host: wait limits."""
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
