"""Routing where there is nothing, or next to nothing, to route."""
import pytest

from test_gpu_route import env  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E", [1, 8, 256])
def test_counts_of_no_tokens_are_zero(env, E):
    pop, torch, dev = env
    r = pop.PopRouter(E, 1)
    counts = torch.full((E,), -7, dtype=torch.int32, device=dev)
    e, w = r.route(torch.zeros((0, E), device=dev), counts=counts)
    assert e.shape == (0, 1) and w.shape == (0, 1)
    assert counts.tolist() == [0] * E
    r.route(torch.zeros((5, E), device=dev), counts=counts)
    assert counts.tolist() == [5] + [0] * (E - 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r.route(torch.zeros((0, E), dtype=torch.bfloat16, device=dev), counts=counts, stream=side)
    side.synchronize()
    assert counts.tolist() == [0] * E
