"""Routing calls of several threads at once."""
import threading

import pytest
import torch

import mixture_experts_routing_moe_gb300 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("route,sizes", [
    (lambda l: moe.moe_route_sigmoid_grouped(l, 3, 1, 1), (290, 400, 500)),
    (lambda l: moe.moe_route(l, l.shape[1] - 8), (800, 900, 1000)),
])
def test_threads_with_routes_of_other_sizes(route, sizes):
    """The kernel's limit of shared memory is the process's: a call of one size does not take it from a
    larger call of another thread, between that one's look and its launch."""
    start, raised = threading.Barrier(len(sizes)), []

    def work(E):
        logits = torch.randn(5, E, device=DEV)
        start.wait()
        try:
            for _ in range(2000):
                route(logits)
        except Exception as e:  # noqa: BLE001
            raised.append(e)

    threads = [threading.Thread(target=work, args=(E,)) for E in sizes]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not raised
