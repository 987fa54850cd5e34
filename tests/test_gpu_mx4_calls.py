"""Microscaled 4-bit calls from several threads and on other streams than the current one."""
import threading

import pytest
import torch

import mixture_experts_routing_moe_gb300 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"


def weights(E, H, I, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return [moe.moe_mx4_quantize(torch.randn(*s, generator=g, device=DEV) * s[2] ** -0.5)
            for s in ((E, I, H), (E, I, H), (E, H, I))]


def calls(seed, T, E, H, I, k):
    """(layer for few tokens, experts over rows) as functions without arguments."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    w = weights(E, H, I, seed)
    x = torch.randn(T, H, generator=g, device=DEV).bfloat16()
    router = (torch.randn(E, H, generator=g, device=DEV) * H ** -0.5).bfloat16()
    rows = torch.randn(E * 24, H, generator=g, device=DEV).bfloat16()
    off = torch.arange(E + 1, device=DEV, dtype=torch.int32) * 24
    return (lambda: moe.moe_mx4_forward_tokens(x, router, *w, top_k=k),
            lambda: moe.moe_mx4_experts_forward_dispatched(rows, off, *w))


def test_two_threads_on_one_stream():
    """Both threads stay on the default stream; each result is that of the same call on its own."""
    jobs = [calls(1, 6, 8, 512, 384, 2), calls(2, 11, 12, 256, 640, 3)]
    want = [[f() for f in job] for job in jobs]
    torch.cuda.synchronize()
    start, wrong = threading.Barrier(2), []

    def work(n):
        start.wait()
        for i in range(150):
            got = [f() for f in jobs[n]]
            if i % 10 == 0 and not all(torch.equal(a, b) for a, b in zip(got, want[n])):
                wrong.append((n, i))

    threads = [threading.Thread(target=work, args=(n,)) for n in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong
