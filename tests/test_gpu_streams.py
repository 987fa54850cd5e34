"""Calls of the layer's entry points on a given stream that is not the current one: what they write
lies in memory of that stream."""
import pytest
import torch

import mixture_experts_routing_moe_gb300 as moe
from mixture_experts_routing_moe_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


def flat(r):
    if isinstance(r, dict):
        r = [r[n] for n in sorted(r) if n != "ws"]
    return [r] if isinstance(r, torch.Tensor) else list(r)


def test_a_given_streams_memory_is_its_own():
    """The current stream has work queued on memory that it has given back, as much as each buffer of
    the call; neither results nor workspaces lie there."""
    T, E, H, I, k = 600, 4, 256, 384, 2
    g = torch.Generator(device=DEV)
    g.manual_seed(3)

    def normal(*s):
        return (torch.randn(*s, generator=g, device=DEV) * s[-1] ** -0.5).bfloat16()

    x, logits = normal(T, H) * 16, normal(T, E) * 2
    gate, up, down = normal(E, I, H), normal(E, I, H), normal(E, H, I)
    idx, w = moe.moe_route(logits, k)
    d = moe.moe_dispatch(x, idx, E)
    y = moe.moe_experts_forward_dispatched(d["x_d"], d["offsets"], gate, up, down)
    sizes = [T * k * H * 2, T * H * 2, T * k * 4, T * k * 2, E * I * H * 4, (E + 1) * 4,
             B.forward_workspace_bytes(T, E, H, I, k, logits.dtype, x.dtype),
             B.experts_workspace_bytes(T * k, E, H, I, x.dtype)]
    jobs = [
        lambda s: moe.moe_route(logits, k, stream=s),
        lambda s: moe.moe_dispatch(x, idx, E, stream=s),
        lambda s: moe.moe_experts_forward_dispatched(d["x_d"], d["offsets"], gate, up, down, stream=s),
        lambda s: moe.moe_combine(y, d["row_of_slot"], w, stream=s),
        lambda s: moe.moe_forward(x, logits, gate, up, down, k, stream=s),
        lambda s: moe.moe_combine_backward(y, d["row_of_slot"], w, x, stream=s),
        lambda s: moe.moe_experts_backward(d["x_d"], d["offsets"], gate, up, down, y, stream=s),
        lambda s: moe.moe_dispatch_backward(y, d["row_of_slot"], T, k, stream=s),
    ]
    side = torch.cuda.Stream()
    for job in jobs:
        want = flat(job(None))
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        torch.cuda._sleep(20_000_000)
        for n in sizes:
            torch.empty(n, dtype=torch.uint8, device=DEV).fill_(1)
        got = flat(job(side))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
