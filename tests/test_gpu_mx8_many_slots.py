"""The 8-bit layer on both sides of 2048 slots, where the launches that dispatch its tokens change: against
the float64 oracle, bit for bit against its stages, with ids that name no expert, and on a workspace that
is all it has asked for.  Tolerances are those of the smaller layers."""
import numpy as np
import pytest
import torch

import mixture_experts_routing_moe_gb300 as moe
from test_gpu_mx8 import DEV, check_within, experts_reference, half_step, layer, np64

pytestmark = pytest.mark.gpu
# T, E, H, I, k: exactly 2048 slots, one more, thousands; pairs and single CTAs; every expert of a token's
SIZES = [(256, 16, 96, 64, 8), (683, 5, 72, 50, 3), (1024, 4, 64, 33, 2), (2048, 3, 40, 72, 1), (2049, 2, 40, 72, 1),
         (3000, 24, 200, 160, 4), (3000, 64, 136, 96, 4), (40, 60, 72, 40, 52), (2500, 3, 100, 264, 3)]


@pytest.mark.parametrize("dtype,wdt", [(torch.bfloat16, torch.float32), (torch.float32, torch.float16)])
@pytest.mark.parametrize("T,E,H,I,k", SIZES)
def test_layer(dtype, wdt, T, E, H, I, k):
    x, xv, packed, w, idx, ids, gate = layer(T, E, H, I, k, T + E)
    gate = torch.from_numpy(gate).to(wdt)
    ws = torch.full((moe.mx8_forward_workspace_bytes(T, E, H, I, k, dtype) + 256,), 255, dtype=torch.uint8, device=DEV)
    out = moe.moe_mx8_forward(x, idx, gate.to(DEV), *packed, dtype=dtype, ws=ws[:-256])
    assert moe.moe_device_status(ws) == 0 and (ws[-256:] == 255).all()
    ref, tol = np.zeros((T, H)), np.zeros((T, H))
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if len(t):
            y, d = experts_reference(xv[t], [m[e] for m in w], H, I)
            p = np64(gate)[t, j][:, None]
            np.add.at(ref, t, p * y)
            np.add.at(tol, t, p * (d * (1 + torch.finfo(dtype).eps) + half_step(dtype, y) + k * 2.0 ** -23 * np.abs(y)))
    tol = tol * (1 + torch.finfo(dtype).eps) + half_step(dtype, ref)
    check_within(np64(out), ref, tol, dtype)
    d = moe.moe_mx8_dispatch(*x, idx, E, H)
    y = moe.moe_mx8_experts_forward_dispatched((d["codes"], d["scales"]), d["offsets"], *packed, dtype=dtype)
    assert torch.equal(moe.moe_combine(y, d["row_of_slot"], gate.to(DEV)), out)


@pytest.mark.parametrize("T,k", [(1024, 2), (1025, 2), (700, 3), (4000, 4)])
def test_ids_that_name_no_expert(T, k):
    x, _, packed, _, idx, _, gate = layer(T, 4, 64, 96, k, 3)
    g = torch.from_numpy(gate).float().to(DEV)
    ws = torch.empty(moe.mx8_forward_workspace_bytes(T, 4, 64, 96, k, torch.bfloat16), dtype=torch.uint8, device=DEV)
    want = moe.moe_mx8_forward(x, idx, g, *packed, ws=ws)
    assert moe.moe_device_status(ws) == 0
    bad = [0, T // 2, T - 1]
    good = np.delete(np.arange(T), bad)
    ids = idx.view(torch.int32)
    ids[0, 0], ids[T // 2, k - 1], ids[T - 1, 1] = 4, -1, 1 << 20
    out = moe.moe_mx8_forward(x, idx, g, *packed, ws=ws)
    assert moe.moe_device_status(ws) == 8
    assert torch.isnan(out[bad]).all() and torch.equal(out[good], want[good])
    ids[:] = 7
    assert torch.isnan(moe.moe_mx8_forward(x, idx, g, *packed, ws=ws)).all() and moe.moe_device_status(ws) == 8


@pytest.mark.parametrize("T", [1024, 1025])
def test_repeats_and_graphs(T):
    """The same bits every time, on another stream, and from two graphs of the two paths in turn."""
    x, _, packed, _, idx, _, gate = layer(T, 6, 128, 96, 2, 5)
    g = torch.from_numpy(gate).float().to(DEV)
    call = lambda n, **kw: moe.moe_mx8_forward((x[0][:n], x[1][:n]), idx[:n], g[:n], *packed, **kw)  # noqa: E731
    want = {n: call(n) for n in (T, 17)}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(T, stream=side)
    side.synchronize()
    assert torch.equal(got, want[T])
    graphs, out = {}, {}
    for n in want:
        graphs[n] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[n]):
            out[n] = call(n)
    for _ in range(3):
        for n in want:
            out[n].zero_()
            graphs[n].replay()
        assert torch.equal(call(T), want[T])
        torch.cuda.synchronize()
        assert all(torch.equal(out[n], want[n]) for n in want)
