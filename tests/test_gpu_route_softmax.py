"""The grouped softmax router on the GPU against the float64 oracle: ids are equal; weights are FP32
probabilities, off by 2.5e-6 + 6.5e-8 * 32 (the sum of exponentials, as route_softmax.cu derives it) and
by 8 more roundings, plus half a step of their type.
"""
import numpy as np
import pytest
import torch

import mixture_experts_routing_moe_gb300 as moe
from oracle import front_oracle as F

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [torch.float32, torch.float16, torch.bfloat16]


def np64(t):
    return t.double().cpu().numpy()


def check(logits, k, G, SG, two, renorm=True, scale=1.0, bias=None):
    idx, w = moe.moe_route_softmax_grouped(logits.to(DEV), k, G, SG, group_top_two=two, renormalize=renorm,
                                           scale=scale, bias=None if bias is None else bias.to(DEV))
    ids, ref = F.route_softmax_grouped(np64(logits), k, G, SG, two, renorm, scale,
                                       None if bias is None else np64(bias))
    got = idx.view(torch.int32).cpu().numpy()
    assert (got == ids).all(), np.argwhere(got != ids)[:4]
    g, fin = np64(w), np.isfinite(ref)
    assert w.dtype == logits.dtype and (np.isnan(g) == np.isnan(ref)).all()
    tiny = torch.finfo(logits.dtype).tiny * 2 ** -3 + 1e-38
    tol = (4.6e-6 + 8 * 2.0 ** -24 + torch.finfo(logits.dtype).eps / 2) * np.abs(ref) + tiny
    assert (np.abs(g - ref)[fin] <= tol[fin]).all()


def logits_of(T, E, dtype, seed, spread=2.0):
    return torch.from_numpy(spread * np.random.default_rng(seed).standard_normal((T, E))).to(dtype)


def bias_of(E, seed):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(E) / E).float()


SHAPES = [(1, 1, 1, 1, 1), (3, 2, 2, 1, 1), (40, 8, 2, 4, 2), (300, 64, 6, 8, 3), (300, 160, 6, 8, 3),
          (200, 256, 8, 8, 4), (100, 256, 8, 1, 1), (33, 153, 11, 3, 2), (20, 512, 64, 16, 8),
          (9, 1024, 40, 128, 100), (9, 1000, 16, 5, 5), (7, 1023, 5, 11, 2), (50, 96, 33, 6, 5), (5, 31, 31, 1, 1)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,E,k,G,SG", SHAPES)
@pytest.mark.parametrize("two", [False, True])
def test_matches_the_definition(dtype, T, E, k, G, SG, two):
    if two and E // G < 2:
        return
    x = logits_of(T, E, dtype, T + E + G)
    check(x, k, G, SG, two)
    check(x, k, G, SG, two, renorm=False, scale=2.5, bias=bias_of(E, E))
    check(x, k, G, SG, two, renorm=False, bias=torch.zeros(E))           # balancing's first step: ties
    check(x, k, G, SG, two, scale=0.5, bias=100 * bias_of(E, E + 1))


@pytest.mark.parametrize("two", [False, True])
@pytest.mark.parametrize("with_bias", [False, True])
def test_near_ties_are_decided_in_64_bits(two, with_bias):
    """FP32 logits a few units apart, far below what FP32 probabilities resolve."""
    rng = np.random.default_rng(5)
    x = torch.from_numpy((1.0 + rng.integers(0, 40, (400, 64)) * 2.0 ** -23).astype(np.float32))
    x[::2] += torch.from_numpy(rng.integers(0, 2, (200, 64)).astype(np.float32))
    bias = None
    if with_bias:
        bias = torch.from_numpy((rng.integers(-3, 4, 64) * 2.0 ** -31).astype(np.float32))
    for k, G, SG in ((8, 8, 3), (6, 4, 2), (20, 1, 1), (5, 16, 9)):
        check(x, k, G, SG, two, renorm=False, bias=bias)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("two", [False, True])
def test_all_ties(dtype, two):
    x = torch.zeros(3, 128, dtype=dtype)
    x[1, ::2] = -0.0
    x[2, 64:] = 1.0
    for bias in (None, torch.zeros(128), torch.full((128,), -0.25)):
        check(x, 8, 8, 3, two, bias=bias)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bias", [None, 1])
@pytest.mark.parametrize("two", [False, True])
def test_rows_that_hold_infinities_and_nan(dtype, bias, two):
    x = logits_of(9, 64, dtype, 3)
    x[0, 7] = float("nan")
    x[1, 9] = float("inf")
    x[2] = float("-inf")
    x[3, 3:] = float("-inf")                   # fewer finite logits than slots
    x[4, ::2] = float("-inf")
    x[5] = torch.finfo(dtype).min
    x[6, 10] = torch.finfo(dtype).max
    x[7, 8:] = torch.finfo(dtype).min
    check(x, 8, 8, 4, two, renorm=False, bias=None if bias is None else bias_of(64, 1))
    check(x, 8, 1, 1, two, renorm=False, bias=None if bias is None else bias_of(64, 1))


@pytest.mark.parametrize("two", [False, True])
def test_bias_that_leaves_experts_out(two):
    x, bias = logits_of(40, 64, torch.float32, 8), bias_of(64, 8)
    bias[10:30] = float("-inf")
    check(x, 8, 8, 4, two, bias=bias)
    bias[:] = float("-inf")
    bias[5], bias[41] = 0.0, 0.1               # fewer than slots
    check(x, 8, 8, 4, two, renorm=False, bias=bias)
    bias = bias_of(64, 9)
    bias[13] = float("inf")                    # always taken
    check(x, 8, 8, 4, two, bias=bias)
    bias[13] = float("nan")
    check(x, 8, 8, 4, two, bias=bias)
    bias = bias_of(64, 9)
    bias[20] = 3e38
    check(x, 8, 8, 4, two, bias=bias)


def test_a_bias_against_every_likely_expert():
    """Renormalised weights of experts whose probabilities vanish in FP32."""
    x, bias = logits_of(20, 64, torch.float32, 4), torch.zeros(64)
    x[:, :32] += 150.0
    bias[32:] = 1.5
    check(x, 8, 8, 3, True, renorm=True, bias=bias)
    check(x, 8, 1, 1, False, renorm=True, bias=bias)


def test_large_batches_and_rows_on_any_element():
    x = logits_of(70001, 40, torch.bfloat16, 6)
    flat = torch.zeros(70001 * 40 + 1, dtype=torch.bfloat16, device=DEV)
    flat[1:] = x.to(DEV).view(-1)
    a = moe.moe_route_softmax_grouped(x.to(DEV), 4, 5, 2)
    b = moe.moe_route_softmax_grouped(flat[1:].view(70001, 40), 4, 5, 2)
    assert torch.equal(a[0].view(torch.int32), b[0].view(torch.int32)) and torch.equal(a[1], b[1])
    check(x[-300:], 4, 5, 2, True)


@pytest.mark.parametrize("scoring", ["weights", "gradient"])
def test_the_gradient_of_its_weights(scoring):
    """moe_selected_router_weights repeats the weights from the ids, so its backward is theirs."""
    x, bias = logits_of(50, 64, torch.float32, 2).to(DEV), bias_of(64, 3).to(DEV)
    idx, w = moe.moe_route_softmax_grouped(x, 6, 8, 3, scale=2.0, bias=bias)
    if scoring == "weights":
        again = moe.moe_selected_router_weights(x, idx, "softmax", True, 2.0)
        assert (again - w).abs().max() <= 2e-5
        return
    gw = torch.randn(50, 6, device=DEV)
    got = moe.moe_selected_router_backward(x, idx, gw, "softmax", True, 2.0)
    l = x.double().requires_grad_()
    p = torch.softmax(l, -1).gather(1, idx.view(torch.int32).long())
    (p / p.sum(-1, keepdim=True) * 2.0 * gw).sum().backward()
    assert (got - l.grad).abs().max() <= 1e-5


@pytest.mark.parametrize("dtype,T", [(torch.bfloat16, 40), (torch.float32, 9), (torch.bfloat16, 700)])
def test_forward_is_the_stages(dtype, T):
    E, H, I = 16, 64, 96
    g = torch.Generator(device=DEV).manual_seed(T)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV).to(dtype)  # noqa: E731
    x, gate, up, down = n(T, H), n(E, I, H) / 8, n(E, I, H) / 8, n(E, H, I) / 10
    logits = torch.randn(T, E, generator=g, device=DEV)
    bias = torch.randn(E, generator=g, device=DEV) / E
    out = moe.moe_forward_softmax_grouped(x, logits, gate, up, down, 3, 4, 2, scale=1.5, bias=bias)
    idx, w = moe.moe_route_softmax_grouped(logits, 3, 4, 2, scale=1.5, bias=bias)
    d = moe.moe_dispatch(x, idx, E)
    y = moe.moe_experts_forward_dispatched(d["x_d"], d["offsets"], gate, up, down)
    assert torch.equal(moe.moe_combine(y, d["row_of_slot"], w), out)
    one = moe.moe_forward_softmax_grouped(x, logits, gate, up, down, 3, 1, 1, group_top_two=False)
    plain = moe.moe_forward(x, logits, gate, up, down, 3)
    assert (one.double() - plain.double()).abs().max() <= 2e-2 * plain.double().abs().max()


def test_streams_graphs_and_empty():
    x, bias = logits_of(500, 256, torch.bfloat16, 1).to(DEV), bias_of(256, 1).to(DEV)
    call = lambda **kw: moe.moe_route_softmax_grouped(x, 8, 8, 4, bias=bias, **kw)  # noqa: E731
    idx, w = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(stream=side)
    side.synchronize()
    assert torch.equal(got[0].view(torch.int32), idx.view(torch.int32)) and torch.equal(got[1], w)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = call()
    got[1].zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0].view(torch.int32), idx.view(torch.int32)) and torch.equal(got[1], w)
    empty = moe.moe_route_softmax_grouped(x[:0], 8, 8, 4)
    assert empty[0].shape == (0, 8) and empty[1].shape == (0, 8)


def test_refusals():
    x, b = torch.zeros(4, 64, device=DEV), torch.zeros(64, device=DEV)
    route = moe.moe_route_softmax_grouped
    for error, call in [
            (ValueError, lambda: route(x.cpu(), 2, 4, 2)), (ValueError, lambda: route(x[:, ::2], 2, 4, 2)),
            (moe.MoeError, lambda: route(x.double(), 2, 4, 2)), (moe.MoeError, lambda: route(x, 2, 5, 2)),
            (moe.MoeError, lambda: route(x, 33, 4, 2)), (moe.MoeError, lambda: route(x, 2, 4, 5)),
            (moe.MoeError, lambda: route(x, 2, 64, 2)), (moe.MoeError, lambda: route(x, 2, 4, 2, scale=0.0)),
            (moe.MoeError, lambda: route(x, 2, 4, 2, bias=b.half())),
            (moe.MoeError, lambda: route(x, 2, 4, 2, bias=b[:63])),
            (moe.MoeError, lambda: route(x, 2, 4, 2, w=torch.empty(4, 3, device=DEV))),
            (moe.MoeError, lambda: route(x, 2, 4, 2, idx=torch.empty(4, 2, dtype=torch.int32, device=DEV)))]:
        with pytest.raises(error):
            call()
