"""Norm, router, dispatch, 8-bit experts and combine together, as a model runs them: the example's block,
its gradients against float64 autograd, a captured step, and the module-wide promises of the bindings."""
import pytest
import torch

import mixture_experts_routing_moe_gb300 as moe
from examples import mx8_layer

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("tokens,hidden,inter,experts", [(300, 256, 384, 16), (40, 200, 96, 32)])
def test_block(tokens, hidden, inter, experts):
    """e4m3 leaves each activation off by 2^-4 of it at most, twice (the tokens, the experts' inner values);
    a sum of many is not off by more, relatively, in the 2-norm."""
    prompt, few = mx8_layer.run(tokens, hidden, inter, experts, top_k=4, groups=8, selected=4)
    assert prompt < 2 * 2.0 ** -4 and few < 2 * 2.0 ** -4


def test_block_gradients():
    """Against float64 autograd of the same block for the same choice.  16 bits round y, the experts'
    operands and the gradients between the calls: each by 2^-9 of its value or less, some six of them."""
    t = mx8_layer.train()
    w = {k: v.double().requires_grad_() for k, v in t["weights"].items() if k != "bias"}
    x, stream, d = t["x"].double().requires_grad_(), t["stream"].double(), t["d"].double()
    s = (x + stream)
    s16 = s + (s.detach().to(torch.bfloat16).double() - s.detach())         # the stream is kept in 16 bits
    n = s16 * torch.rsqrt((s16 * s16).mean(-1, keepdim=True) + 1e-6) * w["norm"]
    idx = t["idx"].view(torch.int32).long()
    p = torch.softmax(n @ w["router"].T, -1).gather(1, idx)
    p = p / p.sum(-1, keepdim=True)
    out = 0
    for j in range(idx.shape[1]):
        gate, up, down = (w[k][idx[:, j]] for k in ("gate", "up", "down"))
        g, u = (torch.einsum("th,tih->ti", n, m) for m in (gate, up))
        out = out + p[:, j, None] * torch.einsum("ti,thi->th", torch.nn.functional.silu(g) * u, down)
    ((out + s16) * d).sum().backward()

    def near(got, want):
        return float((got.double() - want).norm() / want.norm()) < 6 * 2.0 ** -8

    assert near(t["out"], out.detach()) and near(t["dx"], x.grad) and near(t["dnorm"], w["norm"].grad)
    assert near(t["drouter"], w["router"].grad)
    assert all(near(t["d" + k], w[k].grad) for k in ("gate", "up", "down"))


def test_a_captured_step_with_eager_ones_between():
    """A step of the block as one graph: replays on new inputs give the eager step's bits, and leave the
    eager calls' workspaces alone."""
    weights, normal = mx8_layer.make(256, 384, 16, 3)
    block = mx8_layer.Mx8Block(**weights, top_k=2, groups=4, selected=2)
    x, stream = normal(5, 256), normal(5, 256)
    xs, ss = x.clone(), stream.clone()
    block(xs, ss.clone())
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, s = block(xs, ss)
    for i in range(3):
        x, stream = normal(5, 256), normal(5, 256)
        want, want_stream = block(x, stream.clone())
        block(normal(300, 256), normal(300, 256))
        xs.copy_(x), ss.copy_(stream)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(s, want_stream), i


def test_two_streams_at_once():
    """Calls of different sizes on two streams, in flight together."""
    weights, normal = mx8_layer.make(512, 768, 16, 4)
    block = mx8_layer.Mx8Block(**weights, top_k=2, groups=4, selected=2)
    inputs = [(normal(n, 512), normal(n, 512)) for n in (700, 3, 64)]
    want = [block(x, s.clone())[0] for x, s in inputs]
    streams = [torch.cuda.Stream() for _ in inputs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for (x, s), st in zip(inputs, streams):
            with torch.cuda.stream(st):
                got.append(block(x, s.clone())[0])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_rows_behind_the_last_group_stay():
    """Experts over more rows than the groups have leave the others' output as it was."""
    x = moe.moe_mx8_quantize(torch.randn(10, 64, device=DEV))
    gate, up = (moe.moe_mx8_quantize(torch.randn(2, 96, 64, device=DEV)) for _ in range(2))
    down = moe.moe_mx8_quantize(torch.randn(2, 64, 96, device=DEV))
    y = torch.full((10, 64), 7.0, device=DEV)
    off = torch.tensor([0, 3, 6], dtype=torch.int32, device=DEV)
    moe.moe_mx8_experts_forward_dispatched(x, off, gate, up, down, y=y)
    assert (y[6:] == 7).all() and not (y[:6] == 7).any()
