"""A block of a model around experts held in 8-bit blocks, for a prompt and for single tokens.

    python examples/mx8_layer.py [--tokens 2048] [--hidden 2048] [--inter 768] [--experts 64]

The experts' weights are quantised once (moe_mx8_quantize).  A step adds the last layer's output to the
residual stream and normalises it (moe_rms_norm), which gives the router 16 bits and the experts 8-bit
blocks; experts are chosen among the best groups of them (moe_route_softmax_grouped, with a bias that
balances their load), and moe_mx8_forward takes the tokens through them.  The block is compared with the
same block in 16 bits on the weights that the blocks stand for.  train() runs the 16-bit block with
gradients: the router's weights, the experts and the norm each have their backward call.
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import mixture_experts_routing_moe_gb300 as moe  # noqa: E402


class Mx8Block:
    """Norm and router in 16 bits, expert weights in 8-bit blocks."""

    def __init__(self, norm, router, bias, gate, up, down, top_k, groups, selected):
        self.norm, self.router, self.bias = norm, router, bias
        self.choice = dict(top_k=top_k, groups=groups, selected_groups=selected, bias=bias)
        self.gate, self.up, self.down = (moe.moe_mx8_quantize(w) for w in (gate, up, down))

    def __call__(self, x, stream):
        """x: the last layer's output, stream: the residual stream, both [T, H] -> (this layer's
        output, the stream with x added, in place)."""
        n = moe.moe_rms_norm(x, self.norm, residual=stream, sum=stream, blocks=True)
        idx, w = moe.moe_route_softmax_grouped(n["y"].float() @ self.router.float().T, **self.choice)
        return moe.moe_mx8_forward((n["codes"], n["scales"]), idx, w, self.gate, self.up, self.down,
                                   dtype=x.dtype), stream


def make(hidden, inter, experts, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).bfloat16()

    weights = dict(norm=1 + normal(hidden, std=0.1), router=normal(experts, hidden, std=hidden ** -0.5),
                   bias=torch.randn(experts, generator=g, device="cuda") / experts,
                   gate=normal(experts, inter, hidden, std=hidden ** -0.5),
                   up=normal(experts, inter, hidden, std=hidden ** -0.5),
                   down=normal(experts, hidden, inter, std=inter ** -0.5))
    return weights, normal


def run(tokens=2048, hidden=2048, inter=768, experts=64, top_k=4, groups=8, selected=4, steps=4, seed=0):
    """Relative errors of the block against the 16-bit one: of a prompt, and the largest of single
    tokens and small batches that follow."""
    weights, normal = make(hidden, inter, experts, seed)
    block = Mx8Block(**weights, top_k=top_k, groups=groups, selected=selected)
    gate, up = (moe.moe_mx8_dequantize(*m, hidden) for m in (block.gate, block.up))
    down = moe.moe_mx8_dequantize(*block.down, inter)

    def error(n):
        x, stream = normal(n, hidden), normal(n, hidden)
        y = moe.moe_rms_norm(x, weights["norm"], residual=stream)["y"]
        want = moe.moe_forward_softmax_grouped(y, y.float() @ weights["router"].float().T, gate, up, down,
                                               **block.choice).float()
        got, _ = block(x, stream)
        return float((got.float() - want).norm() / want.norm())

    return error(tokens), max(error(n) for n in range(1, steps + 1))


def train(tokens=512, hidden=256, inter=384, experts=16, top_k=4, groups=4, selected=2, seed=0):
    """One step's gradients of sum(out * d) of the 16-bit block: dict of the inputs' (x and stream
    alike), the norm's, the router's and the experts' gradients, and what they belong to."""
    weights, normal = make(hidden, inter, experts, seed)
    x, stream, d = normal(tokens, hidden), normal(tokens, hidden), normal(tokens, hidden)
    router = weights["router"].float()
    n = moe.moe_rms_norm(x, weights["norm"], residual=stream, stats=True)
    logits = n["y"].float() @ router.T
    idx, w = moe.moe_route_softmax_grouped(logits, top_k, groups, selected, bias=weights["bias"])
    p = moe.moe_dispatch(n["y"], idx, experts)
    experts_w = weights["gate"], weights["up"], weights["down"]
    y = moe.moe_experts_forward_dispatched(p["x_d"], p["offsets"], *experts_w)
    out = moe.moe_combine(y, p["row_of_slot"], w)
    # backward: the output also goes on along the stream, whose gradient is d here
    dy, dw = moe.moe_combine_backward(y, p["row_of_slot"], w, d)
    dx_d, dgate, dup, ddown = moe.moe_experts_backward(p["x_d"], p["offsets"], *experts_w, dy)
    dn = moe.moe_dispatch_backward(dx_d, p["row_of_slot"], tokens, top_k).float()
    dlogits = moe.moe_selected_router_backward(logits, idx, dw, "softmax")
    dn += dlogits @ router
    dx, dnorm = moe.moe_rms_norm_backward(dn.to(x.dtype), n["sum"], weights["norm"], n["rstd"], dsum=d)
    return dict(x=x, stream=stream, d=d, weights=weights, idx=idx, out=out, dx=dx, dnorm=dnorm,
                drouter=dlogits.T @ n["y"].float(), dgate=dgate, dup=dup, ddown=ddown)


def main():
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--inter", type=int, default=768)
    ap.add_argument("--experts", type=int, default=64)
    a = ap.parse_args()
    prompt, few = run(a.tokens, a.hidden, a.inter, a.experts)
    print(f"prompt: relative error {prompt:.4f} against the 16-bit block")
    print(f"single tokens: {few:.4f}")


if __name__ == "__main__":
    main()
