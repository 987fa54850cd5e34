"""A MoE layer whose expert weights are held in 4-bit blocks, for a prompt and for single tokens.

    python examples/mx4_layer.py [--tokens 2048] [--hidden 2048] [--inter 768] [--experts 64]

The weights are quantised once (moe_mx4_quantize), all but the router's: which experts a token takes
is decided by logits of its 16 bits and the router's, in a prompt as in single tokens.  The prompt's
tokens go through moe_route, moe_dispatch, the experts in blocks and moe_combine; the tokens that
follow, a few at a time, take moe_mx4_forward_tokens, which routes them itself.  Both are compared with
the 16-bit layer on the weights that the blocks stand for (moe_mx4_dequantize), routed in FP32.  A
dense projection in blocks (moe_mx4_product) takes the prompt's result on to a vocabulary.
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import mixture_experts_routing_moe_gb300 as moe  # noqa: E402


class Mx4Layer:
    """Router weights in 16 bits, expert weights and a head [V, H] in blocks."""

    def __init__(self, router, gate, up, down, head, top_k):
        self.router, self.top_k = router, top_k
        self.gate, self.up, self.down = (moe.moe_mx4_quantize(w) for w in (gate, up, down))
        self.head_mx4 = moe.moe_mx4_quantize(head)
        self.ws = None

    def prompt(self, x):
        """x [T, H], any T: expert weights and activations in blocks, routing in FP32."""
        E = self.router.shape[0]
        idx, w = moe.moe_route(x.float() @ self.router.float().T, self.top_k)
        d = moe.moe_dispatch(x, idx, E)
        y = moe.moe_mx4_experts_forward_dispatched(d["x_d"], d["offsets"], self.gate, self.up,
                                                   self.down)
        return moe.moe_combine(y, d["row_of_slot"], w)

    def head(self, out):
        """out [T, H] -> [T, V] in FP32, weights and activations in blocks."""
        return moe.moe_mx4_product(*moe.moe_mx4_quantize(out), *self.head_mx4, dtype=torch.float32)

    def step(self, x):
        """x [T, H] with T <= 64: activations stay in 16 bits, one workspace serves every step."""
        if self.ws is None:
            E, I = self.gate[0].shape[:2]
            need = moe.mx4_tokens_workspace_bytes(64, E, x.shape[1], I, self.top_k, x.dtype)
            self.ws = torch.empty(need, dtype=torch.uint8, device=x.device)
        return moe.moe_mx4_forward_tokens(x, self.router, self.gate, self.up, self.down,
                                          self.top_k, ws=self.ws)


def run(tokens=2048, hidden=2048, inter=768, experts=64, top_k=4, steps=8, seed=0):
    """Relative errors against the 16-bit layer on the same weights, each routing its own tokens: of a
    prompt (or of the head on it, if that is larger), and of single tokens."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).bfloat16()

    router = normal(experts, hidden, std=hidden ** -0.5)
    layer = Mx4Layer(router, normal(experts, inter, hidden, std=hidden ** -0.5),
                     normal(experts, inter, hidden, std=hidden ** -0.5),
                     normal(experts, hidden, inter, std=inter ** -0.5),
                     normal(4 * hidden, hidden, std=hidden ** -0.5), top_k)
    gate, up = (moe.moe_mx4_dequantize(*m, hidden) for m in (layer.gate, layer.up))
    down = moe.moe_mx4_dequantize(*layer.down, inter)

    def error(a, b):
        return float((a.float() - b.float()).norm() / b.float().norm())

    def reference(x):
        return moe.moe_forward(x, x.float() @ router.float().T, gate, up, down, top_k)

    x = normal(tokens, hidden)
    out = layer.prompt(x)
    head = moe.moe_mx4_dequantize(*layer.head_mx4, hidden, torch.float32)
    prompt = max(error(out, reference(x)), error(layer.head(out), out.float() @ head.T))
    single = 0.0
    for n in range(1, steps + 1):
        x = normal(n, hidden)
        single = max(single, error(layer.step(x), reference(x)))
    return prompt, single


def main():
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--inter", type=int, default=768)
    ap.add_argument("--experts", type=int, default=64)
    a = ap.parse_args()
    prompt, single = run(a.tokens, a.hidden, a.inter, a.experts)
    print(f"prompt (activations in 4 bits): relative error {prompt:.3f} against the 16-bit layer")
    print(f"single tokens (activations in 16 bits): {single:.5f}")


if __name__ == "__main__":
    main()
