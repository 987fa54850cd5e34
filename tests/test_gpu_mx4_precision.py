"""How exactly the microscaled 4-bit products treat what is not in 4 bits: activations of the few-token
layer, the SwiGLU between the experts' products.

Weights have one code in a row, so that a result is one product or one SwiGLU value and its error is
that of the parts alone.
"""
import numpy as np
import pytest
import torch

import mixture_experts_routing_moe_gb300 as moe
from oracle import mx4_oracle as M

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -23  # a unit of FP32 arithmetic, twice its half step


def picks(rows, cols, value=1.0):
    """[len(cols), rows] weights whose row i is `value` in column cols[i]: codes, scales on the GPU."""
    w = np.zeros((len(cols), rows))
    w[np.arange(len(cols)), cols] = value
    c, s = M.quantize(w)
    return torch.from_numpy(c)[None].to(DEV), torch.from_numpy(s)[None].to(DEV)


def tops(v):
    return np.repeat(np.abs(v).reshape(-1, 32).max(-1), 32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", [1, 5, 30])
@pytest.mark.parametrize("ratio", [64, 1024])
def test_values_beside_a_large_one_keep_their_16_bits(dtype, T, ratio):
    """Each block of x has one value `ratio` times as large as the rest, which the weights of most rows
    leave out; so has each block of a.  The rest counts with no more error than its own rounding to
    16 bits, beside FP32 arithmetic."""
    rng = np.random.default_rng(T * 7 + ratio)
    H, I = 256, 384
    x = rng.uniform(0.5, 1.0, (T, H)) * rng.choice([-1.0, 1.0], (T, H))
    big = np.arange(0, H, 32) + rng.integers(0, 32, H // 32)
    x[:, big] *= ratio
    small = np.setdiff1d(np.arange(H), big)
    xs = torch.from_numpy(x).to(dtype)
    gate_at, up_at = rng.choice(small, I), rng.choice(small, I)
    wide = np.arange(0, I, 32) + rng.integers(0, 32, I // 32)
    up_at[wide] = rng.choice(big, I // 32)        # a of these rows is the large one of its block
    down_at = rng.integers(0, I, H)
    w = [picks(H, gate_at), picks(H, up_at), picks(I, down_at)]
    router = torch.zeros(1, H, dtype=dtype, device=DEV)
    out = moe.moe_mx4_forward_tokens(xs.to(DEV), router, *w, top_k=1)
    got, eps = out.double().cpu().numpy(), torch.finfo(dtype).eps
    for t in range(T):
        v = xs[t].double().numpy()
        dv = U * tops(v)                          # what the terms leave of x
        g, u = v[gate_at], v[up_at]
        a = M.silu_mul(g, u)
        # terms add up in FP32, then exp, an addition, a division and two products; |silu'| < 1.1
        dg, du = dv[gate_at] + 16 * U * np.abs(g), dv[up_at] + 16 * U * np.abs(u)
        da = 1.1 * dg * np.abs(u) + np.abs(M.silu_mul(g, 1.0)) * du + 1.1 * dg * du + 16 * U * np.abs(a)
        ar = np.abs(a) + da
        da = da + eps / 2 * ar                    # rounded to 16 bits
        dy = da + U * tops(ar) + 16 * U * ar      # the terms of a, their sum
        ref = a[down_at]
        tol = dy[down_at] * (1 + eps) + eps / 2 * np.abs(ref)
        assert (np.abs(got[t] - ref) <= tol).all(), np.max(np.abs(got[t] - ref) / tol)
        # the bound above is that of 16 bits: no looser than two roundings and a little
        few = ~np.isin(down_at, wide)
        assert (tol[few] <= (2 * eps + 4e-3 * (ratio > 64)) * np.abs(ref[few])).all()
