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


@pytest.mark.parametrize("rows", [16, 200])
def test_swiglu_of_the_experts_far_below_zero(rows):
    """silu(g) down to g = -88, where 1 + exp(-g) is the largest that FP32 holds, times a large u."""
    H, I = 64, 64
    x = np.zeros((rows, H))
    x[:, 0], x[:, 1] = -4.0 * (1 + np.arange(rows) % 16), -24.0   # one block: scale 16 or less
    x[:, 32] = 2.0 ** 100                                          # the other
    g_cols = {0: 1.0, 1: 1.0}
    gate, up, down = np.zeros((I, H)), np.zeros((I, H)), np.zeros((H, I))
    for c, v in g_cols.items():
        gate[:, c] = v
    up[:, 32], down[:, 5] = 1.0, 1.0
    w = [tuple(torch.from_numpy(t)[None].to(DEV) for t in M.quantize(m)) for m in (gate, up, down)]
    off = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    y = moe.moe_mx4_experts_forward_dispatched(torch.from_numpy(x).float().to(DEV), off, *w)
    xq = M.fake(x)
    g, u = xq[:, 0] + xq[:, 1], xq[:, 32]
    assert g.min() == -88 and g.max() > -32
    a = M.silu_mul(g, u)
    # no a is near a border between codes, so the products are exact
    assert (M.quantize_slack(np.repeat(a[:, None], 64, 1), 1e-4) == 0).all()
    ref = M.fake(np.repeat(a[:, None], 64, 1))[:, 5]
    assert (y.double().cpu().numpy() == ref[:, None]).all()


def test_swiglu_of_the_experts_to_a_few_units():
    """Four million values of a from exact g and u, g from about -100 to 100: each takes its code, or
    where it is within eight units of FP32 of a border, either code."""
    rng = np.random.default_rng(17)
    n = 2048
    x = rng.standard_normal((n, n)) * np.exp2(rng.uniform(-3, 5, (n, 1)))
    x = torch.from_numpy(np.clip(x, -80, 80)).float()
    weights, sums = [], []
    xq = M.fake(x.double().numpy())
    for _ in range(2):      # three values of x with 2^0, 2^-3 and 2^-6, which FP32 adds up exactly
        w, total = np.zeros((n, n)), 0.0
        for part, shift in zip(np.split(np.arange(1536), 3), (0, 3, 6)):
            at = rng.choice(part, n)
            w[np.arange(n), at] = 2.0 ** -shift
            total = total + xq[:, at] * 2.0 ** -shift
        weights.append(tuple(torch.from_numpy(t)[None].to(DEV) for t in M.quantize(w)))
        sums.append(total)
    off = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    y = moe.moe_mx4_experts_forward_dispatched(x.to(DEV), off, *weights, picks(n, np.arange(n)))
    a = M.silu_mul(*sums)
    err = np.abs(y.double().cpu().numpy() - M.fake(a))
    wrong = err > M.quantize_slack(a, 8 * U)
    assert not wrong.any(), (wrong.sum(), sums[0][wrong][:4])
