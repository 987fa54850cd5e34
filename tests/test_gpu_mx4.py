"""Microscaled 4-bit quantisation, product and experts on the GPU against the float64 oracle.

Tolerances.  Quantised bytes and decoded values are exact.  A product's FP32 sums of exact terms
are held to (K + 64) 2^-23 times the sum of the terms' magnitudes (each of at most K + 64 additions
off by one unit), plus half a step of the output type, eps / 2 relative to the value.
"""
import numpy as np
import pytest
import torch

import mixture_experts_routing_moe_gb300 as moe
from mixture_experts_routing_moe_gb300 import binding as B
from oracle import mx4_oracle as M

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [torch.float32, torch.float16, torch.bfloat16]


def rows_of(rows, K, dtype, seed, spread=8):
    """Normal rows whose magnitudes differ by up to 2^spread, with values on code borders."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, K)) * np.exp2(rng.integers(-spread, spread + 1, (rows, 1)))
    x[:, ::5] = np.round(x[:, ::5] * 4) / 4
    return torch.from_numpy(x).to(dtype)


def np64(t):
    return t.double().cpu().numpy()


def blocks(x):
    """(codes, scales) of a float64 array, on the GPU and as bytes."""
    c, s = M.quantize(x)
    return torch.from_numpy(c).to(DEV), torch.from_numpy(s).to(DEV), c, s


def half_step(dtype, ref):
    return torch.finfo(dtype).eps / 2 * np.abs(ref) + torch.finfo(dtype).tiny


def check_within(got, ref, tol, dtype):
    """|got - ref| <= tol; a value that may round past the type's largest may be that infinity."""
    over = (np.abs(ref) + tol >= torch.finfo(dtype).max) & (got == np.copysign(np.inf, ref))
    with np.errstate(invalid="ignore"):
        err = np.where(over, 0.0, np.abs(got - ref))
    assert (err <= tol).all(), (np.nanmax(err), np.argwhere(~(err <= tol))[:4])


# ------------------------------------------------------------------------------ quantisation
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,K", [(1, 1), (1, 31), (3, 32), (5, 33), (2, 127), (7, 128), (4, 130),
                                    (33, 256), (9, 1357), (2, 5000), (300, 96), (1, 8192)])
def test_quantize_bytes(dtype, rows, K):
    x = rows_of(rows, K, dtype, rows * 10007 + K)
    codes, scales = moe.moe_mx4_quantize(x.to(DEV))
    c, s = M.quantize(np64(x))
    assert (codes.cpu().numpy() == c).all() and (scales.cpu().numpy() == s).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad", [1, 8])
def test_quantize_strided_rows(dtype, pad):
    x = rows_of(40, 200 + pad, dtype, 3).to(DEV)
    codes, scales = moe.moe_mx4_quantize(x[:, :200])
    c, s = M.quantize(np64(x)[:, :200])
    assert (codes.cpu().numpy() == c).all() and (scales.cpu().numpy() == s).all()
    v = torch.full((40, 200 + pad), 7.0, dtype=dtype, device=DEV)
    moe.moe_mx4_dequantize(codes, scales, 200, out=v[:, :200])
    assert (v[:, 200:] == 7).all()
    assert torch.equal(v[:, :200].cpu(), torch.from_numpy(M.values(c, s, 200)).to(dtype))


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_special_values(dtype):
    x = torch.zeros(8, 96, dtype=dtype)
    tiny = torch.finfo(dtype).smallest_normal
    x[0, 3] = float("nan")
    x[1, 40], x[1, 41] = float("inf"), 1.0
    x[2, 95], x[2, 0] = float("-inf"), -3.0
    x[3, :] = -0.0
    x[4, :32] = tiny / 8                              # subnormals
    x[4, 32:64] = torch.finfo(dtype).max
    x[5, 64:] = torch.linspace(-8, 8, 32).to(dtype)
    x[6, 0], x[6, 1] = 7.96875, 4.5
    x[7, ::2] = 1e-7
    codes, scales = moe.moe_mx4_quantize(x.to(DEV))
    c, s = M.quantize(np64(x))
    assert (codes.cpu().numpy() == c).all() and (scales.cpu().numpy() == s).all()
    v = np64(moe.moe_mx4_dequantize(codes, scales, 96, torch.float32))
    ref = M.values(c, s, 96)
    assert (np.isnan(v) == np.isnan(ref)).all() and (v[~np.isnan(v)] == ref[~np.isnan(v)]).all()


def test_quantize_subnormal_and_largest_scales():
    x = torch.zeros(3, 32)
    x[0, :4] = torch.tensor([2.0 ** -126, 2.0 ** -128, 2.0 ** -130, 2.0 ** -149])
    x[1, :3] = torch.tensor([3.4e38, -1e38, 1e30])
    x[2, 0] = 2.0 ** -140
    codes, scales = moe.moe_mx4_quantize(x.to(DEV))
    c, s = M.quantize(np64(x))
    assert (codes.cpu().numpy() == c).all() and (scales.cpu().numpy() == s).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_dequantize_every_code_and_scale(dtype):
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1)            # 512 values = 16 blocks
    scales = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 16)
    v = moe.moe_mx4_dequantize(codes.to(DEV), scales.to(DEV), 512, dtype).cpu()
    ref = torch.from_numpy(M.values(codes.numpy(), scales.numpy())).to(dtype)
    assert (torch.isnan(v) == torch.isnan(ref)).all()
    ok = ~torch.isnan(ref)
    assert torch.equal(v[ok], ref[ok])


def test_quantize_weights_and_empty():
    x = rows_of(6, 64, torch.bfloat16, 1).view(2, 3, 64)
    codes, scales = moe.moe_mx4_quantize(x.to(DEV))
    assert codes.shape == (2, 3, 32) and scales.shape == (2, 3, 4)
    c, s = M.quantize(np64(x))
    assert (codes.cpu().numpy() == c).all() and (scales.cpu().numpy() == s).all()
    codes, scales = moe.moe_mx4_quantize(torch.empty(0, 64, device=DEV))
    assert codes.shape == (0, 32)
    assert moe.moe_mx4_dequantize(codes, scales, 64).shape == (0, 64)


# ------------------------------------------------------------------------------------ product
def offsets_of(sizes):
    o = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    return torch.from_numpy(o).to(DEV), o


def check_product(sizes, N, K, dtype, seed, extra_rows=0):
    rng = np.random.default_rng(seed)
    E, rows = len(sizes), int(sum(sizes)) + extra_rows
    A = rng.standard_normal((rows, K)) * np.exp2(rng.integers(-6, 7, (rows, 1)))
    W = rng.standard_normal((E, N, K)) * np.exp2(rng.integers(-6, 7, (E, N, 1)))
    ac, asc, c, s = blocks(A)
    bc, bsc, wc, ws_ = blocks(W)
    a, w = M.values(c, s, K), M.values(wc, ws_, K)
    off, o = offsets_of(sizes)
    out = torch.full((rows, N), 42.0, dtype=dtype, device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    moe.moe_mx4_product(ac, asc, bc, bsc, offsets=off, out=out, ws=ws)
    assert moe.moe_device_status(ws) == 0
    got = np64(out)
    for e in range(E):
        g, x = got[o[e]:o[e + 1]], a[o[e]:o[e + 1]]
        ref, mag = x @ w[e].T, np.abs(x) @ np.abs(w[e]).T
        tol = (K + 64) * 2.0 ** -23 * mag + half_step(dtype, ref)
        check_within(g, ref, tol, dtype)
    assert (got[o[-1]:] == 42).all()          # rows past the groups are not written


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("sizes,N,K", [
    ([1], 1, 32), ([1], 256, 256), ([128], 256, 512), ([130], 300, 96), ([3, 0, 5], 33, 64),
    ([0, 0, 7], 129, 224), ([127, 1, 129, 64], 384, 1024), ([400], 511, 2080), ([5] * 40, 72, 288),
    ([257, 31], 520, 4096)])
def test_product(dtype, sizes, N, K):
    check_product(sizes, N, K, dtype, sum(sizes) * 31 + N + K)


def test_product_rows_past_the_groups():
    check_product([9, 4], 64, 128, torch.float32, 5, extra_rows=6)
    check_product([0, 0], 64, 128, torch.bfloat16, 6, extra_rows=3)


def test_product_many_tiles_in_flight():
    check_product([700, 3, 0, 900, 1300], 1160, 416, torch.bfloat16, 8)


def test_product_one_group_without_offsets():
    rng = np.random.default_rng(3)
    ac, asc, c, s = blocks(rng.standard_normal((37, 160)))
    bc, bsc, wc, wsc = blocks(rng.standard_normal((50, 160)))
    out = moe.moe_mx4_product(ac, asc, bc, bsc, dtype=torch.float32)
    a, w = M.values(c, s), M.values(wc, wsc)
    assert (np.abs(np64(out) - a @ w.T) <= 300 * 2.0 ** -23 * (np.abs(a) @ np.abs(w).T)).all()


def test_product_extreme_scales():
    """Scale bytes from both ends of the range meet in one product."""
    K = 64
    A, W = np.ones((4, K)), np.ones((8, K))
    ac, asc, *_ = blocks(A)
    bc, bsc, *_ = blocks(W)
    asc[:, :2], bsc[:, :2] = 252, 0           # ones are codes of 4 with byte 125
    out = np64(moe.moe_mx4_product(ac, asc, bc, bsc, dtype=torch.float32))
    assert (out == 64 * 16 * 2.0 ** (252 - 127) * 2.0 ** -127).all()


def test_product_nan_block_stays_in_its_rows():
    rng = np.random.default_rng(4)
    A, W = rng.standard_normal((140, 320)), rng.standard_normal((70, 320))
    A[133, 300], W[60, 7] = np.nan, np.inf
    ac, asc, *_ = blocks(A)
    bc, bsc, *_ = blocks(W)
    out = np64(moe.moe_mx4_product(ac, asc, bc, bsc))
    bad = np.zeros((140, 70), bool)
    bad[133], bad[:, 60] = True, True
    assert (np.isnan(out) == bad).all()


def test_product_bad_offsets_stay_in_bounds():
    """Offsets that decrease or pass the rows are cut to [0, rows]; nothing outside is touched."""
    rng = np.random.default_rng(5)
    ac, asc, c, s = blocks(rng.standard_normal((20, 64)))
    bc, bsc, wc, wsc = blocks(rng.standard_normal((3, 16, 64)))
    off = torch.tensor([0, 12, 6, 900], dtype=torch.int32, device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    out = moe.moe_mx4_product(ac, asc, bc, bsc, offsets=off, dtype=torch.float32, ws=ws)
    assert moe.moe_device_status(ws) == 0
    a, w = M.values(c, s), M.values(wc, wsc)
    got = np64(out)
    assert np.allclose(got[:6], a[:6] @ w[0].T, rtol=1e-5, atol=1e-4)
    assert np.allclose(got[12:], a[12:] @ w[2].T, rtol=1e-5, atol=1e-4)


def test_product_on_another_stream_and_in_a_graph():
    rng = np.random.default_rng(6)
    ac, asc, c, s = blocks(rng.standard_normal((64, 256)))
    bc, bsc, wc, wsc = blocks(rng.standard_normal((128, 256)))
    want = moe.moe_mx4_product(ac, asc, bc, bsc)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = moe.moe_mx4_product(ac, asc, bc, bsc, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out, ws = torch.empty_like(want), torch.empty(256, dtype=torch.uint8, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_mx4_product(ac, asc, bc, bsc, out=out, ws=ws)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


# ------------------------------------------------------------------------------------ experts
def check_experts(sizes, H, I, dtype, seed):
    rng = np.random.default_rng(seed)
    E, rows = len(sizes), int(sum(sizes))
    x = torch.from_numpy(rng.standard_normal((rows, H))).to(dtype)
    gate, up = (rng.standard_normal((E, I, H)) / np.sqrt(H) for _ in range(2))
    down = rng.standard_normal((E, H, I)) / np.sqrt(I)
    packed = [blocks(m) for m in (gate, up, down)]
    w = [M.values(p[2], p[3]) for p in packed]
    off, o = offsets_of(sizes)
    ws = torch.empty(moe.mx4_experts_workspace_bytes(rows, H, I), dtype=torch.uint8, device=DEV)
    y = moe.moe_mx4_experts_forward_dispatched(x.to(DEV), off, *[p[:2] for p in packed], ws=ws)
    assert moe.moe_device_status(ws) == 0 and y.dtype == dtype
    got, xq = np64(y), M.fake(np64(x))
    for e in range(E):
        r = slice(o[e], o[e + 1])
        if not sizes[e]:
            continue
        g, u = xq[r] @ w[0][e][:, :H].T, xq[r] @ w[1][e][:, :H].T
        # FP32 sums of g and u, then exp, a division and two products (a few 2^-23 each)
        dg = (H + 64) * 2.0 ** -23 * (np.abs(xq[r]) @ np.abs(w[0][e][:, :H]).T)
        du = (H + 64) * 2.0 ** -23 * (np.abs(xq[r]) @ np.abs(w[1][e][:, :H]).T)
        a = M.silu_mul(g, u)
        da = 1.1 * dg * np.abs(u) + np.abs(M.silu_mul(g, 1.0)) * du + 1.1 * dg * du
        rel = (da / np.maximum(np.abs(a), 1e-30) + 16 * 2.0 ** -23)
        slack, low = np.zeros_like(a), 0.0
        for lim in (1e-5, 1e-4, 1e-3, 1e-2, 1.0):     # the slack that each value's error reaches
            slack = np.where((rel > low) & (rel <= lim), M.quantize_slack(a, lim), slack)
            low = lim
        # where a is all but zero against its block its code is 0 whatever its relative error
        top = np.abs(np.pad(a, ((0, 0), (0, -I % 32)))).reshape(len(a), -1, 32).max(-1).repeat(32, -1)[:, :I]
        slack = np.where((np.abs(a) + da) < top / 32, 0.0, slack)
        aq = M.fake(a)
        ref = aq @ w[2][e][:, :I].T
        mag = np.abs(aq) @ np.abs(w[2][e][:, :I]).T
        tol = (I + 64) * 2.0 ** -23 * mag + slack @ np.abs(w[2][e][:, :I]).T
        tol = tol * (1 + torch.finfo(dtype).eps) + half_step(dtype, ref)
        check_within(got[r], ref, tol, dtype)
        assert np.linalg.norm(got[r] - ref) <= (torch.finfo(dtype).eps + 5e-3) * np.linalg.norm(ref)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("sizes,H,I", [([1], 32, 32), ([2, 0, 5], 64, 160), ([130, 3], 256, 72),
                                       ([40, 0, 300], 200, 416), ([64, 200], 512, 768)])
def test_experts(dtype, sizes, H, I):
    check_experts(sizes, H, I, dtype, sum(sizes) + H + I)


def test_experts_nan_row_and_empty():
    rng = np.random.default_rng(9)
    x = torch.from_numpy(rng.standard_normal((6, 64))).to(torch.bfloat16)
    x[2, 5] = float("nan")
    packed = [blocks(rng.standard_normal(s))[:2] for s in ((2, 96, 64), (2, 96, 64), (2, 64, 96))]
    off, _ = offsets_of([4, 2])
    y = np64(moe.moe_mx4_experts_forward_dispatched(x.to(DEV), off, *packed))
    assert np.isnan(y[2]).all() and np.isfinite(np.delete(y, 2, 0)).all()
    off0, _ = offsets_of([0, 0])
    y = moe.moe_mx4_experts_forward_dispatched(x[:0].to(DEV), off0, *packed)
    assert y.shape == (0, 64)


# ------------------------------------------------------------------------------------- tokens
def layer(T, E, H, I, dtype, seed):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((T, H))).to(dtype)
    router = torch.from_numpy(rng.standard_normal((E, H)) / np.sqrt(H)).to(dtype)
    shapes = ((E, I, H), (E, I, H), (E, H, I))
    packed = [blocks(rng.standard_normal(s) / np.sqrt(s[2])) for s in shapes]
    return x, router, packed


def tokens_reference(x, router, packed, idx, w):
    """(out, tolerance without the last rounding) for a given selection and its weights."""
    dtype = x.dtype
    eps = torch.finfo(dtype).eps
    xs, wt = np64(x), [M.values(p[2], p[3]) for p in packed]
    T, H, I = xs.shape[0], xs.shape[1], wt[0].shape[1]
    out, tol = np.zeros((T, H)), np.zeros((T, H))
    u, term = 2.0 ** -23, 2.0 ** -14
    for t in range(T):
        for j, e in enumerate(idx[t]):
            gate, up, down = (m[e] for m in wt)
            g, v = gate @ xs[t], up @ xs[t]
            # sums of 5 K products (the terms of x) in FP32, and terms that together are within
            # 2^-14 of their block's largest value: a value scaled to at most 4 is within 1/2 of a
            # code, five terms eight times apart leave 2^-13, and the largest is at least 2
            top = np.repeat(np.abs(xs[t]).reshape(-1, 32).max(-1), 32)
            mag_g = (5 * H + 64) * u * (np.abs(gate) @ np.abs(xs[t])) + term * (np.abs(gate) @ top)
            mag_v = (5 * H + 64) * u * (np.abs(up) @ np.abs(xs[t])) + term * (np.abs(up) @ top)
            a = M.silu_mul(g, v)
            da = 1.1 * mag_g * np.abs(v) + np.abs(M.silu_mul(g, 1.0)) * mag_v + 1.1 * mag_g * mag_v
            da += eps / 2 * (np.abs(a) + da) + torch.finfo(dtype).tiny   # rounded to the type
            ar = torch.from_numpy(a).to(dtype).double().numpy()
            y = down @ a
            top = np.repeat(np.abs(ar).reshape(-1, 32).max(-1), 32)
            dy = np.abs(down) @ (da + term * top) + (5 * I + 64) * u * (np.abs(down) @ np.abs(a))
            out[t] += w[t, j] * y
            tol[t] += w[t, j] * (dy + 64 * u * np.abs(y))
    return out, tol


def check_tokens(T, E, H, I, k, dtype, renorm, seed):
    x, router, packed = layer(T, E, H, I, dtype, seed)
    ws = torch.empty(moe.mx4_tokens_workspace_bytes(T, E, H, I, k, dtype), dtype=torch.uint8,
                     device=DEV)
    idx = torch.empty(T, k, dtype=torch.uint32, device=DEV)
    w = torch.empty(T, k, dtype=torch.float32, device=DEV)
    out = moe.moe_mx4_forward_tokens(x.to(DEV), router.to(DEV), *[p[:2] for p in packed], top_k=k,
                                     renormalize=renorm, idx=idx, w=w, ws=ws)
    assert moe.moe_device_status(ws) == 0 and out.dtype == dtype
    # selection: descending logits, none left out that is larger by more than the sums' error
    logits = np64(x) @ np64(router).T
    err = (H + 64) * 2.0 ** -23 * (np.abs(np64(x)) @ np.abs(np64(router)).T)
    got = idx.view(torch.int32).cpu().numpy()
    for t in range(T):
        l, d = logits[t][got[t]], err[t].max()
        assert len(set(got[t])) == k and (np.diff(l) <= 2 * d).all()
        rest = np.delete(logits[t], got[t])
        assert not len(rest) or rest.max() <= l[-1] + 2 * d
    p = np.exp(logits - logits.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    ref_w = np.take_along_axis(p, got, 1)
    if renorm:
        ref_w /= ref_w.sum(-1, keepdims=True)
    gw = np64(w)
    # a logit off by err moves a weight by that factor; the rest is a few FP32 roundings
    assert (np.abs(gw - ref_w) <= ref_w * (4 * err.max() + 64 * 2.0 ** -23)).all()
    ref, tol = tokens_reference(x, router, packed, got, gw)
    check_within(np64(out), ref, tol * (1 + torch.finfo(dtype).eps) + half_step(dtype, ref), dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,E,H,I,k,renorm", [
    (1, 1, 128, 128, 1, True), (1, 8, 256, 384, 2, True), (3, 5, 640, 128, 5, False),
    (8, 16, 512, 256, 4, True), (9, 33, 128, 640, 3, False), (33, 2, 256, 128, 2, True),
    (64, 6, 384, 256, 2, True), (64, 64, 128, 128, 16, True), (17, 200, 256, 128, 8, True),
    (5, 1024, 128, 128, 32, False), (40, 1, 1152, 1280, 1, True),
    (64, 1, 256, 384, 1, True), (39, 3, 128, 2176, 2, True), (38, 2, 640, 1152, 1, False)])
def test_tokens(dtype, T, E, H, I, k, renorm):
    check_tokens(T, E, H, I, k, dtype, renorm, T * 1000 + E + H + I)


def test_tokens_repeats_and_other_streams():
    """The same bits every time, on any stream, after another layer has used the workspace, and
    from a captured graph."""
    x, router, packed = layer(12, 16, 512, 384, torch.bfloat16, 3)
    args = [x.to(DEV), router.to(DEV)] + [p[:2] for p in packed]
    ws = torch.empty(moe.mx4_tokens_workspace_bytes(64, 16, 512, 384, 8, torch.bfloat16),
                     dtype=torch.uint8, device=DEV)
    want = moe.moe_mx4_forward_tokens(*args, top_k=4, ws=ws)
    moe.moe_mx4_forward_tokens(*args, top_k=8, ws=ws)
    for _ in range(20):
        assert torch.equal(moe.moe_mx4_forward_tokens(*args, top_k=4, ws=ws), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = moe.moe_mx4_forward_tokens(*args, top_k=4, ws=ws, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_mx4_forward_tokens(*args, top_k=4, ws=ws, out=out)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_tokens_wide_range_of_values(dtype):
    """Activations whose blocks span the type's range keep their 16 bits (no overflow in terms)."""
    x, router, packed = layer(4, 4, 256, 256, dtype, 7)
    rng = np.random.default_rng(8)
    scale = np.exp2(rng.integers(-8, 9, (4, 8, 1)))
    xs = torch.from_numpy(np64(x).reshape(4, 8, 32) * scale).reshape(4, 256).to(dtype)
    xs[0, :32] = 0
    xs[1, 5] = torch.finfo(dtype).smallest_normal
    idx = torch.empty(4, 2, dtype=torch.uint32, device=DEV)
    w = torch.empty(4, 2, dtype=torch.float32, device=DEV)
    out = moe.moe_mx4_forward_tokens(xs.to(DEV), (router / 64).to(DEV), *[p[:2] for p in packed],
                                     top_k=2, idx=idx, w=w)
    ref, tol = tokens_reference(xs, router, packed, idx.view(torch.int32).cpu().numpy(), np64(w))
    check_within(np64(out), ref, tol * (1 + torch.finfo(dtype).eps) + half_step(dtype, ref), dtype)


def test_tokens_ties_and_bad_rows():
    x, router, packed = layer(6, 8, 128, 128, torch.bfloat16, 11)
    router[:] = router[0]                                   # every logit equal: lowest ids
    x[2, 7], x[4, 100] = float("nan"), float("inf")
    idx = torch.empty(6, 3, dtype=torch.uint32, device=DEV)
    w = torch.empty(6, 3, dtype=torch.float32, device=DEV)
    out = moe.moe_mx4_forward_tokens(x.to(DEV), router.to(DEV), *[p[:2] for p in packed], top_k=3,
                                     idx=idx, w=w)
    assert (idx.view(torch.int32).cpu().numpy() == [0, 1, 2]).all()
    bad = np.array([False, False, True, False, True, False])
    assert (np.isnan(np64(w)).all(-1) == bad).all()
    assert (np.isnan(np64(out)).all(-1) == bad).all() and np.isfinite(np64(out)[~bad]).all()
    assert np.allclose(np64(w)[~bad], 1 / 3, atol=1e-6)


def test_experts_on_another_stream_keep_their_workspace():
    """A call on a side stream: the workspace it made for itself is not handed out again while that
    stream still works (the current stream allocates and overwrites as much right after)."""
    rng = np.random.default_rng(21)
    E, H, I, rows = 4, 512, 768, 2048
    x = torch.from_numpy(rng.standard_normal((rows, H))).to(torch.bfloat16).to(DEV)
    packed = [blocks(rng.standard_normal(s))[:2] for s in ((E, I, H), (E, I, H), (E, H, I))]
    off, _ = offsets_of([rows // E] * E)
    want = moe.moe_mx4_experts_forward_dispatched(x, off, *packed)
    side = torch.cuda.Stream()
    for _ in range(5):
        side.wait_stream(torch.cuda.current_stream())
        got = moe.moe_mx4_experts_forward_dispatched(x, off, *packed, stream=side)
        for _ in range(4):
            torch.empty(moe.mx4_experts_workspace_bytes(rows, H, I), dtype=torch.uint8,
                        device=DEV).fill_(255)
        side.synchronize()
        assert torch.equal(got, want)


def test_graph_and_eager_calls_do_not_share_a_workspace():
    """A captured call has a workspace of its own: its replays leave the one that the stream's eager
    calls keep as it is."""
    x, router, packed = layer(8, 16, 512, 384, torch.bfloat16, 31)
    args = [x.to(DEV), router.to(DEV)] + [p[:2] for p in packed]
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        want = moe.moe_mx4_forward_tokens(*args, top_k=4)
        kept = B._mx4_kept[(torch.cuda.current_device(), s.cuda_stream)]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out = moe.moe_mx4_forward_tokens(*args, top_k=4)
        kept.fill_(0xAA)
        g.replay()
        s.synchronize()
    assert torch.equal(out, want) and (kept == 0xAA).all()
    with torch.cuda.stream(s):
        assert torch.equal(moe.moe_mx4_forward_tokens(*args, top_k=4), want)


def test_tokens_none():
    _, router, packed = layer(1, 4, 128, 128, torch.bfloat16, 2)
    out = moe.moe_mx4_forward_tokens(torch.empty(0, 128, dtype=torch.bfloat16, device=DEV),
                                     router.to(DEV), *[p[:2] for p in packed], top_k=2)
    assert out.shape == (0, 128)


# -------------------------------------------------------------------- other layouts and sizes
def shifted(t, by):
    """A contiguous copy of t that starts `by` bytes after a 256-byte boundary."""
    flat = torch.empty(t.numel() + 256, dtype=torch.uint8, device=DEV)
    view = flat[by:by + t.numel()].view(t.shape)
    view.copy_(t)
    return view


@pytest.mark.parametrize("K", [512, 1024, 2048])
def test_product_scales_on_any_word(K):
    """Scale rows of 16 and 32 bytes whose base is a multiple of 4 or 16 only."""
    rng = np.random.default_rng(K)
    ac, asc, c, s = blocks(rng.standard_normal((200, K)))
    bc, bsc, wc, wsc = blocks(rng.standard_normal((300, K)))
    want = moe.moe_mx4_product(ac, asc, bc, bsc, dtype=torch.float32)
    a, w = M.values(c, s), M.values(wc, wsc)
    assert (np.abs(np64(want) - a @ w.T) <= (K + 64) * 2.0 ** -23 * (np.abs(a) @ np.abs(w).T)).all()
    for by in (4, 16):
        got = moe.moe_mx4_product(shifted(ac, 16), shifted(asc, by), bc, shifted(bsc, by),
                                  dtype=torch.float32)
        assert torch.equal(got, want)


def test_tokens_scales_on_any_word():
    x, router, packed = layer(6, 8, 512, 1024, torch.bfloat16, 5)
    args = [x.to(DEV), router.to(DEV)]
    want = moe.moe_mx4_forward_tokens(*args, *[p[:2] for p in packed], top_k=3)
    for by in (4, 16):
        moved = [(shifted(p[0], 16), shifted(p[1], by)) for p in packed]
        assert torch.equal(moe.moe_mx4_forward_tokens(*args, *moved, top_k=3), want)


def test_outputs_on_any_element():
    """out of 16-bit elements that starts on an odd element: no vector stores."""
    x, router, packed = layer(5, 4, 256, 128, torch.float16, 6)
    args = [x.to(DEV), router.to(DEV)] + [p[:2] for p in packed]
    want = moe.moe_mx4_forward_tokens(*args, top_k=2)
    out = torch.zeros(5 * 256 + 1, dtype=torch.float16, device=DEV)[1:].view(5, 256)
    assert torch.equal(moe.moe_mx4_forward_tokens(*args, top_k=2, out=out), want)
    c, s = moe.moe_mx4_quantize(x.to(DEV))
    want = moe.moe_mx4_product(c, s, c, s, dtype=torch.float16)
    out = torch.zeros(26, dtype=torch.float16, device=DEV)[1:].view(5, 5)
    assert torch.equal(moe.moe_mx4_product(c, s, c, s, out=out), want)


def test_quantize_past_32_bits():
    """More than 2^31 values: the last rows land where they belong."""
    rows, K = (1 << 18) + 9, 8192
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device=DEV)
    tail = rows_of(9, K, torch.bfloat16, 77)
    x[-9:] = tail.to(DEV)
    codes, scales = moe.moe_mx4_quantize(x)
    c, s = M.quantize(np64(tail))
    assert (codes[-9:].cpu().numpy() == c).all() and (scales[-9:].cpu().numpy() == s).all()
    assert not codes[:-9].any() and not scales[:-9].any()
    v = moe.moe_mx4_dequantize(codes, scales, K, out=x)
    assert torch.equal(v[-9:].cpu(), torch.from_numpy(M.values(c, s)).to(torch.bfloat16))


def test_product_past_32_bits():
    """An output of more than 2^31 values."""
    rng = np.random.default_rng(12)
    N, rows = 8192, (1 << 18) + 5
    bc, bsc, wc, wsc = blocks(rng.standard_normal((N, 64)))
    ac, asc, c, s = blocks(rng.standard_normal((261, 64)))
    a_codes = torch.zeros(rows, 32, dtype=torch.uint8, device=DEV)
    a_scales = torch.zeros(rows, 4, dtype=torch.uint8, device=DEV)
    a_codes[-261:], a_scales[-261:] = ac, asc
    out = moe.moe_mx4_product(a_codes, a_scales, bc, bsc)
    ref = M.values(c, s) @ M.values(wc, wsc).T
    mag = np.abs(M.values(c, s)) @ np.abs(M.values(wc, wsc)).T
    got = np64(out[-261:])
    assert (np.abs(got - ref) <= 128 * 2.0 ** -23 * mag + half_step(torch.bfloat16, ref)).all()
    assert not out[:-261].any()


def test_layer_example():
    """The example's two paths against the 16-bit layer on the decoded weights.  Four-bit activations
    leave each value off by up to an eighth of it, which a sum of many does not enlarge; 16-bit ones
    leave the rounding of a and of the output."""
    from examples import mx4_layer
    prompt, single = mx4_layer.run(tokens=300, hidden=256, inter=384, experts=8, top_k=2, steps=4)
    assert prompt < 0.3 and single < 4 * 2.0 ** -8


# ----------------------------------------------------------------------------------- refusals
def test_refusals():
    x = torch.zeros(4, 64, device=DEV)
    c, s = moe.moe_mx4_quantize(x)
    with pytest.raises(ValueError):
        moe.moe_mx4_quantize(x.t())
    with pytest.raises(ValueError):
        moe.moe_mx4_quantize(x.cpu())
    with pytest.raises(moe.MoeError):
        moe.moe_mx4_quantize(x.double())
    with pytest.raises(moe.MoeError):
        moe.moe_mx4_dequantize(c, s, 96)
    with pytest.raises(moe.MoeError):
        moe.moe_mx4_dequantize(c, s[:3], 64)
    with pytest.raises(moe.MoeError):
        moe.moe_mx4_dequantize(c.to(torch.int32), s, 64)
    with pytest.raises(moe.MoeError):
        moe.moe_mx4_dequantize(c, s, 64, torch.float64)
    with pytest.raises(moe.MoeError):
        moe.moe_mx4_product(c, s, *moe.moe_mx4_quantize(torch.zeros(3, 96, device=DEV)))
    w = moe.moe_mx4_quantize(torch.zeros(2, 3, 64, device=DEV))
    with pytest.raises(moe.MoeError):
        moe.moe_mx4_product(c, s, *w)                         # two groups need offsets
    with pytest.raises(moe.MoeError):
        moe.moe_mx4_product(c, s, *w, offsets=torch.zeros(3, dtype=torch.int64, device=DEV))
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV)
    with pytest.raises(moe.MoeError):                         # down of another shape
        moe.moe_mx4_experts_forward_dispatched(x, off, w, w, w)
    with pytest.raises(moe.MoeError):
        moe.moe_mx4_product(c, s, *w, offsets=off, ws=torch.empty(64, dtype=torch.uint8, device=DEV))


def test_tokens_refusals():
    x, router, packed = layer(2, 4, 128, 128, torch.bfloat16, 2)
    x, router, ws = x.to(DEV), router.to(DEV), [p[:2] for p in packed]
    for bad in (dict(top_k=5), dict(top_k=0), dict(top_k=2, idx=torch.zeros(2, 2, device=DEV)),
                dict(top_k=2, ws=torch.empty(256, dtype=torch.uint8, device=DEV))):
        with pytest.raises(moe.MoeError):
            moe.moe_mx4_forward_tokens(x, router, *ws, **bad)
    with pytest.raises(moe.MoeError):
        moe.moe_mx4_forward_tokens(x, router.half(), *ws, top_k=2)
    with pytest.raises(moe.MoeError):
        moe.moe_mx4_forward_tokens(x.float(), router.float(), *ws, top_k=2)
    with pytest.raises(moe.MoeError):
        moe.moe_mx4_forward_tokens(x.repeat(33, 1), router, *ws, top_k=2)
    with pytest.raises(moe.MoeError):
        moe.moe_mx4_forward_tokens(x, router[:3].contiguous(), *ws, top_k=2)
