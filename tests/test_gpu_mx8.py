"""Microscaled 8-bit quantisation, dispatch, product, experts and layer on the GPU against the float64
oracle.

Tolerances.  Quantised bytes and decoded values are exact.  A product's FP32 sums of exact terms are
held to (K + 64) 2^-23 times the sum of the terms' magnitudes (each of at most K + 64 additions off by
one unit), plus half a step of the output type, eps / 2 relative to the value.
"""
import numpy as np
import pytest
import torch

import mixture_experts_routing_moe_gb300 as moe
from mixture_experts_routing_moe_gb300 import binding as B
from oracle import mx4_oracle as M4
from oracle import mx8_oracle as M

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [torch.float32, torch.float16, torch.bfloat16]


def rows_of(rows, K, dtype, seed, spread=8):
    """Normal rows whose magnitudes differ by up to 2^spread, with values on code borders."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, K)) * np.exp2(rng.integers(-spread, spread + 1, (rows, 1)))
    x[:, ::5] = np.round(x[:, ::5] * 16) / 16
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


def same_bytes(codes, scales, x):
    c, s = M.quantize(x)
    assert (codes.cpu().numpy() == c).all() and (scales.cpu().numpy() == s).all()


# ------------------------------------------------------------------------------ quantisation
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,K", [(1, 1), (1, 31), (3, 32), (5, 33), (2, 127), (7, 128), (4, 130),
                                    (33, 256), (9, 1357), (2, 5000), (300, 96), (1, 8192)])
def test_quantize_bytes(dtype, rows, K):
    x = rows_of(rows, K, dtype, rows * 10007 + K)
    same_bytes(*moe.moe_mx8_quantize(x.to(DEV)), np64(x))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad", [1, 8])
def test_quantize_strided_rows(dtype, pad):
    x = rows_of(40, 200 + pad, dtype, 3).to(DEV)
    codes, scales = moe.moe_mx8_quantize(x[:, :200])
    same_bytes(codes, scales, np64(x)[:, :200])
    v = torch.full((40, 200 + pad), 7.0, dtype=dtype, device=DEV)
    moe.moe_mx8_dequantize(codes, scales, 200, out=v[:, :200])
    assert (v[:, 200:] == 7).all()
    ref = M.values(codes.cpu().numpy(), scales.cpu().numpy(), 200)
    assert torch.equal(v[:, :200].cpu(), torch.from_numpy(ref).to(dtype))


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_special_values(dtype):
    x = torch.zeros(8, 96, dtype=dtype)
    x[0, 3] = float("nan")
    x[1, 40], x[1, 41] = float("inf"), 1.0
    x[2, 95], x[2, 0] = float("-inf"), -3.0
    x[3, :] = -0.0
    x[4, :32] = torch.finfo(dtype).smallest_normal / 8       # subnormals
    x[4, 32:64] = torch.finfo(dtype).max
    x[5, 64:] = torch.linspace(-8, 8, 32).to(dtype)
    x[6, 0], x[6, 1], x[6, 32], x[6, 64] = 448.0, 0.01, 450.0, 1.75
    x[7, ::2] = 1e-7
    codes, scales = moe.moe_mx8_quantize(x.to(DEV))
    same_bytes(codes, scales, np64(x))
    v = np64(moe.moe_mx8_dequantize(codes, scales, 96, torch.float32))
    # rounded once to FP32: the largest FP32 number's code stands for 2^128, an infinity there
    ref = M.values(codes.cpu().numpy(), scales.cpu().numpy(), 96)
    ref = torch.from_numpy(ref).float().double().numpy()
    assert (np.isnan(v) == np.isnan(ref)).all() and (v[~np.isnan(v)] == ref[~np.isnan(v)]).all()


def test_quantize_subnormal_and_largest_scales():
    x = torch.zeros(4, 32)
    x[0, :4] = torch.tensor([2.0 ** -126, 2.0 ** -128, 2.0 ** -130, 2.0 ** -149])
    x[1, :3] = torch.tensor([3.4e38, -1e38, 1e30])
    x[2, 0] = 2.0 ** -140
    x[3, :2] = torch.tensor([448 * 2.0 ** -127, 449 * 2.0 ** -127])
    same_bytes(*moe.moe_mx8_quantize(x.to(DEV)), np64(x))


@pytest.mark.parametrize("dtype", TYPES)
def test_dequantize_every_code_and_scale(dtype):
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1)            # 8 blocks a row
    scales = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 8)
    v = moe.moe_mx8_dequantize(codes.to(DEV), scales.to(DEV), 256, dtype).cpu()
    ref = torch.from_numpy(M.values(codes.numpy(), scales.numpy())).to(dtype)
    assert (torch.isnan(v) == torch.isnan(ref)).all()
    ok = ~torch.isnan(ref)
    assert torch.equal(v[ok], ref[ok])


def test_quantize_weights_and_empty():
    x = rows_of(6, 64, torch.bfloat16, 1).view(2, 3, 64)
    codes, scales = moe.moe_mx8_quantize(x.to(DEV))
    assert codes.shape == (2, 3, 64) and scales.shape == (2, 3, 4)
    same_bytes(codes, scales, np64(x))
    codes, scales = moe.moe_mx8_quantize(torch.empty(0, 64, device=DEV))
    assert codes.shape == (0, 64)
    assert moe.moe_mx8_dequantize(codes, scales, 64).shape == (0, 64)


def test_quantize_past_32_bits():
    """More than 2^31 values: the last rows land where they belong."""
    rows, K = (1 << 18) + 9, 8192
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device=DEV)
    tail = rows_of(9, K, torch.bfloat16, 77)
    x[-9:] = tail.to(DEV)
    codes, scales = moe.moe_mx8_quantize(x)
    same_bytes(codes[-9:], scales[-9:], np64(tail))
    assert not codes[:-9].any() and not scales[:-9].any()
    v = moe.moe_mx8_dequantize(codes, scales, K, out=x)
    ref = M.values(codes[-9:].cpu().numpy(), scales[-9:].cpu().numpy())
    assert torch.equal(v[-9:].cpu(), torch.from_numpy(ref).to(torch.bfloat16))


# ------------------------------------------------------------------------------------ product
def offsets_of(sizes):
    o = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    return torch.from_numpy(o).to(DEV), o


def check_product(sizes, N, K, dtype, seed, extra_rows=0):
    rng = np.random.default_rng(seed)
    E, rows = len(sizes), int(sum(sizes)) + extra_rows
    A = rng.standard_normal((rows, K)) * np.exp2(rng.integers(-6, 7, (rows, 1)))
    W = rng.standard_normal((E, N, K)) * np.exp2(rng.integers(-6, 7, (E, N, 1)))
    # a scale of its own for each block, so that no two of a row are alike
    A *= np.exp2(rng.integers(-3, 4, (rows, -(-K // 32)))).repeat(32, 1)[:, :K]
    W *= np.exp2(rng.integers(-3, 4, (E, N, -(-K // 32)))).repeat(32, 2)[..., :K]
    ac, asc, c, s = blocks(A)
    bc, bsc, wc, ws_ = blocks(W)
    a, w = M.values(c, s, K), M.values(wc, ws_, K)
    off, o = offsets_of(sizes)
    out = torch.full((rows, N), 42.0, dtype=dtype, device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    moe.moe_mx8_product(ac, asc, bc, bsc, offsets=off, out=out, ws=ws)
    assert moe.moe_device_status(ws) == 0
    got = np64(out)
    for e in range(E):
        g, x = got[o[e]:o[e + 1]], a[o[e]:o[e + 1]]
        ref, mag = x @ w[e].T, np.abs(x) @ np.abs(w[e]).T
        check_within(g, ref, (K + 64) * 2.0 ** -23 * mag + half_step(dtype, ref), dtype)
    assert (got[o[-1]:] == 42).all()          # rows past the groups are not written


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("sizes,N,K", [
    ([1], 1, 32), ([1], 256, 256), ([128], 256, 512), ([130], 300, 96), ([3, 0, 5], 33, 64),
    ([0, 0, 7], 129, 224), ([127, 1, 129, 64], 384, 1024), ([400], 511, 2080), ([5] * 40, 72, 288),
    ([257, 31], 520, 4096), ([1, 1], 2000, 1), ([200, 180], 264, 1056), ([3, 1, 0, 2], 64, 2176),
    ([128], 65, 1100), ([20, 7], 1030, 4128), ([2] * 10, 1000, 288), ([1, 0, 3] * 4, 1100, 1500)])
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
    out = moe.moe_mx8_product(ac, asc, bc, bsc, dtype=torch.float32)
    a, w = M.values(c, s), M.values(wc, wsc)
    assert (np.abs(np64(out) - a @ w.T) <= 300 * 2.0 ** -23 * (np.abs(a) @ np.abs(w).T)).all()
    assert moe.moe_mx8_product(ac[:0], asc[:0], bc, bsc).shape == (0, 50)


def test_product_extreme_scales():
    """Scale bytes from both ends of the range meet in one product."""
    K = 64
    ac, asc, *_ = blocks(np.ones((4, K)))
    bc, bsc, *_ = blocks(np.ones((8, K)))
    asc[:, :2], bsc[:, :2] = 247, 0           # ones are codes of 256 with byte 119
    out = np64(moe.moe_mx8_product(ac, asc, bc, bsc, dtype=torch.float32))
    assert (out == 64 * 65536 * 2.0 ** (247 - 127) * 2.0 ** -127).all()


def test_product_nan_block_stays_in_its_rows():
    rng = np.random.default_rng(4)
    A, W = rng.standard_normal((140, 320)), rng.standard_normal((70, 320))
    A[133, 300], W[60, 7] = np.nan, np.inf
    ac, asc, *_ = blocks(A)
    bc, bsc, *_ = blocks(W)
    ac[20, 40] = 0x7F                          # a NaN among the codes
    out = np64(moe.moe_mx8_product(ac, asc, bc, bsc))
    bad = np.zeros((140, 70), bool)
    bad[133], bad[20], bad[:, 60] = True, True, True
    assert (np.isnan(out) == bad).all()


def test_product_bad_offsets_stay_in_bounds():
    """Offsets that decrease or pass the rows are cut to [0, rows]; nothing outside is touched."""
    rng = np.random.default_rng(5)
    ac, asc, c, s = blocks(rng.standard_normal((20, 64)))
    bc, bsc, wc, wsc = blocks(rng.standard_normal((3, 16, 64)))
    off = torch.tensor([0, 12, 6, 900], dtype=torch.int32, device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    out = moe.moe_mx8_product(ac, asc, bc, bsc, offsets=off, dtype=torch.float32, ws=ws)
    assert moe.moe_device_status(ws) == 0
    a, w = M.values(c, s), M.values(wc, wsc)
    got = np64(out)
    assert np.allclose(got[:6], a[:6] @ w[0].T, rtol=1e-5, atol=1e-4)
    assert np.allclose(got[12:], a[12:] @ w[2].T, rtol=1e-5, atol=1e-4)


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
    want = moe.moe_mx8_product(ac, asc, bc, bsc, dtype=torch.float32)
    for by in (4, 16):
        got = moe.moe_mx8_product(shifted(ac, 16), shifted(asc, by), bc, shifted(bsc, by),
                                  dtype=torch.float32)
        assert torch.equal(got, want)


def test_product_past_32_bits():
    """An output of more than 2^31 values."""
    rng = np.random.default_rng(12)
    N, rows = 8192, (1 << 18) + 5
    bc, bsc, wc, wsc = blocks(rng.standard_normal((N, 64)))
    ac, asc, c, s = blocks(rng.standard_normal((261, 64)))
    a_codes = torch.zeros(rows, 64, dtype=torch.uint8, device=DEV)
    a_scales = torch.zeros(rows, 4, dtype=torch.uint8, device=DEV)
    a_codes[-261:], a_scales[-261:] = ac, asc
    out = moe.moe_mx8_product(a_codes, a_scales, bc, bsc)
    ref = M.values(c, s) @ M.values(wc, wsc).T
    mag = np.abs(M.values(c, s)) @ np.abs(M.values(wc, wsc)).T
    assert (np.abs(np64(out[-261:]) - ref) <= 128 * 2.0 ** -23 * mag + half_step(torch.bfloat16, ref)).all()
    assert not out[:-261].any()


def test_output_on_any_element():
    """out of 16-bit elements that starts on an odd element: no vector stores."""
    c, s = moe.moe_mx8_quantize(rows_of(5, 256, torch.float16, 6).to(DEV))
    want = moe.moe_mx8_product(c, s, c, s, dtype=torch.float16)
    out = torch.zeros(26, dtype=torch.float16, device=DEV)[1:].view(5, 5)
    assert torch.equal(moe.moe_mx8_product(c, s, c, s, out=out), want)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("sizes", [[3, 0, 5], [200, 180, 1]])
@pytest.mark.parametrize("N", [8, 72, 264, 1000])
def test_output_inside_another_tensor(dtype, sizes, N):
    """Rows of whole 16 bytes that are no whole lines, at an address that 32 does not divide: the same
    values as in a tensor of its own, and nothing written before, behind or past the groups."""
    K, E, rows = 160, len(sizes), sum(sizes) + 2
    a = moe.moe_mx8_quantize(rows_of(rows, K, dtype, N).to(DEV))
    b = moe.moe_mx8_quantize(rows_of(E * N, K, dtype, N + 1).to(DEV).view(E, N, K))
    off, _ = offsets_of(sizes)
    want = moe.moe_mx8_product(*a, *b, offsets=off, dtype=dtype)
    pad = 16 // want.element_size()
    room = torch.full((rows * N + 3 * pad,), 42.0, dtype=dtype, device=DEV)
    out = room[pad:pad + rows * N].view(rows, N)
    assert out.data_ptr() % 32 == 16
    moe.moe_mx8_product(*a, *b, offsets=off, out=out)
    assert torch.equal(out[:-2], want[:-2])
    assert (out[-2:] == 42).all() and (room[:pad] == 42).all() and (room[pad + rows * N:] == 42).all()


# ----------------------------------------------------------------------------------- dispatch
def routed(T, E, k, seed, bad=()):
    """Different experts for each token, as idx and the slots' rows in a stable order."""
    rng = np.random.default_rng(seed)
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int64).reshape(T, k)
    for t, j in bad:
        idx[t, j] = E + 3
    flat = idx.reshape(-1)
    order = np.argsort(np.where(flat < E, flat, E), kind="stable")
    order = order[: int((flat < E).sum())]
    row = np.full(T * k, 0xFFFFFFFF, np.int64)
    row[order] = np.arange(len(order))
    return torch.from_numpy(idx.astype(np.int32)).to(DEV).view(torch.uint32), idx, order, row


@pytest.mark.parametrize("T,E,k,H", [(1, 1, 1, 1), (5, 4, 2, 33), (700, 8, 3, 160), (3000, 64, 8, 96),
                                     (40, 300, 70, 50)])
def test_dispatch(T, E, k, H):
    idx, flat, order, row = routed(T, E, k, T + E, bad=[(0, 0)] if T > 1 else ())
    c, s, cb, sb = blocks(np.random.default_rng(T).standard_normal((T, H)))
    d = moe.moe_mx8_dispatch(c, s, idx, E, H)
    n = len(order)
    assert (d["codes"][:n].cpu().numpy() == cb[order // k]).all()
    assert (d["scales"][:n].cpu().numpy() == sb[order // k]).all()
    assert (d["token_of_row"][:n].view(torch.int32).cpu().numpy() == order // k).all()
    assert (d["row_of_slot"].view(torch.int32).cpu().numpy().astype(np.int64) & 0xFFFFFFFF == row).all()
    count = np.bincount(flat[flat < E], minlength=E)
    assert (np.diff(d["offsets"].cpu().numpy()) == count).all()
    assert moe.moe_device_status(d["ws"]) == (8 if T > 1 else 0)


# ------------------------------------------------------------------------------------ experts
def experts_reference(x, w, H, I):
    """(y, tolerance before the last rounding) of rows x [n, H] for one expert's gate, up, down."""
    g, u = x @ w[0][:, :H].T, x @ w[1][:, :H].T
    # FP32 sums of g and u, then exp, a reciprocal and products (a few 2^-23 each)
    dg = (H + 64) * 2.0 ** -23 * (np.abs(x) @ np.abs(w[0][:, :H]).T)
    du = (H + 64) * 2.0 ** -23 * (np.abs(x) @ np.abs(w[1][:, :H]).T)
    a = M4.silu_mul(g, u)
    da = 1.1 * dg * np.abs(u) + np.abs(M4.silu_mul(g, 1.0)) * du + 1.1 * dg * du
    rel = da / np.maximum(np.abs(a), 1e-30) + 16 * 2.0 ** -23
    slack, low = np.zeros_like(a), 0.0
    for lim in (1e-5, 1e-4, 1e-3, 1e-2, 1.0):     # the slack that each value's error reaches
        slack = np.where((rel > low) & (rel <= lim), M.quantize_slack(a, lim), slack)
        low = lim
    # a value that its error may move by more than itself: its own and its neighbours' steps
    slack = np.where(rel > 1, 2 * (np.abs(a) + da), slack)
    aq = M.fake(a)
    y = aq @ w[2][:, :I].T
    return y, ((I + 64) * 2.0 ** -23 * np.abs(aq) + slack) @ np.abs(w[2][:, :I]).T


def weights(E, H, I, rng):
    packed = [blocks(rng.standard_normal(n) / np.sqrt(n[2])) for n in ((E, I, H), (E, I, H), (E, H, I))]
    return packed, [M.values(p[2], p[3]) for p in packed]


def check_experts(sizes, H, I, dtype, seed):
    rng = np.random.default_rng(seed)
    E, rows = len(sizes), int(sum(sizes))
    xc, xs, c, s = blocks(rng.standard_normal((rows, H)))
    x = M.values(c, s, H)
    packed, w = weights(E, H, I, rng)
    off, o = offsets_of(sizes)
    ws = torch.empty(moe.mx8_experts_workspace_bytes(rows, I), dtype=torch.uint8, device=DEV)
    y = moe.moe_mx8_experts_forward_dispatched((xc, xs), off, *[p[:2] for p in packed], dtype=dtype,
                                               ws=ws)
    assert moe.moe_device_status(ws) == 0 and y.dtype == dtype
    for e in range(E):
        if sizes[e]:
            ref, tol = experts_reference(x[o[e]:o[e + 1]], [m[e] for m in w], H, I)
            tol = tol * (1 + torch.finfo(dtype).eps) + half_step(dtype, ref)
            got = np64(y)[o[e]:o[e + 1]]
            check_within(got, ref, tol, dtype)
            assert np.linalg.norm(got - ref) <= (torch.finfo(dtype).eps + 2e-3) * np.linalg.norm(ref)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("sizes,H,I", [([1], 32, 32), ([2, 0, 5], 64, 160), ([130, 3], 256, 72),
                                       ([40, 0, 300], 200, 416), ([64, 200], 512, 768), ([7], 33, 1),
                                       ([1, 5, 0, 1], 2080, 100), ([100], 160, 1000),
                                       ([1] * 8, 288, 768), ([3, 0, 1] * 4, 100, 790)])
def test_experts(dtype, sizes, H, I):
    check_experts(sizes, H, I, dtype, sum(sizes) + H + I)


def test_experts_nan_row_and_empty():
    rng = np.random.default_rng(9)
    x = rng.standard_normal((6, 64))
    x[2, 5] = np.nan
    xc, xs, *_ = blocks(x)
    packed = [p[:2] for p in weights(2, 64, 96, rng)[0]]
    off, _ = offsets_of([4, 2])
    y = np64(moe.moe_mx8_experts_forward_dispatched((xc, xs), off, *packed))
    assert np.isnan(y[2]).all() and np.isfinite(np.delete(y, 2, 0)).all()
    off0, _ = offsets_of([0, 0])
    y = moe.moe_mx8_experts_forward_dispatched((xc[:0], xs[:0]), off0, *packed)
    assert y.shape == (0, 64)


# -------------------------------------------------------------------------------------- layer
def layer(T, E, H, I, k, seed):
    rng = np.random.default_rng(seed)
    xc, xs, c, s = blocks(rng.standard_normal((T, H)))
    packed, w = weights(E, H, I, rng)
    idx, ids, *_ = routed(T, E, k, seed)
    gate = rng.random((T, k)) + 0.1
    return (xc, xs), M.values(c, s, H), [p[:2] for p in packed], w, idx, ids, gate / gate.sum(-1, keepdims=True)


@pytest.mark.parametrize("dtype,wdt", [(torch.bfloat16, torch.float32), (torch.float16, torch.float16),
                                       (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("T,E,H,I,k", [(1, 1, 32, 32, 1), (1, 8, 256, 384, 2), (3, 5, 72, 50, 5),
                                       (64, 16, 128, 96, 4), (300, 3, 200, 160, 2), (33, 64, 64, 33, 8)])
def test_layer(dtype, wdt, T, E, H, I, k):
    x, xv, packed, w, idx, ids, gate = layer(T, E, H, I, k, T + E + H)
    gate = torch.from_numpy(gate).to(wdt)
    ws = torch.empty(moe.mx8_forward_workspace_bytes(T, E, H, I, k, dtype), dtype=torch.uint8, device=DEV)
    out = moe.moe_mx8_forward(x, idx, gate.to(DEV), *packed, dtype=dtype, ws=ws)
    assert moe.moe_device_status(ws) == 0 and out.dtype == dtype
    ref, tol = np.zeros((T, H)), np.zeros((T, H))
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if len(t):
            y, d = experts_reference(xv[t], [m[e] for m in w], H, I)
            p = np64(gate)[t, j][:, None]
            np.add.at(ref, t, p * y)
            # y rounded to the type, then k products and sums in FP32
            np.add.at(tol, t, p * (d * (1 + torch.finfo(dtype).eps) + half_step(dtype, y) + k * 2.0 ** -23 * np.abs(y)))
    tol = tol * (1 + torch.finfo(dtype).eps) + half_step(dtype, ref)
    check_within(np64(out), ref, tol, dtype)
    # and the same bits from the stages
    d = moe.moe_mx8_dispatch(*x, idx, E, H)
    y = moe.moe_mx8_experts_forward_dispatched((d["codes"], d["scales"]), d["offsets"], *packed, dtype=dtype)
    assert torch.equal(moe.moe_combine(y, d["row_of_slot"], gate.to(DEV)), out)


@pytest.mark.parametrize("T", [6, 60])
def test_layer_bad_id_and_empty(T):
    x, _, packed, _, idx, _, gate = layer(T, 4, 64, 96, 2, 3)
    g = torch.from_numpy(gate).float().to(DEV)
    want = np64(moe.moe_mx8_forward(x, idx, g, *packed))
    idx.view(torch.int32)[3, 1] = 4
    idx.view(torch.int32)[4, 0] = -1
    ws = torch.empty(moe.mx8_forward_workspace_bytes(T, 4, 64, 96, 2, torch.bfloat16), dtype=torch.uint8,
                     device=DEV)
    out = np64(moe.moe_mx8_forward(x, idx, g, *packed, ws=ws))
    assert moe.moe_device_status(ws) == 8
    assert np.isnan(out[3:5]).all() and (np.delete(out, [3, 4], 0) == np.delete(want, [3, 4], 0)).all()
    idx.view(torch.int32)[:] = 7                                # none left
    assert np.isnan(np64(moe.moe_mx8_forward(x, idx, g, *packed, ws=ws))).all()
    out = moe.moe_mx8_forward((x[0][:0], x[1][:0]), idx[:0], g[:0], *packed)
    assert out.shape == (0, 64)


@pytest.mark.parametrize("T,E,k", [(8, 1, 1), (16, 2, 2), (9, 3, 3), (64, 1, 1), (64, 2, 1), (1, 64, 64), (21, 3, 3)])
def test_few_tokens_that_share_experts(T, E, k):
    """Many slots for an expert, and one for each of many."""
    x, xv, packed, w, idx, ids, gate = layer(T, E, 96, 160, k, T)
    dtype = torch.float32
    out = np64(moe.moe_mx8_forward(x, idx, torch.from_numpy(gate).float().to(DEV), *packed, dtype=dtype))
    gate = np64(torch.from_numpy(gate).float())
    ref, tol = np.zeros((T, 96)), np.zeros((T, 96))
    for e in range(E):
        t, j = np.nonzero(ids == e)
        y, d = experts_reference(xv[t], [m[e] for m in w], 96, 160)
        p = gate[t, j][:, None]
        np.add.at(ref, t, p * y)
        np.add.at(tol, t, p * (d + (k + 2) * 2.0 ** -23 * np.abs(y)))
    check_within(out, ref, tol * 1.001 + half_step(dtype, ref), dtype)


def test_few_tokens_the_same_expert_twice():
    """A token that names an expert in two slots gets it with both weights."""
    x, _, packed, _, idx, _, gate = layer(4, 6, 64, 96, 2, 3)
    idx.view(torch.int32)[:] = torch.tensor([[2, 2], [2, 1], [5, 5], [1, 1]], device=DEV)
    g = torch.from_numpy(gate).float().to(DEV)
    out = moe.moe_mx8_forward(x, idx, g, *packed, dtype=torch.float32)
    one = moe.moe_mx8_forward(x, idx[:, :1].contiguous(), g.sum(-1, keepdim=True), *packed, dtype=torch.float32)
    same = torch.tensor([0, 2, 3], device=DEV)
    assert torch.allclose(out[same], one[same], rtol=1e-5, atol=1e-5 * float(out.abs().max()))


def test_few_tokens_special_blocks():
    """Scales from both ends, NaN blocks of tokens and of weights, NaN codes."""
    x, xv, packed, w, idx, ids, gate = layer(3, 3, 64, 64, 3, 7)
    g = torch.from_numpy(gate).float().to(DEV)
    want = moe.moe_mx8_forward(x, idx, g, *packed, dtype=torch.float32)
    xs, scales = x[1].clone(), [p[1].clone() for p in packed]
    xs[:, :2] -= 60                                            # x 2^-60, gate and up 2^60, exactly
    scales[0][..., :2] += 60
    scales[1][..., :2] += 60
    moved = [(packed[0][0], scales[0]), (packed[1][0], scales[1]), packed[2]]
    assert torch.equal(moe.moe_mx8_forward((x[0], xs), idx, g, *moved, dtype=torch.float32), want)
    xs = x[1].clone()
    xs[1, 1] = 255
    out = moe.moe_mx8_forward((x[0], xs), idx, g, *packed, dtype=torch.float32)
    assert torch.isnan(out[1]).all() and torch.equal(out[[0, 2]], want[[0, 2]])
    codes = x[0].clone()
    codes[2, 40] = 0x7F
    out = moe.moe_mx8_forward((codes, x[1]), idx, g, *packed, dtype=torch.float32)
    assert torch.isnan(out[2]).all() and torch.equal(out[:2], want[:2])
    down = packed[2][1].clone()
    down[0, 10, 0] = 255                                       # expert 0's row 10: column 10 of all tokens
    out = moe.moe_mx8_forward(x, idx, g, packed[0], packed[1], (packed[2][0], down), dtype=torch.float32)
    bad = torch.isnan(out)
    assert bad[:, 10].all() and bad.sum() == 3
    assert torch.equal(out[~bad], want[~bad])
    # products whose scales meet outside FP32's exponents
    xs, scales = x[1].clone(), packed[0][1].clone()
    xs[:], scales[:] = 0, 0
    out = moe.moe_mx8_forward((x[0], xs), idx, g, (packed[0][0], scales), *packed[1:], dtype=torch.float32)
    assert (out == 0).all()


def test_layer_repeats_streams_and_graphs():
    """The same bits every time, on any stream, after another size has used the workspace, from two
    graphs replayed in turn, and with eager calls between them."""
    x, _, packed, _, idx, _, gate = layer(40, 16, 512, 384, 4, 5)
    g = torch.from_numpy(gate).float().to(DEV)
    want = moe.moe_mx8_forward(x, idx, g, *packed)
    few = lambda **kw: moe.moe_mx8_forward((x[0][:3], x[1][:3]), idx[:3], g[:3], *packed, **kw)  # noqa: E731
    want3 = few()
    assert torch.equal(want3, want[:3])
    for _ in range(10):
        assert torch.equal(moe.moe_mx8_forward(x, idx, g, *packed), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = moe.moe_mx8_forward(x, idx, g, *packed, stream=side)
    for _ in range(4):                                  # memory freed here is not the side stream's
        torch.empty(4 << 20, dtype=torch.uint8, device=DEV).fill_(255)
    side.synchronize()
    assert torch.equal(got, want)
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.graph(graphs[0]):
        a = moe.moe_mx8_forward(x, idx, g, *packed)
    with torch.cuda.graph(graphs[1]):
        b = few()
    for _ in range(3):
        a.zero_(), b.zero_()
        graphs[0].replay(), graphs[1].replay()
        assert torch.equal(moe.moe_mx8_forward(x, idx, g, *packed), want)
        torch.cuda.synchronize()
        assert torch.equal(a, want) and torch.equal(b, want3)


# ----------------------------------------------------------------------------------- refusals
def test_refusals():
    x = torch.zeros(4, 64, device=DEV)
    c, s = moe.moe_mx8_quantize(x)
    w = moe.moe_mx8_quantize(torch.zeros(2, 3, 64, device=DEV))
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV)
    idx = torch.zeros(4, 1, dtype=torch.int32, device=DEV).view(torch.uint32)
    g = torch.ones(4, 1, device=DEV)
    up, down = moe.moe_mx8_quantize(torch.zeros(2, 32, 64, device=DEV)), moe.moe_mx8_quantize(torch.zeros(2, 64, 32, device=DEV))
    for error, call in [
            (ValueError, lambda: moe.moe_mx8_quantize(x.t())),
            (ValueError, lambda: moe.moe_mx8_quantize(x.cpu())),
            (moe.MoeError, lambda: moe.moe_mx8_quantize(x.double())),
            (moe.MoeError, lambda: moe.moe_mx8_quantize(x, codes=c[:3])),
            (moe.MoeError, lambda: moe.moe_mx8_dequantize(c, s, 96)),
            (moe.MoeError, lambda: moe.moe_mx8_dequantize(c, s[:3], 64)),
            (moe.MoeError, lambda: moe.moe_mx8_dequantize(c.to(torch.int32), s, 64)),
            (moe.MoeError, lambda: moe.moe_mx8_dequantize(c, s, 64, torch.float64)),
            (moe.MoeError, lambda: moe.moe_mx8_dequantize(c, s, 64, out=torch.empty(3, 64, device=DEV))),
            (moe.MoeError, lambda: moe.moe_mx8_product(c, s, *moe.moe_mx8_quantize(torch.zeros(3, 96, device=DEV)))),
            (moe.MoeError, lambda: moe.moe_mx8_product(c, s, *w)),     # two groups need offsets
            (moe.MoeError, lambda: moe.moe_mx8_product(c, s, *w, offsets=off.long())),
            (moe.MoeError, lambda: moe.moe_mx8_product(c, s, *w, offsets=off, ws=torch.empty(64, dtype=torch.uint8, device=DEV))),
            (moe.MoeError, lambda: moe.moe_mx8_product(c, s, *w, offsets=off, out=torch.empty(4, 4, device=DEV))),
            (moe.MoeError, lambda: moe.moe_mx8_experts_forward_dispatched((c, s), off, w, w, w)),
            (moe.MoeError, lambda: moe.moe_mx8_experts_forward_dispatched((c, s), off[:2], up, up, down)),
            (moe.MoeError, lambda: moe.moe_mx8_dispatch(c, s, idx.view(torch.int32), 2, 64)),
            (moe.MoeError, lambda: moe.moe_mx8_dispatch(c, s, idx, 2, 96)),
            (moe.MoeError, lambda: moe.moe_mx8_forward((c, s), idx[:3], g[:3], up, up, down)),
            (moe.MoeError, lambda: moe.moe_mx8_forward((c, s), idx, g[:, :0], up, up, down)),
            (moe.MoeError, lambda: moe.moe_mx8_forward((c, s), idx, g.double(), up, up, down)),
            (moe.MoeError, lambda: moe.moe_mx8_forward((c, s), idx, g, up, up, down, dtype=torch.float64)),
    ]:
        with pytest.raises(error):
            call()
    assert moe.moe_mx8_forward((c, s), idx, g, up, up, down).shape == (4, 64)


def test_a_timeout_status_is_cleared_by_the_next_call():
    c, s = moe.moe_mx8_quantize(torch.ones(4, 64, device=DEV))
    ws = torch.full((256,), 255, dtype=torch.uint8, device=DEV)
    moe.moe_mx8_product(c, s, c, s, ws=ws)
    assert B.lib().moe_device_status(ws.data_ptr(), 256, None) == 0
