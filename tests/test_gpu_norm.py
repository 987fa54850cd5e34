"""The residual norm and its gradient on the GPU against the float64 oracle.

Tolerances.  The sum is FP32 addition rounded once: exact.  A sum of squares runs through at most
H / 32 + 64 FP32 additions in a row (a lane's values, the warp's and the block's trees), all of one
sign, so r is off by half of that many 2^-24 and six more roundings follow up to y; then half a
step of the type.  Blocks may differ from the oracle's by quantize_slack() of that error.
"""
import numpy as np
import pytest
import torch

import mixture_experts_routing_moe_gb300 as moe
from oracle import front_oracle as F
from oracle import mx8_oracle as M

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [torch.float32, torch.float16, torch.bfloat16]
U = 2.0 ** -24
SIZES = [(1, 1), (1, 8), (3, 31), (2, 33), (5, 256), (7, 257), (40, 264), (9, 1000), (33, 1357), (700, 96),
         (6, 2048), (3000, 520), (5, 4104), (700, 7168), (3, 8200), (2, 16392), (2, 33000), (3, 40001)]


def np64(t):
    return t.double().cpu().numpy()


def half_step(dtype, ref):
    return torch.finfo(dtype).eps / 2 * np.abs(ref) + torch.finfo(dtype).tiny


def stream(T, H, dtype, seed, pad=0):
    """Rows of different lengths with a few outlying columns, cut out of a wider buffer."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, H + pad)) * np.exp(0.5 * rng.standard_normal((T, 1)))
    x *= 1 + 15 * (rng.random(H + pad) < 0.01)
    return torch.from_numpy(x).to(dtype).to(DEV)[:, :H]


def weight(H, dtype, seed):
    return torch.from_numpy(1 + 0.2 * np.random.default_rng(seed).standard_normal(H)).to(dtype).to(DEV)


def rel_of(H):
    return (H / 32 + 64) * U / 2 + 6 * U


def check_forward(x, res, w, eps, out, H):
    s = x if res is None else (x.float() + res.float()).to(x.dtype)
    if res is not None:
        assert torch.equal(out["sum"], s)
    y, r = F.rms_norm(np64(s), np64(w), eps)
    rel = rel_of(H)
    if "y" in out:
        assert (np.abs(np64(out["y"]) - y) <= rel * np.abs(y) + half_step(x.dtype, y)).all()
    if "rstd" in out:
        assert (np.abs(np64(out["rstd"]) - r) <= (rel + 2 * U) * r).all()
    if "codes" in out:
        got = M.values(out["codes"].cpu().numpy(), out["scales"].cpu().numpy(), H)
        # (subnormal results: an absolute 2^-149)
        assert (np.abs(got - M.fake(y)) <= M.quantize_slack(y, rel) + 1e-44).all()
        pad = out["scales"][..., -(-H // 32):]
        assert not pad.any() and not out["codes"][..., H:].any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,H", SIZES)
def test_forward(dtype, T, H):
    x, res, w = stream(T, H, dtype, H), stream(T, H, dtype, H + 1), weight(H, dtype, 2)
    out = moe.moe_rms_norm(x, w, 1e-5, residual=res, blocks=True, stats=True)
    check_forward(x, res, w, 1e-5, out, H)
    # and the blocks are those of the FP32 result: of y itself where y is FP32
    if dtype == torch.float32:
        c, s = moe.moe_mx8_quantize(out["y"])
        assert torch.equal(c, out["codes"]) and torch.equal(s, out["scales"])
    out = moe.moe_rms_norm(x, w, 0.0)
    assert set(out) == {"y"}
    check_forward(x, None, w, 0.0, out, H)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,H,pad", [(50, 200, 1), (50, 200, 8), (700, 1357, 3), (3, 34000, 5)])
def test_strided_rows_and_other_weights(dtype, T, H, pad):
    x, res = stream(T, H, dtype, 1, pad), stream(T, H, dtype, 2, pad + 8)
    w = weight(H, torch.float32, 3)
    total = torch.full((T, H + pad), 7.0, dtype=dtype, device=DEV)
    y = torch.full((T, H + 8), 7.0, dtype=dtype, device=DEV)
    out = moe.moe_rms_norm(x, w, 1e-6, residual=res, sum=total[:, :H], y=y[:, :H], blocks=True, stats=True)
    check_forward(x, res, w, 1e-6, out, H)
    assert (total[:, H:] == 7).all() and (y[:, H:] == 7).all()     # between the rows


def test_rows_on_any_element():
    flat = torch.randn(1 + 40 * 64, device=DEV).half()
    x = flat[1:].view(40, 64)
    w = weight(64, torch.float16, 3)
    want = moe.moe_rms_norm(x.clone(), w, blocks=True)
    got = moe.moe_rms_norm(x, w, blocks=True)
    check_forward(x, None, w, 1e-6, got, 64)
    assert (np64(got["y"]) - np64(want["y"]) <= 2 * half_step(torch.float16, np64(want["y"]))).all()


@pytest.mark.parametrize("T,H", [(37, 136), (5, 33), (700, 4096), (3, 40000)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_in_place(dtype, T, H):
    x, res, w = stream(T, H, dtype, 1), stream(T, H, dtype, 2), weight(H, dtype, 3)
    want = moe.moe_rms_norm(x, w, residual=res)
    r = res.clone()
    got = moe.moe_rms_norm(x, w, residual=r, sum=r)
    assert got["sum"] is r and torch.equal(r, want["sum"]) and torch.equal(got["y"], want["y"])
    a = x.clone()
    got = moe.moe_rms_norm(a, w, residual=res, sum=a)
    assert torch.equal(a, want["sum"]) and torch.equal(got["y"], want["y"])
    a, r = x.clone(), res.clone()
    got = moe.moe_rms_norm(a, w, residual=r, sum=r, y=a)
    assert torch.equal(r, want["sum"]) and torch.equal(a, want["y"])
    a = x.clone()
    moe.moe_rms_norm(a, w, y=a)
    assert torch.equal(a, moe.moe_rms_norm(x, w)["y"])


def test_outputs_asked_for():
    x, res, w = stream(6, 96, torch.bfloat16, 1), stream(6, 96, torch.bfloat16, 2), weight(96, torch.bfloat16, 3)
    full = moe.moe_rms_norm(x, w, residual=res, blocks=True, stats=True)
    assert set(full) == {"sum", "y", "codes", "scales", "rstd"}
    only = moe.moe_rms_norm(x, w, residual=res, values=False, blocks=True)
    assert set(only) == {"sum", "codes", "scales"} and torch.equal(only["codes"], full["codes"])
    given = {"codes": torch.empty_like(full["codes"]), "scales": torch.empty_like(full["scales"])}
    got = moe.moe_rms_norm(x.view(2, 3, 96), w, residual=res.view(2, 3, 96), stats=True,
                           codes=given["codes"].view(2, 3, -1), scales=given["scales"].view(2, 3, -1))
    assert got["rstd"].shape == (2, 3) and torch.equal(given["codes"], full["codes"])
    assert moe.moe_rms_norm(x[:0], w, residual=res[:0], blocks=True)["codes"].shape == (0, 96)


@pytest.mark.parametrize("H", [64, 65, 40000])
def test_special_rows(H):
    x = torch.randn(6, H, device=DEV).bfloat16()
    x[1] = 0
    x[2, 40] = float("nan")
    x[3, 0] = float("inf")
    x[4] = -0.0
    w = weight(H, torch.bfloat16, 1)
    out = moe.moe_rms_norm(x, w, 1e-6, blocks=True, stats=True)
    y = np64(out["y"])
    assert (y[[1, 4]] == 0).all() and np.isnan(y[2]).all()
    assert np.isnan(y[3, 0]) and (y[3, 1:] == 0).all()            # inf / inf, and x / inf
    assert np.isfinite(y[[0, 5]]).all()
    s = out["scales"].cpu().numpy()[:, :-(-H // 32)]
    assert (s[2] == 255).all() and (s[1] == 0).all() and s[3, 0] == 255 and (s[3, 1:] == 0).all()
    assert not out["codes"][2].any()
    assert np.isnan(np64(moe.moe_rms_norm(x, w, 0.0)["y"])[1]).all()   # 0 / 0


def test_many_values():
    """More than 2^31 values: the last rows land where they belong."""
    T, H = (1 << 18) + 9, 8192
    x = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)
    x[-9:] = stream(9, H, torch.bfloat16, 3)
    w = weight(H, torch.bfloat16, 1)
    out = moe.moe_rms_norm(x, w, blocks=True)
    want = moe.moe_rms_norm(x[-9:].clone(), w, blocks=True)
    # (few rows are summed in another order)
    assert (np.abs(np64(out["y"][-9:]) - np64(want["y"])) <= 3 * half_step(torch.bfloat16, np64(want["y"]))).all()
    assert not out["y"][:-9].any() and not out["codes"][:-9].any() and out["scales"][-1].any()


# ----------------------------------------------------------------------------------- gradient
def gradient_case(T, H, dtype, pad=0, wdt=None):
    s, w = stream(T, H, dtype, 5, pad), weight(H, wdt or dtype, 6)
    rng = np.random.default_rng(7)
    dy, ds = (torch.from_numpy(rng.standard_normal((T, H + pad))).to(dtype).to(DEV)[:, :H] for _ in range(2))
    rstd = torch.from_numpy(F.rms_norm(np64(s), 1.0, 1e-5)[1]).float().to(DEV)
    return s, w, dy, ds, rstd


def check_gradient(s, w, dy, ds, rstd, dx, dw, T, H):
    dtype = s.dtype
    S, W, D = np64(s), np64(w), np64(dy)
    E = 0.0 if ds is None else np64(ds)
    R = np64(rstd)[:, None]
    n = S * R
    dn = D * W
    along = (dn * n).mean(-1, keepdims=True)
    ref = E + R * (dn - n * along)
    # the mean: H / 32 + 68 roundings of terms of either sign; then six on the way
    d_along = (H / 32 + 68) * U * np.abs(dn * n).mean(-1, keepdims=True)
    tol = R * (4 * U * np.abs(dn) + np.abs(n) * (d_along + 6 * U * np.abs(along))) + 2 * U * (np.abs(ref) + np.abs(E))
    assert (np.abs(np64(dx) - ref) <= tol + half_step(dtype, ref)).all()
    tol = (T + 64) * U * np.abs(D * n).sum(0) + 1e-44
    assert (np.abs(np64(dw) - (D * n).sum(0)) <= tol).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,H", SIZES)
def test_gradient(dtype, T, H):
    s, w, dy, ds, rstd = gradient_case(T, H, dtype)
    dx, dw = moe.moe_rms_norm_backward(dy, s, w, rstd, dsum=ds)
    assert dx.dtype == dtype and dw.dtype == torch.float32
    check_gradient(s, w, dy, ds, rstd, dx, dw, T, H)
    dx, dw2 = moe.moe_rms_norm_backward(dy, s, w, rstd)
    check_gradient(s, w, dy, None, rstd, dx, dw2, T, H)
    assert torch.equal(dw, dw2)                               # the same bits


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,H,pad", [(50, 200, 1), (50, 200, 8), (700, 1357, 3), (3, 34000, 5)])
def test_gradient_strided_rows_and_other_weights(dtype, T, H, pad):
    s, w, dy, ds, rstd = gradient_case(T, H, dtype, pad, torch.float32)
    dx = torch.full((T, H + 3), 7.0, dtype=dtype, device=DEV)
    _, dw = moe.moe_rms_norm_backward(dy, s, w, rstd, dsum=ds, dx=dx[:, :H])
    check_gradient(s, w, dy, ds, rstd, dx[:, :H], dw, T, H)
    assert (dx[:, H:] == 7).all()


@pytest.mark.parametrize("T,H", [(37, 136), (5, 33), (3, 40000)])
def test_gradient_in_place(T, H):
    s, w, dy, ds, rstd = gradient_case(T, H, torch.bfloat16)
    want, dw = moe.moe_rms_norm_backward(dy, s, w, rstd, dsum=ds)
    for at in (0, 1):
        a = [dy.clone(), ds.clone()]
        got, dw2 = moe.moe_rms_norm_backward(a[0], s, w, rstd, dsum=a[1], dx=a[at])
        assert got is a[at] and torch.equal(got, want) and torch.equal(dw2, dw)


def test_gradient_is_a_difference():
    """(L(s + h v) - L(s - h v)) / 2h of the forward kernel's own y, in FP32: the difference of two sums
    of 2000 terms of about 1 is off by their roundings, some 2^-24 2000^(1/2) each, over 2h."""
    T, H, h = 4, 500, 0.05
    s, w, dy, _, rstd = gradient_case(T, H, torch.float32)
    rng = np.random.default_rng(8)
    v = torch.from_numpy(rng.standard_normal((T, H))).float().to(DEV)
    dx, dw = moe.moe_rms_norm_backward(dy, s, w, rstd)
    loss = lambda q, u: (moe.moe_rms_norm(q, u, 1e-5)["y"].double() * dy.double()).sum()  # noqa: E731
    d = (loss(s + h * v, w) - loss(s - h * v, w)) / (2 * h)
    along = (dx.double() * v.double()).sum()
    assert abs(float(d - along)) <= 1e-2 * float(dx.double().norm() * v.double().norm()) / T ** 0.5
    v = torch.from_numpy(rng.standard_normal(H)).float().to(DEV)   # linear in the weight: no h^2 term
    d = (loss(s, w + h * v) - loss(s, w - h * v)) / (2 * h)
    assert abs(float(d - (dw.double() * v.double()).sum())) <= 1e-4 * float(dw.double().norm() * v.double().norm())


def test_gradient_without_rows():
    s, w, dy, ds, rstd = gradient_case(3, 64, torch.bfloat16)
    dx, dw = moe.moe_rms_norm_backward(dy[:0], s[:0], w, rstd[:0], dweight=torch.ones(64, device=DEV))
    assert dx.shape == (0, 64) and not dw.any()


# ------------------------------------------------------------------------- streams and graphs
def test_streams_and_graphs():
    """The same bits on another stream and from two graphs of different sizes replayed in turn with
    eager calls between them."""
    s, w, dy, ds, rstd = gradient_case(900, 1024, torch.bfloat16)
    def both(n):
        out = moe.moe_rms_norm(dy[:n], w, residual=s[:n], blocks=True)
        dx, dw = moe.moe_rms_norm_backward(dy[:n], s[:n], w, rstd[:n], dsum=ds[:n])
        return [*out.values(), dx, dw]
    want = {n: [t.clone() for t in both(n)] for n in (900, 5)}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = moe.moe_rms_norm(dy, w, residual=s, blocks=True, stream=side)
    dx, dw = moe.moe_rms_norm_backward(dy, s, w, rstd, dsum=ds, stream=side)
    for _ in range(4):
        torch.empty(4 << 20, dtype=torch.uint8, device=DEV).fill_(255)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip([*out.values(), dx, dw], want[900]))
    graphs, results = {}, {}
    for n in want:
        graphs[n] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[n]):
            results[n] = both(n)
    for _ in range(3):
        for n in want:
            for t in results[n]:
                t.zero_()
            graphs[n].replay()
        assert all(torch.equal(a, b) for a, b in zip(both(900), want[900]))
        torch.cuda.synchronize()
        for n in want:
            assert all(torch.equal(a, b) for a, b in zip(results[n], want[n]))


def test_refusals():
    x, w = torch.zeros(4, 64, device=DEV), torch.ones(64, device=DEV)
    rstd = torch.ones(4, device=DEV)
    for error, call in [
            (ValueError, lambda: moe.moe_rms_norm(x.t(), torch.ones(4, device=DEV))),
            (ValueError, lambda: moe.moe_rms_norm(x.cpu(), w)),
            (moe.MoeError, lambda: moe.moe_rms_norm(x.double(), w)),
            (moe.MoeError, lambda: moe.moe_rms_norm(x, w[:63])),
            (moe.MoeError, lambda: moe.moe_rms_norm(x, w.half())),
            (moe.MoeError, lambda: moe.moe_rms_norm(x, w, -1.0)),
            (moe.MoeError, lambda: moe.moe_rms_norm(x, w, residual=x[:3])),
            (moe.MoeError, lambda: moe.moe_rms_norm(x, w, residual=x.half())),
            (moe.MoeError, lambda: moe.moe_rms_norm(x, w, y=x.half())),
            (moe.MoeError, lambda: moe.moe_rms_norm(x, w, rstd=rstd[:3])),
            (moe.MoeError, lambda: moe.moe_rms_norm(x, w, codes=torch.zeros(4, 32, dtype=torch.uint8, device=DEV))),
            (moe.MoeError, lambda: moe.moe_rms_norm_backward(x, x[:3], w, rstd)),
            (moe.MoeError, lambda: moe.moe_rms_norm_backward(x, x, w, rstd[:3])),
            (moe.MoeError, lambda: moe.moe_rms_norm_backward(x, x, w, rstd, dweight=w.half())),
            (moe.MoeError, lambda: moe.moe_rms_norm_backward(x, x, w, rstd, ws=torch.empty(256, dtype=torch.uint8, device=DEV))),
    ]:
        with pytest.raises(error):
            call()
