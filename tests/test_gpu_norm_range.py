"""The norm of rows whose squares are too small for FP32.

y = s / (mean s^2 + eps)^(1/2) w is of the size of the weights however small a row is, as long as eps
leaves it so; rstd is finite from a root mean square of 2^-128 on.  Tolerances are those of any other row:
the scaling by a power of two in between is exact.
"""
import numpy as np
import pytest
import torch

import mixture_experts_routing_moe_gb300 as moe
from oracle import front_oracle as F
from test_gpu_norm import DEV, U, check_forward, np64, rel_of, weight

pytestmark = pytest.mark.gpu
SCALES = [1e-39, 1e-38, 1e-37, 1e-30, 1e-25, 1e-20, 3e-16, 1e-9, 1.0, 1e9, 1e16]


def rows(T, H, dtype, seed, scales=SCALES, pad=0):
    """Neighbouring rows of very different sizes; a few values in each are small beside the rest."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, H + pad)) * np.take(scales, np.arange(T) % len(scales))[:, None]
    x[:, 1:H:7] *= 2.0 ** -20
    return torch.from_numpy(x).to(dtype).to(DEV)[:, :H]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,H,pad", [(24, 40, 0), (24, 64, 1), (2000, 256, 0), (2400, 600, 8), (2400, 1000, 3), (1500, 2048, 0),
                                     (640, 8200, 0), (24, 16400, 8), (24, 33000, 0), (12, 33001, 1)])
def test_rows_of_any_size(dtype, T, H, pad):
    x, w = rows(T, H, dtype, H, pad=pad), weight(H, dtype, 2)
    out = moe.moe_rms_norm(x, w, 0.0, blocks=True, stats=True)
    r = np64(out["rstd"])
    assert np.isfinite(np64(out["y"])).all()
    finite = np.isfinite(r)
    assert (finite | (np.arange(T) % len(SCALES) == 0)).all()
    ref = F.rms_norm(np64(x), 1.0, 0.0)[1]
    assert (np.abs(r - ref)[finite] <= (rel_of(H) + 4 * U) * ref[finite]).all()
    check_forward(x, None, w, 0.0, {k: v for k, v in out.items() if k != "rstd"}, H)
    # the sum, kept where the residual was, and the same rows' bits
    res = torch.zeros(T, H, dtype=dtype, device=DEV)
    got = moe.moe_rms_norm(x, w, 0.0, residual=res, sum=res, blocks=True, stats=True)
    assert torch.equal(res, x) and all(torch.equal(got[k], out[k]) for k in out)


@pytest.mark.parametrize("eps", [1e-30, 1e-36, 4e-41])
@pytest.mark.parametrize("H", [64, 3000, 33000])
def test_eps_beside_a_small_mean(eps, H):
    """eps and the mean are of one size, below 2^-100 or about it (and eps what FP32 makes of it)."""
    eps = float(np.float32(eps))
    x = rows(30, H, torch.float32, H, scales=[eps ** 0.5 * f for f in (0.01, 0.3, 1, 3, 100)])
    w = weight(H, torch.float32, 3)
    check_forward(x, None, w, eps, moe.moe_rms_norm(x, w, eps, blocks=True, stats=True), H)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("H", [64, 600, 33000])
def test_rows_that_are_not_numbers_stay_so(dtype, H):
    x = rows(8, H, dtype, 1, scales=[1e-30, 1.0])
    x[2] = 0
    x[3, 5] = float("inf")
    x[4, 6] = float("nan")
    x[5] = 1e30                                                 # squares past FP32
    out = moe.moe_rms_norm(x, torch.ones(H, dtype=dtype, device=DEV), 0.0, stats=True)
    y, r = np64(out["y"]), np64(out["rstd"])
    assert np.isnan(y[2]).all() and r[2] == np.inf              # 0 / 0
    assert np.isnan(y[3, 5]) and (np.delete(y[3], 5) == 0).all() and r[3] == 0
    assert np.isnan(y[4]).all() and np.isnan(r[4])
    assert (y[5] == 0).all() and r[5] == 0
    assert np.isfinite(y[[0, 1, 6, 7]]).all() and (np.abs(y[[0, 1, 6, 7]]).max(-1) > 0.1).all()


@pytest.mark.parametrize("H", [64, 3000, 9000])
def test_gradient_of_small_rows(H):
    """dx = r (dy w - n mean(dy w n)): of the size of r."""
    scales = [1e-30, 1e-25, 1e-20, 1e-10, 1.0, 1e10]
    s, w = rows(24, H, torch.float32, 5, scales=scales), weight(H, torch.float32, 6)
    dy = torch.from_numpy(np.random.default_rng(7).standard_normal((24, H))).float().to(DEV)
    rstd = moe.moe_rms_norm(s, w, 0.0, stats=True)["rstd"]
    dx, dw = moe.moe_rms_norm_backward(dy, s, w, rstd)
    S, W, D, R = np64(s), np64(w), np64(dy), np64(rstd)[:, None]
    n, dn = S * R, D * W
    along = (dn * n).mean(-1, keepdims=True)
    d_along = (H / 32 + 68) * U * np.abs(dn * n).mean(-1, keepdims=True)
    tol = R * (6 * U * np.abs(dn) + np.abs(n) * (d_along + 8 * U * np.abs(along))) + 1e-44
    assert (np.abs(np64(dx) - R * (dn - n * along)) <= tol).all()
    assert (np.abs(np64(dw) - (D * n).sum(0)) <= (24 + 64) * U * np.abs(D * n).sum(0)).all()
