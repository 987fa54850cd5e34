"""The 8-bit and front oracles against independent statements of the same definitions, on the CPU."""
import numpy as np
import pytest
import torch

import oracle as O
from oracle import front_oracle as F
from oracle import mx8_oracle as M


def test_grid_is_torchs_e4m3():
    table = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert (M.GRID == table).all() and M.GRID[-1] == 448


def test_codes_are_torchs_rounding():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((50, 160)) * np.exp2(rng.integers(-12, 12, (50, 1)))
    x[:, ::7] = np.round(x[:, ::7] * 16) / 16
    c, s = M.quantize(x)
    scaled = x * np.exp2(127.0 - np.repeat(s[:, :5].astype(float), 32, 1))
    want = torch.from_numpy(scaled).to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8)
    x32 = scaled.astype(np.float32).astype(np.float64) == scaled
    assert (c == want.numpy())[x32].all()
    assert np.abs(scaled).max() <= 448


@pytest.mark.parametrize("top,byte", [(448.0, 127), (449.0, 128), (256.0, 127), (224.0, 126), (225.0, 127),
                                      (1.75, 119), (1.76, 120), (1.0, 119), (0.0, 0),
                                      (2.0 ** -149, 0), (3.4e38, 247)])
def test_scale_of_a_largest_value(top, byte):
    x = np.zeros((1, 32))
    x[0, 3] = top
    assert M.quantize(x)[1][0, 0] == byte


def test_special_blocks():
    x = np.zeros((3, 64))
    x[0, 5], x[1, 40], x[2, 2] = np.nan, -np.inf, -0.0
    c, s = M.quantize(x)
    assert s[:, :2].tolist() == [[255, 0], [0, 255], [0, 0]]
    assert c[0].max() == 0 and c[2, 2] == 128
    v = M.values(c, s)
    assert np.isnan(v[0, :32]).all() and (v[0, 32:] == 0).all()


def test_slack_covers_a_perturbation():
    rng = np.random.default_rng(2)
    a = rng.standard_normal((400, 64))
    for rel in (1e-6, 1e-3, 1e-2):
        b = a * (1 + rel * rng.uniform(-1, 1, a.shape))
        assert (np.abs(M.fake(b) - M.fake(a)) <= M.quantize_slack(a, rel) * (1 + 1e-12)).all()


def test_norm_gradient_is_autograds():
    rng = np.random.default_rng(3)
    s, w, dy, ds = (torch.from_numpy(rng.standard_normal(n)) for n in ((5, 9), 9, (5, 9), (5, 9)))
    s.requires_grad_(), w.requires_grad_()
    y = s * torch.rsqrt((s * s).mean(-1, keepdim=True) + 1e-3) * w
    ((y * dy).sum() + (s * ds).sum()).backward()
    dx, dw = F.rms_norm_backward(dy.numpy(), s.detach().numpy(), w.detach().numpy(), 1e-3, ds.numpy())
    assert np.allclose(dx, s.grad.numpy(), rtol=1e-12) and np.allclose(dw, w.grad.numpy(), rtol=1e-12)


def test_norm_gradient_is_a_difference():
    rng = np.random.default_rng(4)
    s, dy, v = rng.standard_normal((3, 3, 7))
    w = rng.standard_normal(7)
    f = lambda q: (F.rms_norm(q, w, 1e-2)[0] * dy).sum()  # noqa: E731
    h = 1e-6
    d = (f(s + h * v) - f(s - h * v)) / (2 * h)
    assert abs(d - (F.rms_norm_backward(dy, s, w, 1e-2)[0] * v).sum()) < 1e-7


def test_one_group_is_the_plain_router():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((20, 24)).astype(np.float32)
    x[:, 5] = x[:, 11]                                       # ties
    x[3, 0], x[4, 1] = np.nan, np.inf
    x[5] = -np.inf
    x[6, 3:] = -np.inf
    idx, w = F.route_softmax_grouped(x, 6, 1, 1, False, True, 1.0)
    ids, ref = O.route(x, 6, True, "f32")
    assert (idx == ids).all()
    assert np.allclose(w, ref, rtol=1e-6, equal_nan=True)


def test_groups_by_hand():
    p = np.array([[0.30, 0.01, 0.20, 0.19, 0.25, 0.05]])
    x = np.log(p)
    # largest: groups {0,1}: .30, {2,3}: .20, {4,5}: .25; sums of two: .31, .39, .30
    idx, w = F.route_softmax_grouped(x, 2, 3, 1, True, False, 2.0)
    assert idx.tolist() == [[2, 3]] and np.allclose(w, [[0.4, 0.38]])
    idx, w = F.route_softmax_grouped(x, 3, 3, 2, False, True, 1.0)
    assert idx.tolist() == [[0, 4, 5]] and np.allclose(w, np.array([[0.30, 0.25, 0.05]]) / 0.6)
    bias = np.array([0, 0, 0, 0.2, -np.inf, 0])
    idx, w = F.route_softmax_grouped(x, 3, 3, 2, False, False, 1.0, bias)
    assert idx.tolist() == [[3, 0, 2]] and np.allclose(w, [[0.19, 0.30, 0.20]])
