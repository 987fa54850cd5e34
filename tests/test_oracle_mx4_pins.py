"""The microscaled 4-bit oracle against hand-computed values and its own invariants."""
import numpy as np
import pytest

from oracle import mx4_oracle as M


def test_code_values():
    codes = np.array([[0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE] + [0] * 8], np.uint8)
    got = M.values(codes, np.array([[128, 0, 0, 0]], np.uint8))[0, :16]
    want = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6]) * 2
    assert (got == want).all()


def test_ties_go_to_the_even_code():
    x = np.zeros((1, 32))
    x[0, :9] = [4.0, .25, .75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.9]   # scale 1 (max in [4, 8))
    assert list(M.fake(x)[0, :9]) == [4, 0, 1, 1, 2, 2, 4, 4, 6]
    assert list(M.fake(-x)[0, 2:9]) == [-1, -1, -2, -2, -4, -4, -6]
    assert M.quantize(x)[1][0, 0] == 127


@pytest.mark.parametrize("top,byte", [(4.0, 127), (7.999, 127), (8.0, 128), (1.0, 125),
                                      (2.0 ** -125, 0), (2.0 ** -126, 0), (2.0 ** -149, 0),
                                      (2.0 ** -124, 1), (3.0e38, 252), (0.0, 0)])
def test_scale_bytes(top, byte):
    x = np.zeros((1, 32))
    x[0, 5] = top
    assert M.quantize(x)[1][0, 0] == byte


def test_bad_blocks_and_padding():
    x = np.ones((2, 70))
    x[0, 3] = np.nan
    x[1, 40] = -np.inf
    codes, scales = M.quantize(x)
    assert codes.shape == (2, 48) and scales.shape == (2, 4)
    assert list(scales[0]) == [255, 125, 125, 0] and list(scales[1]) == [125, 255, 125, 0]
    assert (codes[0, :16] == 0).all() and (codes[1, 16:32] == 0).all()
    assert (codes[:, 35:] == 0).all()
    v = M.values(codes, scales, 70)
    assert np.isnan(v[0, :32]).all() and (v[0, 32:] == 1).all()


def test_error_of_a_trip_and_its_fixed_points():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((64, 160)) * np.exp2(rng.integers(-20, 20, (64, 1)))
    v = M.fake(x)
    top = np.abs(x).reshape(64, 5, 32).max(-1).repeat(32, -1).reshape(x.shape)
    # half a step of the widest gap (2), or the clipping of (6, 8), in units of the scale
    assert (np.abs(v - x) <= 2 * np.exp2(np.floor(np.log2(top)) - 2)).all()
    assert (M.fake(v)[np.abs(v) > 0] != 0).all()


@pytest.mark.parametrize("seed", range(3))
def test_slack_covers_perturbed_inputs(seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((400, 64))
    x[:200, ::7] = np.round(x[:200, ::7] * 4) / 4      # many values on borders
    x[::3, 0] = 4.0                                    # and maxima on a power of two
    rel = 1e-3
    slack = M.quantize_slack(x, rel)
    for s in (1, -1):
        y = x * (1 + s * rel * 0.999 * rng.random(x.shape))
        assert (np.abs(M.fake(y) - M.fake(x)) <= slack + 1e-12).all()
