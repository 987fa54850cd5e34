"""The norm with weights that are not ordinary numbers, of other types and for long rows, and on rows that
start on any element."""
import numpy as np
import pytest
import torch

import mixture_experts_routing_moe_gb300 as moe
from oracle import front_oracle as F
from test_gpu_norm import DEV, TYPES, check_forward, half_step, np64, rel_of, stream, weight

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,H", [(3, 64), (40, 65), (700, 4096), (300, 1357), (4, 40000)])
def test_weights_that_are_not_numbers_stay_in_their_columns(dtype, T, H):
    x, w = stream(T, H, dtype, 4), weight(H, dtype, 5)
    w[3], w[H - 1], w[33] = float("inf"), -float("inf"), float("nan")
    out = moe.moe_rms_norm(x, w, 1e-6, blocks=True)
    y, odd = np64(out["y"]), [3, 33, H - 1]
    assert not np.isfinite(y[:, odd]).any() and np.isnan(y[:, 33]).all()
    ordinary = np.delete(np.arange(H), odd)
    ref = F.rms_norm(np64(x), np.nan_to_num(np64(w), posinf=0, neginf=0), 1e-6)[0]
    y, ref = y[:, ordinary], ref[:, ordinary]
    assert (np.abs(y - ref) <= rel_of(H) * np.abs(ref) + half_step(dtype, ref)).all()
    s, last = out["scales"].cpu().numpy()[:, :-(-H // 32)], (H - 1) // 32
    assert (s[:, [0, 1, last]] == 255).all() and not (s[:, 2:last] == 255).any()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("H", [16392, 20000, 32768])
@pytest.mark.parametrize("T", [3, 200])
@pytest.mark.parametrize("eps", [1e-6, 0.0])
def test_weights_in_32_bits_for_long_rows(dtype, H, T, eps):
    x, res, w = stream(T, H, dtype, 1), stream(T, H, dtype, 2), weight(H, torch.float32, 3)
    out = moe.moe_rms_norm(x, w, eps, residual=res, blocks=True, stats=True)
    check_forward(x, res, w, eps, out, H)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("at", [1, 3])
@pytest.mark.parametrize("T,H", [(40, 64), (7, 257), (600, 1000), (3, 33000)])
def test_rows_on_any_element(dtype, at, T, H):
    """As rows on 16 bytes, but for the order in which a row's squares are summed: r is off by rel_of(H)
    either way, then half a step of the type."""
    x = stream(T, H, dtype, H)
    flat = torch.zeros(at + T * H, dtype=dtype, device=DEV)
    flat[at:] = x.reshape(-1)
    rows = flat[at:].view(T, H)
    w = weight(H, dtype, 3)
    want, got = moe.moe_rms_norm(x.contiguous(), w, blocks=True), moe.moe_rms_norm(rows, w, blocks=True)
    check_forward(x, None, w, 1e-6, got, H)
    a, b = np64(got["y"]), np64(want["y"])
    assert (np.abs(a - b) <= 2 * rel_of(H) * np.abs(b) + 2 * half_step(dtype, b)).all()
