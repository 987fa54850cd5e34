"""The microscaled products' 16-bit outputs are their 32-bit ones rounded once, however a tile's rows are
stored: by lanes or by whole lines, from single CTAs or pairs, at any width; rows behind the last group and
what lies beside the output keep their values."""
import numpy as np
import pytest
import torch

import mixture_experts_routing_moe_gb300 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"

# rows, groups, N: few rows; many a group of a small output; an output of three full tiles an SM (on 152
# SMs 14.9 million values) on either side; pairs
CASES = [(40, 16, 768), (60, 16, 1000), (2400, 16, 2048), (2400, 16, 1000), (7000, 64, 2048), (7700, 64, 2048),
         (7700, 64, 2056), (16500, 110, 920), (3000, 7, 1000), (3000, 7, 2048), (1000, 1, 264)]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rows,E,N", CASES)
@pytest.mark.parametrize("K", [96, 1000])
def test_16_bit_rows_are_the_32_bit_ones_rounded(bits, dtype, rows, E, N, K):
    quantize, product = ((moe.moe_mx4_quantize, moe.moe_mx4_product) if bits == 4 else
                         (moe.moe_mx8_quantize, moe.moe_mx8_product))
    g = torch.Generator(device=DEV).manual_seed(rows + N + K)
    a = quantize(torch.randn(rows, K, generator=g, device=DEV))
    b = quantize(torch.randn(E, N, K, generator=g, device=DEV) * K ** -0.5)
    cut = np.sort(np.random.default_rng(rows).integers(0, rows - 2, E - 1))   # empty groups among them
    last = rows - 3
    off = torch.tensor([0, *np.minimum(cut, last), last], dtype=torch.int32, device=DEV)
    want = product(*a, *b, offsets=off, dtype=torch.float32)[:last].to(dtype)
    buffer = torch.full((rows + 2, N), 7.0, dtype=dtype, device=DEV)
    got = product(*a, *b, offsets=off, out=buffer[1:-1])
    assert torch.equal(got[:last], want)
    assert (buffer[0] == 7).all() and (buffer[1 + last:] == 7).all()
