"""No tokens: the dispatches' offsets are zeros whatever the memory held, and what follows takes them."""
import pytest
import torch

import mixture_experts_routing_moe_gb300 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("side", [False, True])
@pytest.mark.parametrize("E", [1, 5, 64])
def test_dispatch_of_no_tokens(side, E):
    stream = torch.cuda.Stream() if side else None
    H, I = 64, 96
    x = torch.zeros(0, H, dtype=torch.bfloat16, device=DEV)
    idx = torch.zeros(0, 1, dtype=torch.int32, device=DEV).view(torch.uint32)
    gate, down = torch.randn(E, I, H, device=DEV).bfloat16(), torch.randn(E, H, I, device=DEV).bfloat16()
    packed = [moe.moe_mx8_quantize(m) for m in (gate, gate, down)]
    blocks = moe.moe_mx8_quantize(x)
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(stream):
            torch.full((E + 1,), 7, dtype=torch.int32, device=DEV)       # and freed
        d, d8 = moe.moe_dispatch(x, idx, E, stream=stream), moe.moe_mx8_dispatch(*blocks, idx, E, H, stream=stream)
        y = moe.moe_experts_forward_dispatched(d["x_d"], d["offsets"], gate, gate, down, stream=stream)
        y8 = moe.moe_mx8_experts_forward_dispatched((d8["codes"], d8["scales"]), d8["offsets"], *packed, stream=stream)
        torch.cuda.synchronize()
        assert d["offsets"].tolist() == d8["offsets"].tolist() == [0] * (E + 1)
        assert y.shape == y8.shape == (0, H)
    given = torch.full((E + 1,), 7, dtype=torch.int32, device=DEV)
    assert moe.moe_dispatch(x, idx, E, offsets=given)["offsets"] is given and not given.any()
