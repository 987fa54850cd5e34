"""A dispatch of no tokens gives E + 1 offsets of zero, although the library enqueues nothing for it; without
a GPU: the library, torch's streams and the devices are stood in for."""
import pytest
import torch

from mixture_experts_routing_moe_gb300 import binding as B
from test_front_streams_host import Side, X, streams, u8  # noqa: F401


@pytest.mark.parametrize("tokens", [0, 3])
@pytest.mark.parametrize("blocks", [False, True])
def test_offsets(streams, monkeypatch, tokens, blocks):  # noqa: F811
    real, zeroed = torch.empty, []
    monkeypatch.setattr(torch, "empty", lambda *a, **k: real(*a, **k).fill_(7))
    monkeypatch.setattr(B, "_cuda", lambda *a: None)
    zero = torch.Tensor.zero_
    monkeypatch.setattr(torch.Tensor, "zero_",
                        lambda t: (zeroed.append(torch.cuda.current_stream()), zero(t))[1])
    idx = torch.zeros(tokens, 2, dtype=torch.int32).view(torch.uint32)
    if blocks:
        d = X.moe_mx8_dispatch(u8(tokens, 64), u8(tokens, 4), idx, 5, 64, stream=Side())
    else:
        d = B.moe_dispatch(torch.zeros(tokens, 64).bfloat16(), idx, 5, stream=Side())
    assert d["offsets"].tolist() == [7 if tokens else 0] * 6
    assert zeroed == ([] if tokens else ["side"])                # on the call's stream
