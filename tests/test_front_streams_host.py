"""Which stream the norm's, the grouped router's and the 8-bit operators' bindings allocate on, and which
tensors they refuse, without a GPU: the library, torch's streams and the devices are stood in for."""
import contextlib

import pytest
import torch

from mixture_experts_routing_moe_gb300 import binding as B
from mixture_experts_routing_moe_gb300 import front as F
from mixture_experts_routing_moe_gb300 import mx8 as X


class Side:
    cuda_stream = 7


class Library:
    def __getattr__(self, name):
        return lambda *a: 0 if not name.endswith("_bytes") else 4096


@pytest.fixture
def streams(monkeypatch):
    """Tensors are made on the CPU; made_on lists the streams that were current then."""
    made_on, current = [], ["current"]

    @contextlib.contextmanager
    def on(stream):
        current.append("side" if isinstance(stream, Side) else stream)
        yield
        current.pop()

    real = torch.empty

    def empty(*args, **kwargs):
        made_on.append(current[-1])
        return real(*args, **kwargs)

    for m in (B, X, F):
        monkeypatch.setattr(m, "lib", Library)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1, raising=False)   # the CPU's number
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: None)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current[-1])
    return made_on


def u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


X16, IDX = torch.zeros(6, 64, dtype=torch.bfloat16), torch.zeros(6, 2, dtype=torch.int32).view(torch.uint32)
ROWS, GATE, DOWN = (u8(6, 64), u8(6, 4)), (u8(4, 32, 64), u8(4, 32, 4)), (u8(4, 64, 32), u8(4, 64, 4))
OFF, W16 = torch.zeros(5, dtype=torch.int32), torch.zeros(64, dtype=torch.bfloat16)
CALLS = [
    lambda: F.moe_rms_norm(X16, W16, residual=X16, blocks=True, stats=True, stream=Side()),
    lambda: F.moe_rms_norm_backward(X16, X16, W16, torch.zeros(6), dsum=X16, stream=Side()),
    lambda: F.moe_route_softmax_grouped(torch.zeros(6, 4), 2, 2, 1, stream=Side()),
    lambda: F.moe_forward_softmax_grouped(X16, torch.zeros(6, 4), *[torch.zeros(4, 32, 64).bfloat16()] * 2,
                                          torch.zeros(4, 64, 32).bfloat16(), 2, 2, 1, stream=Side()),
    lambda: X.moe_mx8_quantize(X16, stream=Side()),
    lambda: X.moe_mx8_dequantize(*ROWS, 64, stream=Side()),
    lambda: X.moe_mx8_dispatch(*ROWS, IDX, 4, 64, stream=Side()),
    lambda: X.moe_mx8_product(*ROWS, *GATE, offsets=OFF, stream=Side()),
    lambda: X.moe_mx8_experts_forward_dispatched(ROWS, OFF, GATE, GATE, DOWN, stream=Side()),
    lambda: X.moe_mx8_forward(ROWS, IDX, torch.zeros(6, 2), GATE, GATE, DOWN, stream=Side()),
]


@pytest.mark.parametrize("call", range(len(CALLS)))
def test_outputs_and_workspaces_are_the_given_streams(streams, call):
    CALLS[call]()
    assert streams and set(streams) == {"side"}


@pytest.mark.parametrize("call", range(len(CALLS)))
def test_tensors_of_another_device_are_refused(streams, call, monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    with pytest.raises(ValueError):
        CALLS[call]()
    assert not streams
