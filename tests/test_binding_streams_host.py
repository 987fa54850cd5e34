"""Which stream the binding allocates on, without a GPU: the library and torch's streams are stood in
for."""
import contextlib

import pytest
import torch

from mixture_experts_routing_moe_gb300 import binding as B


class Memory:
    """What torch.empty gives: knows the stream that was current."""
    made_on, current = [], ["current"]
    is_cuda = True

    def __init__(self, *args, **kwargs):
        Memory.made_on.append(Memory.current[-1])
        self.device, self.dtype = kwargs.get("device"), kwargs.get("dtype")

    def record_stream(self, stream):
        pass

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20

    def numel(self):
        return 1 << 30


class Library:
    def __getattr__(self, name):
        return lambda *a: 0 if not name.endswith("_bytes") else 4096


class Side:
    cuda_stream = 7


@pytest.fixture
def on_cpu(monkeypatch):
    Memory.made_on, Memory.current = [], ["current"]

    @contextlib.contextmanager
    def on(stream):
        Memory.current.append("side" if isinstance(stream, Side) else stream)
        yield
        Memory.current.pop()

    real = torch.empty
    x = {n: real(*s, dtype=torch.bfloat16) for n, s in
         (("x", (6, 64)), ("logits", (6, 4)), ("gate", (4, 32, 64)), ("down", (4, 64, 32)),
          ("y", (12, 64)), ("w", (6, 2)))}
    x["idx"] = real(6, 2, dtype=torch.int32)
    monkeypatch.setattr(B, "lib", Library)
    monkeypatch.setattr(B, "_cuda", lambda *a: None)
    monkeypatch.setattr(torch, "empty", Memory)
    monkeypatch.setattr(torch, "empty_like", Memory)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Memory.current[-1])
    return x


CALLS = [
    lambda t: B.moe_route(t["logits"], 2, stream=Side()),
    lambda t: B.moe_route_sigmoid_grouped(t["logits"], 2, 2, 1, stream=Side()),
    lambda t: B.moe_selected_router_weights(t["logits"], t["idx"], stream=Side()),
    lambda t: B.moe_dispatch(t["x"], t["idx"], 4, stream=Side()),
    lambda t: B.moe_experts_forward_dispatched(t["y"], t["idx"], t["gate"], t["gate"], t["down"],
                                               stream=Side()),
    lambda t: B.moe_combine(t["y"], t["idx"], t["w"], stream=Side()),
    lambda t: B.moe_forward(t["x"], t["logits"], t["gate"], t["gate"], t["down"], 2, stream=Side()),
    lambda t: B.moe_forward_sigmoid_grouped(t["x"], t["logits"], t["gate"], t["gate"], t["down"], 2,
                                            2, 1, stream=Side()),
    lambda t: B.moe_forward_with_events(t["x"], t["logits"], t["gate"], t["gate"], t["down"], 2,
                                        True, stream=Side()),
    lambda t: B.moe_combine_backward(t["y"], t["idx"], t["w"], t["x"], stream=Side()),
    lambda t: B.moe_experts_backward(t["y"], t["idx"], t["gate"], t["gate"], t["down"], t["y"],
                                     stream=Side()),
    lambda t: B.moe_dispatch_backward(t["y"], t["idx"], 6, 2, stream=Side()),
]


@pytest.mark.parametrize("call", range(len(CALLS)))
def test_outputs_and_workspaces_are_the_given_streams(on_cpu, call):
    CALLS[call](on_cpu)
    assert Memory.made_on and set(Memory.made_on) == {"side"}
