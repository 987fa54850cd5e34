"""What the binding does on the host around a microscaled 4-bit call, without a GPU."""
import contextlib
import glob
import os
import re
import threading

import pytest
import torch

from mixture_experts_routing_moe_gb300 import binding as B
from mixture_experts_routing_moe_gb300 import build as build_mod


@pytest.fixture
def on_cpu(monkeypatch):
    """Workspaces come from the CPU; no stream is capturing."""
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return torch.device("cpu")


def test_threads_of_one_stream_have_workspaces_of_their_own(on_cpu):
    """A call's launches may interleave with another thread's on the default stream."""
    got, both = [], threading.Barrier(2)

    def ask():
        ws = [B._mx4_ws(None, n, on_cpu, None, 0) for n in (256, 4096, 1024)]
        both.wait()
        got.append([(w.data_ptr(), w.numel()) for w in ws])
        both.wait()

    threads = [threading.Thread(target=ask) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for (pa, na), (pb, nb) in zip(*got):
        assert pa + na <= pb or pb + nb <= pa
    assert all(n >= need for one in got for (_, n), need in zip(one, (256, 4096, 1024)))


def test_kept_workspaces_are_few(on_cpu):
    """A thread that moves over many streams does not keep a buffer for each of them."""
    def run():
        for handle in range(1, 100):
            assert B._mx4_ws(None, 512, on_cpu, None, handle).numel() >= 512
        kept.append(len(B._mx4_kept.of))

    kept = []
    t = threading.Thread(target=run)
    t.start()
    t.join()
    assert kept and kept[0] <= 8


def test_workspace_of_a_given_stream_is_that_streams(monkeypatch):
    """Memory that a call on a given stream writes is allocated on that stream: a block of the current
    one may still be in use there."""
    current, made_on = ["current"], []

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    class Memory:
        device = "cuda"

        def __init__(self, *args, **kwargs):
            made_on.append(current[-1])

        def record_stream(self, stream):
            pass

    monkeypatch.setattr(B, "_empty", Memory)
    monkeypatch.setattr(torch, "empty", Memory)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current[-1])
    for need in (256, 1 << 28):
        B._mx4_ws(None, need, "cuda", "side", 7)
    assert made_on == ["side", "side"] and current == ["current"]


def test_elections_are_made_by_whole_warps():
    """elect.sync waits for every lane that its mask names, so no lane may be kept from it by a
    condition in front: a warp of which some lanes had given up would wait for good."""
    for path in glob.glob(os.path.join(os.path.dirname(B.__file__), "csrc", "*.cu*")):
        with open(path) as f:
            assert not re.findall(r"(?:&&|\|\||\?)\s*elect_one\(\)", f.read()), path


def test_largest_sizes_are_the_documented_ones():
    """One below each limit of moe_mx4.h the call is refused for its missing workspace, at it for its
    shape."""
    build_mod.build()
    fake, top = 0x10000, (1 << 31) - 1024

    def product(rows=1, E=1, N=64, K=64):
        return B.lib().moe_mx4_product(fake, fake, rows, fake, fake, fake, E, N, K, fake, B.MOE_F32,
                                       None, 0, None)
    workspace, shape = 5, 2
    assert product(rows=top - 1) == workspace and product(rows=top) == shape
    assert product(K=(1 << 24) - 1) == workspace and product(K=1 << 24) == shape
    assert product(E=1023, N=top // 1023) == workspace and product(E=1023, N=top // 1023 + 1) == shape
    tiles = lambda rows, N: (-(-rows // 128) + 1) * -(-N // 128)  # noqa: E731
    N = (1 << 24) - 1
    rows = ((top - 1) // -(-N // 128) - 1) * 128
    assert tiles(rows, N) < top and product(rows=rows, N=N) == workspace
    assert tiles(rows + 1, N) >= top and product(rows=rows + 1, N=N) == shape
    wide = (1 << 31) - 1
    assert B.lib().moe_mx4_quantize(fake, B.MOE_F32, 1, 64, wide, fake + 8, fake, None) == 4
    assert B.lib().moe_mx4_quantize(fake, B.MOE_F32, 1, 64, wide + 1, fake, fake, None) == shape
