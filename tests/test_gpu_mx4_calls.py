"""Microscaled 4-bit calls from several threads and on other streams than the current one."""
import threading

import pytest
import torch

import mixture_experts_routing_moe_gb300 as moe
from mixture_experts_routing_moe_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


def weights(E, H, I, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return [moe.moe_mx4_quantize(torch.randn(*s, generator=g, device=DEV) * s[2] ** -0.5)
            for s in ((E, I, H), (E, I, H), (E, H, I))]


def calls(seed, T, E, H, I, k):
    """(layer for few tokens, experts over rows) as functions without arguments."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    w = weights(E, H, I, seed)
    x = torch.randn(T, H, generator=g, device=DEV).bfloat16()
    router = (torch.randn(E, H, generator=g, device=DEV) * H ** -0.5).bfloat16()
    rows = torch.randn(E * 24, H, generator=g, device=DEV).bfloat16()
    off = torch.arange(E + 1, device=DEV, dtype=torch.int32) * 24
    return (lambda: moe.moe_mx4_forward_tokens(x, router, *w, top_k=k),
            lambda: moe.moe_mx4_experts_forward_dispatched(rows, off, *w))


def test_two_threads_on_one_stream():
    """Both threads stay on the default stream; each result is that of the same call on its own."""
    jobs = [calls(1, 6, 8, 512, 384, 2), calls(2, 11, 12, 256, 640, 3)]
    want = [[f() for f in job] for job in jobs]
    torch.cuda.synchronize()
    start, wrong = threading.Barrier(2), []

    def work(n):
        start.wait()
        for i in range(150):
            got = [f() for f in jobs[n]]
            if i % 10 == 0 and not all(torch.equal(a, b) for a, b in zip(got, want[n])):
                wrong.append((n, i))

    threads = [threading.Thread(target=work, args=(n,)) for n in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong


def together(*jobs):
    """Each job in a thread of its own, all started at once; what they raised."""
    start, raised = threading.Barrier(len(jobs)), []

    def work(job):
        start.wait()
        try:
            job()
        except Exception as e:  # noqa: BLE001
            raised.append(e)

    threads = [threading.Thread(target=work, args=(job,)) for job in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return raised


def test_threads_with_layers_of_other_sizes():
    """The kernel's limit of shared memory is the process's: a call of one size does not take it from a
    larger call of another thread, between that one's look and its launch."""
    E, H, I = 8, 256, 256
    w = weights(E, H, I, 3)
    router = torch.randn(E, H, device=DEV).bfloat16()

    def many(T, k):
        x = torch.randn(T, H, device=DEV).bfloat16()
        out = torch.empty_like(x)
        ws = torch.empty(moe.mx4_tokens_workspace_bytes(T, E, H, I, k, x.dtype), dtype=torch.uint8,
                         device=DEV)
        args = [x.data_ptr(), router.data_ptr(), B.MOE_BF16, *(t.data_ptr() for p in w for t in p), T,
                E, H, I, k, 1, out.data_ptr(), None, None, ws.data_ptr(), ws.numel(), None]
        call = B.lib().moe_mx4_forward_tokens

        def job(kept=(x, out, ws)):
            for _ in range(4000):
                status = call(*args)
                assert status == 0, B.STATUS[status]
        return job

    assert not together(many(1, 1), many(9, 2), many(40, 4))


def test_first_call_of_a_thread():
    """A thread that has not used CUDA yet, and is given all the memory: the call makes the context
    current by itself."""
    E, H, I = 4, 256, 256
    w = weights(E, H, I, 3)
    x = torch.randn(5, H, device=DEV).bfloat16()
    router = torch.randn(E, H, device=DEV).bfloat16()
    codes, scales = moe.moe_mx4_quantize(x)
    ws = torch.empty(moe.mx4_tokens_workspace_bytes(5, E, H, I, 2, x.dtype), dtype=torch.uint8,
                     device=DEV)
    for call, out in (
            (lambda o: moe.moe_mx4_product(codes, scales, codes, scales, out=o, ws=ws),
             torch.empty(5, 5, dtype=torch.bfloat16, device=DEV)),
            (lambda o: moe.moe_mx4_forward_tokens(x, router, *w, top_k=2, out=o, ws=ws),
             torch.empty_like(x))):
        want = call(torch.empty_like(out))
        assert not together(lambda: call(out))
        assert torch.equal(out, want)


def block_users(make, given):
    """Calls make() with the side stream while the current one still has work queued on memory that it
    has already given back, as much as each buffer of the call; the result, once all of it is done."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(20_000_000)
    for n in given:
        torch.empty(n, dtype=torch.uint8, device=DEV).fill_(255)
    got = make(side)
    torch.cuda.synchronize()
    return got


def test_a_given_streams_memory_is_its_own():
    """Results and workspace of a call on a given stream do not lie in memory that the current stream's
    queued work still writes."""
    E, H, I = 4, 256, 384
    w = weights(E, H, I, 5)
    g = torch.Generator(device=DEV)
    g.manual_seed(6)
    x = torch.randn(8, H, generator=g, device=DEV).bfloat16()
    router = (torch.randn(E, H, generator=g, device=DEV) * H ** -0.5).bfloat16()
    rows = torch.randn(E * 300, H, generator=g, device=DEV).bfloat16()
    off = torch.arange(E + 1, device=DEV, dtype=torch.int32) * 300
    codes, scales = moe.moe_mx4_quantize(rows)
    ws_rows = moe.mx4_experts_workspace_bytes(E * 300, H, I)
    ws_x = moe.mx4_tokens_workspace_bytes(8, E, H, I, 2, x.dtype)
    jobs = [
        (lambda s: moe.moe_mx4_forward_tokens(x, router, *w, top_k=2, stream=s), (ws_x, 8 * H * 2)),
        (lambda s: moe.moe_mx4_experts_forward_dispatched(rows, off, *w, stream=s),
         (ws_rows, rows.numel() * 2)),
        (lambda s: moe.moe_mx4_product(codes, scales, codes, scales, stream=s),
         (256, rows.shape[0] ** 2 * 2)),
        (lambda s: moe.moe_mx4_dequantize(codes, scales, H, stream=s), (rows.numel() * 2,)),
        (lambda s: torch.cat([t.view(-1) for t in moe.moe_mx4_quantize(rows, stream=s)]),
         (codes.numel(), scales.numel())),
    ]
    for make, given in jobs:
        want = make(None)
        torch.cuda.synchronize()
        got = block_users(make, given)
        assert torch.equal(got, want)


def test_the_examples_prompt_and_steps_choose_the_same_experts():
    """Tokens of a prompt and the same tokens a few at a time: routed alike, so apart by no more than the
    four bits of the prompt's activations."""
    from examples import mx4_layer
    E, H, I, k, T = 16, 256, 384, 2, 64
    g = torch.Generator(device=DEV)
    g.manual_seed(9)

    def normal(*s):
        return (torch.randn(*s, generator=g, device=DEV) * s[-1] ** -0.5).bfloat16()

    layer = mx4_layer.Mx4Layer(normal(E, H), normal(E, I, H), normal(E, I, H), normal(E, H, I),
                               normal(64, H), k)
    x = normal(T, H) * 16
    a, b = layer.prompt(x).float(), layer.step(x).float()
    # a token of other experts would be off by as much as it is large
    off = (a - b).norm(dim=1) / b.norm(dim=1)
    assert off.max() < 0.5
