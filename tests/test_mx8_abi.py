"""The microscaled 8-bit entry points without a GPU: exports, sizes and refusals on the host."""
import pytest

from mixture_experts_routing_moe_gb300 import binding as B
from mixture_experts_routing_moe_gb300 import build as build_mod
from mixture_experts_routing_moe_gb300 import mx8


@pytest.fixture(scope="module")
def L():
    build_mod.build()
    return B.lib()


FAKE = 0x10000  # never dereferenced: every call below is rejected first
F32, F16, BF16 = B.MOE_F32, B.MOE_F16, B.MOE_BF16


def test_exports_every_header_function(L):
    names = [n for n in B.header_functions(B.MX8_HEADER) if n.startswith("moe_mx8_")]
    assert set(names) == {n for n in B._SIGS if n.startswith("moe_mx8_")}
    for n in names:
        assert hasattr(L, n), n


@pytest.mark.parametrize("K,codes,scales", [(1, 32, 4), (32, 32, 4), (33, 64, 4), (128, 128, 4),
                                            (129, 160, 8), (7168, 7168, 224)])
def test_row_sizes(L, K, codes, scales):
    assert L.moe_mx8_code_bytes(K) == codes and L.moe_mx8_scale_bytes(K) == scales
    assert mx8._pitch(K) == (codes, scales)


def test_sizes_out_of_range(L):
    assert L.moe_mx8_code_bytes(0) == 0 and L.moe_mx8_scale_bytes(1 << 24) == 0
    assert L.moe_mx8_experts_workspace_bytes(-1, 64) == 0
    assert L.moe_mx8_experts_workspace_bytes(4, 0) == 0
    assert L.moe_mx8_experts_workspace_bytes(0, 64) >= 256
    assert L.moe_mx8_product_workspace_bytes() == 256
    f = L.moe_mx8_forward_workspace_bytes
    assert f(4, 8, 64, 64, 2, BF16) > 256
    assert f(4, 8, 64, 64, 9, BF16) == 0 and f(4, 8, 64, 64, 2, 7) == 0 and f(-1, 8, 64, 64, 2, BF16) == 0
    assert f(1 << 30, 8, 64, 64, 2, BF16) == 0 and f(4, 1025, 64, 64, 2, BF16) == 0


def test_quantize_rejects(L):
    def q(x=FAKE, dt=BF16, rows=4, K=64, ld=64, c=FAKE, s=FAKE):
        return L.moe_mx8_quantize(x, dt, rows, K, ld, c, s, None)
    assert q(dt=3) == 3
    assert q(rows=-1) == 2 and q(K=0) == 2 and q(ld=63) == 2 and q(K=1 << 24, ld=1 << 24) == 2
    assert q(rows=1 << 31) == 2 and q(ld=1 << 31) == 2
    assert q(x=None) == 1 and q(c=None) == 1 and q(s=None) == 1
    assert q(c=FAKE + 8) == 4 and q(s=FAKE + 2) == 4 and q(x=FAKE + 1) == 4
    assert q(rows=0, x=None, c=None, s=None) == 0


def test_dequantize_rejects(L):
    def d(c=FAKE, s=FAKE, rows=4, K=64, o=FAKE, dt=F16, ld=64):
        return L.moe_mx8_dequantize(c, s, rows, K, o, dt, ld, None)
    assert d(dt=-1) == 3 and d(ld=63) == 2 and d(K=0) == 2 and d(rows=-5) == 2
    assert d(o=None) == 1 and d(c=None) == 1 and d(c=FAKE + 4) == 4 and d(o=FAKE + 1) == 4
    assert d(rows=0, c=None, s=None, o=None) == 0


def test_dispatch_rejects(L):
    need = L.moe_dispatch_workspace_bytes(8, 4, 2)

    def d(c=FAKE, s=FAKE, T=8, H=64, idx=FAKE, E=4, k=2, xc=FAKE, xs=FAKE, off=FAKE, tor=FAKE,
          ros=FAKE, ws=FAKE, wsb=need):
        return L.moe_mx8_dispatch(c, s, T, H, idx, E, k, xc, xs, off, tor, ros, ws, wsb, None)
    assert d(T=-1) == 2 and d(H=0) == 2 and d(E=0) == 2 and d(E=1025) == 2 and d(k=5) == 2
    assert d(k=0) == 2 and d(T=1 << 30) == 2
    assert d(c=None) == 1 and d(xs=None) == 1 and d(idx=None) == 1 and d(off=None) == 1
    assert d(tor=None) == 1 and d(ros=None) == 1
    assert d(c=FAKE + 8) == 4 and d(xc=FAKE + 4) == 4 and d(xs=FAKE + 1) == 4 and d(idx=FAKE + 2) == 4
    assert d(ws=None) == 5 and d(wsb=need - 1) == 5 and d(ws=FAKE + 8) == 5
    assert d(T=0, c=None, idx=None, ws=None) == 0


def test_product_rejects(L):
    def p(a=FAKE, asc=FAKE, rows=8, b=FAKE, bsc=FAKE, off=FAKE, E=2, N=64, K=64, o=FAKE, dt=BF16,
          ws=FAKE, wsb=256):
        return L.moe_mx8_product(a, asc, rows, b, bsc, off, E, N, K, o, dt, ws, wsb, None)
    assert p(dt=4) == 3
    assert p(rows=-1) == 2 and p(N=0) == 2 and p(K=1 << 24) == 2 and p(E=1025) == 2
    assert p(E=1024, N=(1 << 21)) == 2
    assert p(off=None) == 1 and p(a=None) == 1 and p(bsc=None) == 1 and p(o=None) == 1
    assert p(a=FAKE + 8) == 4 and p(bsc=FAKE + 2) == 4 and p(o=FAKE + 1) == 4 and p(off=FAKE + 2) == 4
    assert p(ws=None) == 5 and p(wsb=255) == 5 and p(ws=FAKE + 128) == 5
    assert p(rows=0, a=None, asc=None, o=None) == 0


def test_experts_rejects(L):
    need = L.moe_mx8_experts_workspace_bytes(8, 96)

    def x(xc=FAKE, xs=FAKE, off=FAKE, rows=8, g=FAKE, u=FAKE, d=FAKE, E=2, H=64, I=96, y=FAKE, dt=BF16,
          ws=FAKE, wsb=need):
        return L.moe_mx8_experts_forward_dispatched(xc, xs, off, rows, g, FAKE, u, FAKE, d, FAKE, E, H,
                                                    I, y, dt, ws, wsb, None)
    assert x(dt=5) == 3 and x(rows=-1) == 2 and x(H=0) == 2 and x(I=1 << 24) == 2 and x(E=0) == 2
    assert x(xc=None) == 1 and x(off=None) == 1 and x(u=None) == 1 and x(y=None) == 1
    assert x(g=FAKE + 8) == 4 and x(xs=FAKE + 2) == 4 and x(y=FAKE + 1) == 4
    assert x(wsb=need - 1) == 5 and x(ws=None) == 5
    assert x(rows=0, xc=None, y=None, ws=None) == 0


def test_forward_rejects(L):
    need = L.moe_mx8_forward_workspace_bytes(8, 4, 64, 96, 2, BF16)

    def f(xc=FAKE, xs=FAKE, idx=FAKE, w=FAKE, wdt=F32, g=FAKE, d=FAKE, T=8, E=4, H=64, I=96, k=2,
          o=FAKE, dt=BF16, ws=FAKE, wsb=need):
        return L.moe_mx8_forward(xc, xs, idx, w, wdt, g, FAKE, FAKE, FAKE, d, FAKE, T, E, H, I, k, o,
                                 dt, ws, wsb, None)
    assert f(dt=9) == 3 and f(wdt=9) == 3
    assert f(T=-1) == 2 and f(k=5) == 2 and f(H=0) == 2 and f(E=1025) == 2 and f(T=1 << 30) == 2
    assert f(xc=None) == 1 and f(idx=None) == 1 and f(w=None) == 1 and f(o=None) == 1 and f(d=None) == 1
    assert f(xc=FAKE + 8) == 4 and f(w=FAKE + 2) == 4 and f(o=FAKE + 1) == 4 and f(idx=FAKE + 1) == 4
    assert f(wsb=need - 1) == 5 and f(ws=FAKE + 64) == 5
    assert f(T=0, xc=None, idx=None, ws=None) == 0
