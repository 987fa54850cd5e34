"""The microscaled 4-bit entry points without a GPU: exports, sizes and refusals on the host."""
import pytest

from mixture_experts_routing_moe_gb300 import binding as B
from mixture_experts_routing_moe_gb300 import build as build_mod


@pytest.fixture(scope="module")
def L():
    build_mod.build()
    return B.lib()


FAKE = 0x10000  # never dereferenced: every call below is rejected first
F32, F16, BF16 = B.MOE_F32, B.MOE_F16, B.MOE_BF16


def test_exports_every_header_function(L):
    names = [n for n in B.header_functions(B.MX4_HEADER) if n.startswith("moe_mx4_")]
    assert set(names) == {n for n in B._SIGS if n.startswith("moe_mx4_")}
    for n in names:
        assert hasattr(L, n), n


@pytest.mark.parametrize("K,codes,scales", [(1, 16, 4), (32, 16, 4), (33, 32, 4), (128, 64, 4),
                                            (129, 80, 8), (7168, 3584, 224)])
def test_row_sizes(L, K, codes, scales):
    assert L.moe_mx4_code_bytes(K) == codes and L.moe_mx4_scale_bytes(K) == scales
    assert B._mx4_pitch(K) == (codes, scales)


def test_row_sizes_out_of_range(L):
    assert L.moe_mx4_code_bytes(0) == 0 and L.moe_mx4_scale_bytes(1 << 24) == 0
    assert L.moe_mx4_experts_workspace_bytes(-1, 64, 64) == 0
    assert L.moe_mx4_experts_workspace_bytes(0, 64, 64) >= 256


def test_quantize_rejects(L):
    def q(x=FAKE, dt=BF16, rows=4, K=64, ld=64, c=FAKE, s=FAKE):
        return L.moe_mx4_quantize(x, dt, rows, K, ld, c, s, None)
    assert q(dt=3) == 3
    assert q(rows=-1) == 2 and q(K=0) == 2 and q(ld=63) == 2 and q(K=1 << 24, ld=1 << 24) == 2
    assert q(rows=1 << 31) == 2
    assert q(x=None) == 1 and q(c=None) == 1 and q(s=None) == 1
    assert q(c=FAKE + 8) == 4 and q(s=FAKE + 2) == 4 and q(x=FAKE + 1) == 4
    assert q(rows=0, x=None, c=None, s=None) == 0


def test_dequantize_rejects(L):
    def d(c=FAKE, s=FAKE, rows=4, K=64, o=FAKE, dt=F16, ld=64):
        return L.moe_mx4_dequantize(c, s, rows, K, o, dt, ld, None)
    assert d(dt=-1) == 3 and d(ld=63) == 2 and d(K=0) == 2 and d(rows=-5) == 2
    assert d(o=None) == 1 and d(c=None) == 1 and d(c=FAKE + 4) == 4 and d(o=FAKE + 1) == 4
    assert d(rows=0, c=None, s=None, o=None) == 0


def test_product_rejects(L):
    def p(a=FAKE, asc=FAKE, rows=8, b=FAKE, bsc=FAKE, off=FAKE, E=2, N=64, K=64, o=FAKE, dt=BF16,
          ws=FAKE, wsb=256):
        return L.moe_mx4_product(a, asc, rows, b, bsc, off, E, N, K, o, dt, ws, wsb, None)
    assert p(dt=9) == 3
    for bad in (dict(rows=-1), dict(rows=1 << 31), dict(E=0), dict(E=1025), dict(N=0), dict(K=0),
                dict(N=1 << 24), dict(E=1024, N=1 << 22), dict(rows=(1 << 31) - 2048, N=1 << 20)):
        assert p(**bad) == 2, bad
    assert p(off=None) == 1 and p(a=None) == 1 and p(bsc=None) == 1 and p(o=None) == 1
    assert p(a=FAKE + 4) == 4 and p(bsc=FAKE + 1) == 4 and p(o=FAKE + 1) == 4 and p(off=FAKE + 2) == 4
    assert p(ws=None) == 5 and p(wsb=255) == 5 and p(ws=FAKE + 128) == 5
    assert p(rows=0, a=None, asc=None, o=None, ws=None) == 0


def test_experts_rejects(L):
    need = L.moe_mx4_experts_workspace_bytes(8, 64, 96)

    def f(x=FAKE, dt=BF16, off=FAKE, rows=8, g=FAKE, gs=FAKE, E=2, H=64, I=96, y=FAKE, ws=FAKE,
          wsb=need):
        return L.moe_mx4_experts_forward_dispatched(x, dt, off, rows, g, gs, FAKE, FAKE, FAKE, FAKE,
                                                    E, H, I, y, ws, wsb, None)
    assert f(dt=8) == 3 and f(H=0) == 2 and f(I=0) == 2 and f(E=0) == 2 and f(rows=-1) == 2
    assert f(x=None) == 1 and f(g=None) == 1 and f(off=None) == 1 and f(y=None) == 1
    assert f(gs=FAKE + 2) == 4 and f(y=FAKE + 1) == 4
    assert f(wsb=need - 1) == 5 and f(ws=FAKE + 16) == 5
    assert f(rows=0, x=None, y=None, ws=None) == 0


def test_tokens_rejects(L):
    need = L.moe_mx4_tokens_workspace_bytes(8, 16, 256, 384, 4, BF16)
    assert need > 256
    assert L.moe_mx4_tokens_workspace_bytes(8, 16, 256, 384, 4, F32) == 0
    assert L.moe_mx4_tokens_workspace_bytes(65, 16, 256, 384, 4, BF16) == 0

    def f(x=FAKE, r=FAKE, dt=BF16, g=FAKE, gs=FAKE, T=8, E=16, H=256, I=384, k=4, out=FAKE,
          idx=None, w=None, ws=FAKE, wsb=need):
        return L.moe_mx4_forward_tokens(x, r, dt, g, gs, FAKE, FAKE, FAKE, FAKE, T, E, H, I, k, 1,
                                        out, idx, w, ws, wsb, None)
    assert f(dt=F32) == 3 and f(dt=7) == 3
    for bad in (dict(T=-1), dict(T=65), dict(E=0), dict(E=1025), dict(k=0), dict(k=17),
                dict(E=64, k=33), dict(T=64, k=17, E=64), dict(H=0), dict(I=0),
                dict(E=1024, H=1 << 22)):
        assert f(**bad) == 2, bad
    assert f(H=192) == 4 and f(I=448) == 4 and f(x=FAKE + 8) == 4 and f(g=FAKE + 8) == 4
    assert f(idx=FAKE + 2) == 4 and f(w=FAKE + 1) == 4
    for k in ("x", "r", "g", "gs", "out"):
        assert f(**{k: None}) == 1, k
    assert f(ws=None) == 5 and f(wsb=need - 1) == 5 and f(ws=FAKE + 64) == 5
    assert f(T=0, x=None, out=None, ws=None) == 0
