"""The norm's and the grouped softmax router's entry points without a GPU: exports and refusals."""
import math

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
    names = B.header_functions(B.FRONT_HEADER)
    assert set(names) - set(B.header_functions()) == {
        "moe_rms_norm", "moe_rms_norm_backward", "moe_rms_norm_backward_workspace_bytes",
        "moe_route_softmax_grouped", "moe_forward_softmax_grouped"}
    for n in names:
        assert hasattr(L, n) and n in B._SIGS, n


def test_norm_rejects(L):
    def n(x=FAKE, ldx=64, r=FAKE, ldr=64, w=FAKE, wdt=F32, dt=BF16, T=4, H=64, eps=1e-6, s=FAKE, lds=64,
          y=FAKE, ldy=64, c=FAKE, sc=FAKE, rstd=FAKE):
        return L.moe_rms_norm(x, ldx, r, ldr, w, wdt, dt, T, H, eps, s, lds, y, ldy, c, sc, rstd, None)
    assert n(dt=3) == 3 and n(wdt=F16) == 3 and n(wdt=7) == 3
    assert n(T=-1) == 2 and n(T=1 << 31) == 2 and n(H=0) == 2 and n(H=1 << 24) == 2
    assert n(ldx=63) == 2 and n(ldr=63) == 2 and n(lds=1) == 2 and n(ldy=0) == 2 and n(ldx=1 << 31) == 2
    assert n(eps=-1e-9) == 9 and n(eps=math.nan) == 9 and n(eps=math.inf) == 9
    assert n(x=None) == 1 and n(w=None) == 1 and n(c=None) == 1 and n(sc=None) == 1
    assert n(x=FAKE + 1) == 4 and n(r=FAKE + 1) == 4 and n(w=FAKE + 2) == 4 and n(c=FAKE + 8) == 4
    assert n(sc=FAKE + 2) == 4 and n(rstd=FAKE + 2) == 4 and n(s=FAKE + 1) == 4 and n(y=FAKE + 1) == 4
    assert n(T=0, x=None, w=None) == 0


def test_norm_backward_rejects(L):
    need = L.moe_rms_norm_backward_workspace_bytes(4, 64, BF16)
    assert need >= 256 + 4 * 64 and L.moe_rms_norm_backward_workspace_bytes(0, 64, BF16) >= 256
    assert L.moe_rms_norm_backward_workspace_bytes(4, 0, BF16) == 0
    assert L.moe_rms_norm_backward_workspace_bytes(4, 64, 3) == 0

    def b(dy=FAKE, lddy=64, s=FAKE, lds=64, w=FAKE, wdt=BF16, rstd=FAKE, ds=FAKE, ldds=64, dt=BF16, T=4,
          H=64, dx=FAKE, lddx=64, dw=FAKE, ws=FAKE, wsb=need):
        return L.moe_rms_norm_backward(dy, lddy, s, lds, w, wdt, rstd, ds, ldds, dt, T, H, dx, lddx, dw,
                                       ws, wsb, None)
    assert b(dt=3) == 3 and b(wdt=F16) == 3
    assert b(T=-1) == 2 and b(H=0) == 2 and b(lddy=63) == 2 and b(lds=63) == 2 and b(ldds=3) == 2
    assert b(lddx=63) == 2
    assert b(dy=None) == 1 and b(s=None) == 1 and b(w=None) == 1 and b(rstd=None) == 1
    assert b(dy=FAKE + 1) == 4 and b(dx=FAKE + 1) == 4 and b(dw=FAKE + 2) == 4 and b(rstd=FAKE + 1) == 4
    assert b(wsb=need - 1) == 5 and b(ws=None) == 5 and b(ws=FAKE + 16) == 5
    assert b(T=0, dw=None, dy=None, ws=None) == 0
    assert b(dx=None, dw=None, ws=None, wsb=0) == 0          # nothing asked for


def test_route_rejects(L):
    def r(l=FAKE, dt=BF16, T=4, E=64, k=4, G=8, SG=4, two=1, scale=1.0, idx=FAKE, w=FAKE):
        return L.moe_route_softmax_grouped(l, dt, None, T, E, k, G, SG, two, 1, scale, idx, w, None)
    assert r(dt=3) == 3
    assert r(T=-1) == 2 and r(E=0) == 2 and r(E=1025) == 2 and r(G=7) == 2 and r(G=0) == 2
    assert r(SG=0) == 2 and r(SG=9) == 2 and r(k=0) == 2 and r(k=65) == 2 and r(k=33) == 2
    assert r(G=64, SG=64) == 2                                # sums of two need two in a group
    assert r(E=256, G=256, two=0) == 2                        # more than 128 groups
    assert r(T=1 << 29, k=8) == 2
    assert r(scale=0.0) == 9 and r(scale=-1.0) == 9 and r(scale=math.nan) == 9
    assert r(l=None) == 1 and r(idx=None) == 1 and r(w=None) == 1
    assert r(l=FAKE + 1) == 4 and r(w=FAKE + 1) == 4 and r(idx=FAKE + 2) == 4
    assert r(T=0, l=None, idx=None, w=None) == 0


def test_forward_rejects(L):
    need = L.moe_forward_workspace_bytes(4, 64, 64, 64, 4, F32, BF16)

    def f(x=FAKE, l=FAKE, ldt=F32, wdt=BF16, T=4, E=64, H=64, k=4, G=8, SG=4, scale=1.0, out=FAKE,
          ws=FAKE, wsb=need):
        return L.moe_forward_softmax_grouped(x, l, ldt, None, FAKE, FAKE, FAKE, wdt, T, E, H, 64, k, G,
                                             SG, 1, 1, scale, out, ws, wsb, None)
    assert f(ldt=3) == 3 and f(wdt=3) == 3 and f(G=7) == 2 and f(k=33) == 2 and f(scale=0.0) == 9
    assert f(x=None) == 1 and f(l=None) == 1 and f(out=None) == 1
    assert f(H=60) == 4 and f(wsb=need - 1) == 5
    assert f(T=0, x=None, ws=None) == 0
