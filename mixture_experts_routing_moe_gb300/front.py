"""Binding of what stands in front of the experts (include/moe_front.h): the residual norm, its
gradient, and the softmax router with groups.  Argument marshalling only.
"""
from __future__ import annotations

import functools

import torch

from . import binding as B
from .binding import MoeError, _code, _new, _new_ws, _ptr, _stream, lib
from .mx8 import _given, _pitch, _rows, leading, on_current_device, workspace


def _like(t, x, where: str, name: str) -> int:
    """Checks rows of x's type and shape; returns their stride (0 for None)."""
    if t is None:
        return 0
    if t.shape != x.shape or t.dtype != x.dtype:
        raise MoeError(2, f"{where}: {name} is not like x")
    return leading(t, x.shape[-1], where)


def _weight(weight, x, where: str) -> int:
    on_current_device(where, weight)
    if weight.shape != x.shape[-1:]:
        raise MoeError(2, f"{where}: weight is [H]")
    return _code(weight)


def moe_rms_norm(x, weight, eps: float = 1e-6, residual=None, values: bool = True,
                 blocks: bool = False, stats: bool = False, sum=None, y=None, codes=None,
                 scales=None, rstd=None, stream=None):
    """s = x + residual and y = s / rms(s) * weight -> dict of what is asked for: "sum" (with a
    residual), "y" (values), "codes" and "scales" (blocks: y in 8-bit blocks), "rstd" (stats: float32
    [rows], for the backward).  x, residual [..., H], contiguous or two-dimensional with rows a stride
    apart; weight [H] in x's dtype or float32.  `sum` may be x or residual itself, `y` may be x."""
    where = "moe_rms_norm"
    shape = x.shape
    H = shape[-1]
    ldx = leading(x, H, where)
    dt, wdt = _code(x), _weight(weight, x, where)
    ldr = _like(residual, x, where, "residual")
    T, lead, dev = x.numel() // max(H, 1), tuple(shape[:-1]), x.device
    out = {}
    lds = ldy = 0
    if sum is not None:
        lds = _like(sum, x, where, "sum")
    elif residual is not None:
        sum, lds = _new(shape, x.dtype, dev, stream), H
    if sum is not None:
        out["sum"] = sum
    if y is not None:
        ldy = _like(y, x, where, "y")
    elif values:
        y, ldy = _new(shape, x.dtype, dev, stream), H
    if y is not None:
        out["y"] = y
    if blocks or codes is not None or scales is not None:
        pc, ps = _pitch(H)
        codes = _new((*lead, pc), torch.uint8, dev, stream) if codes is None else codes
        scales = _new((*lead, ps), torch.uint8, dev, stream) if scales is None else scales
        if _rows(codes, scales, H, where)[:-1] != shape[:-1]:
            raise MoeError(2, f"{where}: codes have other rows than x")
        out["codes"], out["scales"] = codes, scales
    if rstd is not None:
        _given(rstd, lead, torch.float32, where, "rstd")
    elif stats:
        rstd = _new(lead, torch.float32, dev, stream)
    if rstd is not None:
        out["rstd"] = rstd
    B._check(lib().moe_rms_norm(x.data_ptr(), ldx, _ptr(residual), ldr, weight.data_ptr(), wdt, dt, T,
                                H, eps, _ptr(sum), lds, _ptr(y), ldy, _ptr(codes), _ptr(scales),
                                _ptr(rstd), _stream(stream)), where)
    return out


@functools.lru_cache(maxsize=4096)
def rms_norm_backward_workspace_bytes(T: int, H: int, dtype) -> int:
    return lib().moe_rms_norm_backward_workspace_bytes(T, H, B.DTYPE_CODE.get(dtype, -1))


def moe_rms_norm_backward(dy, s, weight, rstd, dsum=None, dx=None, dweight=None, ws=None,
                          stream=None):
    """The gradient of moe_rms_norm's y (dy) and sum (dsum, if any) -> (dx, like dy, of x and of the
    residual alike; dweight float32 [H]).  s: the forward's sum (x without a residual); rstd: its
    stats.  dx may be dy or dsum itself."""
    where = "moe_rms_norm_backward"
    H = dy.shape[-1]
    lddy = leading(dy, H, where)
    dt, wdt = _code(dy), _weight(weight, dy, where)
    lds, ldds = _like(s, dy, where, "s"), _like(dsum, dy, where, "dsum")
    T = dy.numel() // max(H, 1)
    _given(rstd, dy.shape[:-1], torch.float32, where, "rstd")
    if dx is None:
        dx, lddx = _new(dy.shape, dy.dtype, dy.device, stream), H
    else:
        lddx = _like(dx, dy, where, "dx")
    if dweight is None:
        dweight = _new((H,), torch.float32, dy.device, stream)
    else:
        _given(dweight, (H,), torch.float32, where, "dweight")
    h = _stream(stream)
    ws = workspace(ws, rms_norm_backward_workspace_bytes(T, H, dy.dtype), dy.device, stream, h, where)
    B._check(lib().moe_rms_norm_backward(dy.data_ptr(), lddy, s.data_ptr(), lds, weight.data_ptr(),
                                         wdt, rstd.data_ptr(), _ptr(dsum), ldds, dt, T, H,
                                         dx.data_ptr(), lddx, dweight.data_ptr(), ws.data_ptr(),
                                         ws.numel(), h), where)
    return dx, dweight


def _bias(bias, E: int, where: str):
    if bias is None:
        return None
    on_current_device(where, bias)
    if bias.dtype != torch.float32 or bias.shape != (E,):
        raise MoeError(3 if bias.dtype != torch.float32 else 2, f"{where}: bias is float32 [E]")
    return bias.data_ptr()


def moe_route_softmax_grouped(logits, top_k: int, groups: int, selected_groups: int,
                              group_top_two: bool = True, renormalize: bool = True,
                              scale: float = 1.0, bias=None, idx=None, w=None, stream=None):
    """moe_route_sigmoid_grouped with softmax scores -> (idx uint32 [T, k], w [T, k])."""
    where = "moe_route_softmax_grouped"
    on_current_device(where, logits)
    T, E = logits.shape
    b = _bias(bias, E, where)
    if idx is None:
        idx = _new((T, top_k), torch.uint32, logits.device, stream)
    else:
        _given(idx, (T, top_k), torch.uint32, where, "idx")
    if w is None:
        w = _new((T, top_k), logits.dtype, logits.device, stream)
    else:
        _given(w, (T, top_k), logits.dtype, where, "w")
    B._check(lib().moe_route_softmax_grouped(
        logits.data_ptr(), _code(logits), b, T, E, top_k, groups, selected_groups,
        int(bool(group_top_two)), int(bool(renormalize)), float(scale), idx.data_ptr(), w.data_ptr(),
        _stream(stream)), where)
    return idx, w


def moe_forward_softmax_grouped(x, logits, gate, up, down, top_k: int, groups: int,
                                selected_groups: int, group_top_two: bool = True,
                                renormalize: bool = True, scale: float = 1.0, bias=None, out=None,
                                ws=None, stream=None):
    """moe_forward with moe_route_softmax_grouped's router -> out [T, H]."""
    where = "moe_forward_softmax_grouped"
    on_current_device(where, x, logits, gate, up, down)
    T, H = x.shape
    E, I, _ = gate.shape
    if logits.shape != (T, E) or gate.shape != (E, I, H) or up.shape != gate.shape or \
            down.shape != (E, H, I) or not x.dtype == gate.dtype == up.dtype == down.dtype:
        raise MoeError(2, f"{where}: x, logits and the expert weights do not belong together")
    b = _bias(bias, E, where)
    if out is None:
        out = _new(x.shape, x.dtype, x.device, stream)
    else:
        _given(out, x.shape, x.dtype, where, "out")
    if ws is None:
        ws = _new_ws(B.forward_workspace_bytes(T, E, H, I, top_k, logits.dtype, x.dtype), x.device,
                     stream)
    on_current_device(where, ws)
    B._check(lib().moe_forward_softmax_grouped(
        x.data_ptr(), logits.data_ptr(), _code(logits), b, gate.data_ptr(), up.data_ptr(),
        down.data_ptr(), _code(gate), T, E, H, I, top_k, groups, selected_groups,
        int(bool(group_top_two)), int(bool(renormalize)), float(scale), out.data_ptr(),
        ws.data_ptr(), ws.numel(), _stream(stream)), where)
    return out
