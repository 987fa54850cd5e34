"""Binding of the microscaled 8-bit (MXFP8) operators (include/moe_mx8.h).  Argument marshalling only.

Rows in blocks are a pair (codes uint8 [..., 32 ceil(K/32)], scales uint8 [..., 4 ceil(K/128)]).
Outputs and workspaces are allocated as in `binding`: on the stream that the call is given.
"""
from __future__ import annotations

import functools

import torch

from . import binding as B
from .binding import DTYPE_CODE, MoeError, _code, _mx4_leading, _mx4_ws, _new, _new_ws, _stream, lib

_u8 = torch.uint8


@functools.lru_cache(maxsize=4096)
def _pitch(K: int):
    """(bytes of codes, bytes of scales) of a row of K values."""
    blocks = -(-K // 32)
    return 32 * blocks, -(-blocks // 4) * 4


@functools.lru_cache(maxsize=4096)
def _scale_shape(shape, K: int):
    """The shape of the scales that go with codes of a shape; None if those are not rows of K."""
    pc, ps = _pitch(K)
    return (*shape[:-1], ps) if len(shape) and shape[-1] == pc else None


def _dtype(dtype, where: str) -> int:
    code = DTYPE_CODE.get(dtype)
    if code is None:
        raise MoeError(3, f"{where}: dtype {dtype}")
    return code


# Small calls take a few microseconds on the GPU, so the checks keep to the attributes they need.
def on_current_device(where: str, *ts):
    """Kernels are launched on the current device: refuses what is not a contiguous tensor there."""
    dev = torch._C._cuda_getDevice()
    for t in ts:
        if t is not None and (t.get_device() != dev or not t.is_contiguous()):
            refuse(where, t, dev)


def refuse(where: str, t, dev: int):
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("libmoe takes contiguous CUDA tensors")
    raise ValueError(f"{where}: a tensor is on {t.device}, the current device is cuda:{dev}")


def leading(t, K: int, where: str) -> int:
    """Elements from one row of K consecutive values to the next, of a tensor on the current device."""
    dev = torch._C._cuda_getDevice()
    if t.get_device() != dev:
        if not t.is_cuda:
            raise ValueError(f"{where} takes CUDA rows of consecutive values")
        refuse(where, t, dev)
    return K if t.is_contiguous() else _mx4_leading(t, K, where)


def _rows(codes, scales, K: int, where: str):
    """Checks one operand in blocks, [..., rows] rows of K values; returns the shape of codes."""
    on_current_device(where, codes, scales)
    if codes.dtype is not _u8 or scales.dtype is not _u8:
        raise MoeError(3, f"{where}: codes and scales are uint8")
    shape = codes.shape
    if scales.shape != _scale_shape(shape, K):
        raise MoeError(2, f"{where}: rows of {K} values have {_pitch(K)} bytes of codes and scales")
    return shape


def _offsets(offsets, E: int, where: str):
    on_current_device(where, offsets)
    if offsets.dtype != torch.int32 or offsets.numel() != E + 1:
        raise MoeError(2, f"{where}: offsets are int32 [E + 1]")
    return offsets.data_ptr()


def _given(t, shape, dtype, where: str, name: str):
    """Checks an output that the caller gave."""
    on_current_device(where, t)
    if t.shape != shape or t.dtype != dtype:
        raise MoeError(2, f"{where}: {name} is {dtype} {tuple(shape)}")
    return t


def moe_mx8_quantize(x, codes=None, scales=None, stream=None):
    """Rows of x [..., K] to blocks -> (codes, scales).  x is contiguous, or two-dimensional with rows
    a stride apart."""
    where = "moe_mx8_quantize"
    shape = x.shape
    K = shape[-1]
    ld = leading(x, K, where)
    dt = _code(x)
    pc, ps = _pitch(K)
    lead = tuple(shape[:-1])
    codes = _new((*lead, pc), _u8, x.device, stream) if codes is None else codes
    scales = _new((*lead, ps), _u8, x.device, stream) if scales is None else scales
    if _rows(codes, scales, K, where)[:-1] != shape[:-1]:
        raise MoeError(2, f"{where}: codes have other rows than x")
    B._check(lib().moe_mx8_quantize(x.data_ptr(), dt, x.numel() // max(K, 1), K, ld,
                                    codes.data_ptr(), scales.data_ptr(), _stream(stream)), where)
    return codes, scales


def moe_mx8_dequantize(codes, scales, K: int, dtype=torch.bfloat16, out=None, stream=None):
    """The values of rows of K values in blocks -> out [..., K] of dtype."""
    where = "moe_mx8_dequantize"
    shape = _rows(codes, scales, K, where)
    if out is None:
        dt, ld = _dtype(dtype, where), K
        out = _new((*shape[:-1], K), dtype, codes.device, stream)
    else:
        if out.shape != (*shape[:-1], K):
            raise MoeError(2, f"{where}: out has another shape")
        dt, ld = _code(out), leading(out, K, where)
    B._check(lib().moe_mx8_dequantize(codes.data_ptr(), scales.data_ptr(),
                                      out.numel() // max(K, 1), K, out.data_ptr(), dt, ld,
                                      _stream(stream)), where)
    return out


def workspace(ws, need: int, device, stream, handle: int, where: str):
    """The caller's workspace, or one as the 4-bit operators keep them."""
    if ws is not None:
        on_current_device(where, ws)
        return ws
    return _mx4_ws(None, need if need > 256 else 256, device, stream, handle)


def _idx(idx, T: int, where: str) -> int:
    on_current_device(where, idx)
    if idx.dtype != torch.uint32 or idx.dim() != 2 or idx.shape[0] != T:
        raise MoeError(2, f"{where}: idx is uint32 [T, top_k]")
    return idx.shape[1]


def moe_mx8_dispatch(codes, scales, idx, E: int, H: int, ws=None, stream=None):
    """moe_dispatch of T tokens in blocks -> dict(codes, scales, offsets, token_of_row, row_of_slot,
    ws)."""
    where = "moe_mx8_dispatch"
    shape = _rows(codes, scales, H, where)
    if len(shape) != 2:
        raise MoeError(2, f"{where}: tokens are [T, bytes]")
    T = shape[0]
    k = _idx(idx, T, where)
    R, dev = T * k, codes.device
    out = {"codes": _new((R, shape[1]), _u8, dev, stream),
           "scales": _new((R, scales.shape[1]), _u8, dev, stream),
           "offsets": _new(E + 1, torch.int32, dev, stream),
           "token_of_row": _new(R, torch.uint32, dev, stream),
           "row_of_slot": _new(R, torch.uint32, dev, stream)}
    if ws is None:
        ws = _new_ws(B.dispatch_workspace_bytes(T, E, k), dev, stream)
    on_current_device(where, ws)
    B._check(lib().moe_mx8_dispatch(codes.data_ptr(), scales.data_ptr(), T, H, idx.data_ptr(), E, k,
                                    *(t.data_ptr() for t in out.values()), ws.data_ptr(),
                                    ws.numel(), _stream(stream)), where)
    if T == 0:
        B._no_rows(out["offsets"], stream)
    return {**out, "ws": ws}


def moe_mx8_product(a_codes, a_scales, b_codes, b_scales, offsets=None, dtype=torch.bfloat16,
                    out=None, ws=None, stream=None):
    """A [rows] times B [E, N] (or [N]) by groups of rows -> out [rows, N] of dtype.  The rows of A
    and B hold the same number of blocks; offsets int32 [E + 1] on the device, or None for one
    group."""
    where = "moe_mx8_product"
    K = a_codes.shape[-1]
    sa, sb = _rows(a_codes, a_scales, K, where), _rows(b_codes, b_scales, K, where)
    if len(sa) != 2 or len(sb) not in (2, 3):
        raise MoeError(2, f"{where}: A is [rows, bytes], B [N, bytes] or [E, N, bytes]")
    rows, N = sa[0], sb[-2]
    E = sb[0] if len(sb) == 3 else 1
    off = None if offsets is None else _offsets(offsets, E, where)
    if out is None:
        dt = _dtype(dtype, where)
        out = _new((rows, N), dtype, a_codes.device, stream)
    else:
        dt = _code(_given(out, (rows, N), out.dtype, where, "out"))
    s = _stream(stream)
    ws = workspace(ws, 256, out.device, stream, s, where)
    B._check(lib().moe_mx8_product(a_codes.data_ptr(), a_scales.data_ptr(), rows, b_codes.data_ptr(),
                                   b_scales.data_ptr(), off, E, N, K, out.data_ptr(), dt,
                                   ws.data_ptr(), ws.numel(), s), where)
    return out


def _expert_weights(gate, up, down, H: int, where: str):
    """Checks (codes, scales) of gate, up [E, I] rows of H and down [E, H] rows of I -> (E, I)."""
    sg = _rows(*gate, H, where)
    if len(sg) != 3:
        raise MoeError(2, f"{where}: expert weights are [E, rows, bytes]")
    E, I = sg[0], sg[1]
    if _rows(*up, H, where) != sg or _rows(*down, I, where)[:-1] != (E, H):
        raise MoeError(2, f"{where}: gate, up and down do not belong together")
    return E, I


@functools.lru_cache(maxsize=4096)
def mx8_experts_workspace_bytes(rows: int, I: int) -> int:
    return lib().moe_mx8_experts_workspace_bytes(rows, I)


def moe_mx8_experts_forward_dispatched(x, offsets, gate, up, down, dtype=torch.bfloat16, y=None,
                                       ws=None, stream=None):
    """SwiGLU experts over dispatched rows in blocks -> y [rows, H] of dtype.  x: (codes, scales) of
    [rows, H]; gate, up, down: of [E, I, H], [E, I, H] and [E, H, I]."""
    where = "moe_mx8_experts_forward_dispatched"
    H = down[0].shape[-2]
    shape = _rows(*x, H, where)
    if len(shape) != 2:
        raise MoeError(2, f"{where}: x is [rows, bytes]")
    E, I = _expert_weights(gate, up, down, H, where)
    off, rows = _offsets(offsets, E, where), shape[0]
    if y is None:
        dt = _dtype(dtype, where)
        y = _new((rows, H), dtype, x[0].device, stream)
    else:
        dt = _code(_given(y, (rows, H), y.dtype, where, "y"))
    s = _stream(stream)
    ws = workspace(ws, mx8_experts_workspace_bytes(rows, I), y.device, stream, s, where)
    B._check(lib().moe_mx8_experts_forward_dispatched(
        x[0].data_ptr(), x[1].data_ptr(), off, rows, gate[0].data_ptr(), gate[1].data_ptr(),
        up[0].data_ptr(), up[1].data_ptr(), down[0].data_ptr(), down[1].data_ptr(), E, H, I,
        y.data_ptr(), dt, ws.data_ptr(), ws.numel(), s), where)
    return y


@functools.lru_cache(maxsize=4096)
def mx8_forward_workspace_bytes(T: int, E: int, H: int, I: int, top_k: int, dtype) -> int:
    return lib().moe_mx8_forward_workspace_bytes(T, E, H, I, top_k, DTYPE_CODE.get(dtype, -1))


def moe_mx8_forward(x, idx, w, gate, up, down, dtype=torch.bfloat16, out=None, ws=None, stream=None):
    """The layer from routed tokens in blocks on (dispatch, experts, combine) -> out [T, H] of dtype.
    x: (codes, scales) of [T, H]; idx uint32 and w [T, top_k] as the routers give them."""
    where = "moe_mx8_forward"
    H = down[0].shape[-2]
    shape = _rows(*x, H, where)
    if len(shape) != 2:
        raise MoeError(2, f"{where}: x is [T, bytes]")
    T = shape[0]
    k = _idx(idx, T, where)
    on_current_device(where, w)
    if w.shape != idx.shape:
        raise MoeError(2, f"{where}: w is [T, top_k]")
    E, I = _expert_weights(gate, up, down, H, where)
    if out is None:
        dt = _dtype(dtype, where)
        out = _new((T, H), dtype, x[0].device, stream)
    else:
        dt = _code(_given(out, (T, H), out.dtype, where, "out"))
    s = _stream(stream)
    ws = workspace(ws, mx8_forward_workspace_bytes(T, E, H, I, k, out.dtype), out.device, stream, s,
                   where)
    B._check(lib().moe_mx8_forward(
        x[0].data_ptr(), x[1].data_ptr(), idx.data_ptr(), w.data_ptr(), _code(w),
        gate[0].data_ptr(), gate[1].data_ptr(), up[0].data_ptr(), up[1].data_ptr(),
        down[0].data_ptr(), down[1].data_ptr(), T, E, H, I, k, out.data_ptr(), dt, ws.data_ptr(),
        ws.numel(), s), where)
    return out
