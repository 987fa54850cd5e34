"""ctypes binding of libmoe (include/moe.h).  Argument marshalling only.

Every function here takes torch CUDA tensors, checks that they are contiguous CUDA tensors,
allocates missing outputs / workspace with torch (device memory is the one thing torch is used
for) on the stream that the call is given (the current one by default), and passes raw pointers,
sizes and that stream to the C ABI.  All computation runs in libmoe's kernels; there is no CPU path.
A missing or unbuilt library raises at first use.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "moe.h")
MX4_HEADER = os.path.join(os.path.dirname(_HERE), "include", "moe_mx4.h")
MX8_HEADER = os.path.join(os.path.dirname(_HERE), "include", "moe_mx8.h")
FRONT_HEADER = os.path.join(os.path.dirname(_HERE), "include", "moe_front.h")

MOE_F32, MOE_F16, MOE_BF16 = 0, 1, 2
DTYPE_CODE = {torch.float32: MOE_F32, torch.float16: MOE_F16, torch.bfloat16: MOE_BF16}
STATUS = {0: "MOE_OK", 1: "MOE_ERR_NULL", 2: "MOE_ERR_SHAPE", 3: "MOE_ERR_DTYPE",
          4: "MOE_ERR_ALIGN", 5: "MOE_ERR_WORKSPACE", 6: "MOE_ERR_CUDA", 7: "MOE_ERR_TIMEOUT",
          8: "MOE_ERR_INDEX", 9: "MOE_ERR_ARG"}

_i64, _int, _sz, _vp = ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p
_f32 = ctypes.c_float
_SIGS = {
    "moe_abi_version": (_int, []),
    "moe_status_string": (ctypes.c_char_p, [_int]),
    "moe_route": (_int, [_vp, _int, _i64, _i64, _int, _int, _vp, _vp, _vp]),
    "moe_route_sigmoid_grouped": (_int, [_vp, _int, _vp, _i64, _i64, _int, _int, _int, _int, _int,
                                         _f32, _vp, _vp, _vp]),
    "moe_selected_router_weights": (_int, [_vp, _int, _vp, _int, _i64, _i64, _int, _int, _int,
                                           _f32, _vp, _vp]),
    "moe_selected_router_backward": (_int, [_vp, _int, _vp, _int, _vp, _i64, _i64, _int, _int,
                                            _int, _f32, _vp, _vp]),
    "moe_dispatch_workspace_bytes": (_sz, [_i64, _i64, _int]),
    "moe_dispatch": (_int, [_vp, _int, _i64, _i64, _vp, _i64, _int, _vp, _vp, _vp, _vp, _vp, _sz,
                            _vp]),
    "moe_dispatch_static": (_int, [_vp, _int, _i64, _i64, _vp, _i64, _int, _vp, _vp, _vp, _vp,
                                   _vp]),
    "moe_experts_workspace_bytes": (_sz, [_i64, _i64, _i64, _i64, _int]),
    "moe_experts_forward_dispatched": (_int, [_vp, _vp, _i64, _vp, _vp, _vp, _int, _i64, _i64,
                                              _i64, _vp, _vp, _sz, _vp]),
    "moe_combine": (_int, [_vp, _int, _vp, _vp, _int, _i64, _i64, _int, _vp, _vp]),
    "moe_forward_workspace_bytes": (_sz, [_i64, _i64, _i64, _i64, _int, _int, _int]),
    "moe_forward": (_int, [_vp, _vp, _int, _vp, _vp, _vp, _int, _i64, _i64, _i64, _i64, _int, _int,
                           _vp, _vp, _sz, _vp]),
    "moe_forward_sigmoid_grouped": (_int, [_vp, _vp, _int, _vp, _vp, _vp, _vp, _int, _i64, _i64,
                                           _i64, _i64, _int, _int, _int, _int, _int, _f32, _vp,
                                           _vp, _sz, _vp]),
    "moe_forward_with_events": (_int, [_vp, _vp, _int, _vp, _vp, _vp, _int, _i64, _i64, _i64,
                                       _i64, _int, _int, _vp, _vp, _sz, _vp, _vp]),
    "moe_forward_fused": (_int, [_i64, _i64, _i64, _i64, _int, _int, _int]),
    "moe_wait_selftest": (_int, [_vp, _sz, _vp]),
    "moe_combine_backward": (_int, [_vp, _int, _vp, _vp, _int, _vp, _i64, _i64, _int, _vp, _vp,
                                    _vp]),
    "moe_experts_backward_workspace_bytes": (_sz, [_i64, _i64]),
    "moe_experts_backward": (_int, [_vp, _vp, _i64, _vp, _vp, _vp, _int, _i64, _i64, _i64, _vp,
                                    _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "moe_dispatch_backward": (_int, [_vp, _int, _vp, _i64, _i64, _int, _vp, _vp]),
    "moe_device_status": (_int, [_vp, _sz, _vp]),
    "moe_mx4_code_bytes": (_sz, [_i64]),
    "moe_mx4_scale_bytes": (_sz, [_i64]),
    "moe_mx4_quantize": (_int, [_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp]),
    "moe_mx4_dequantize": (_int, [_vp, _vp, _i64, _i64, _vp, _int, _i64, _vp]),
    "moe_mx4_product_workspace_bytes": (_sz, []),
    "moe_mx4_product": (_int, [_vp, _vp, _i64, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _int, _vp,
                               _sz, _vp]),
    "moe_mx4_experts_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "moe_mx4_experts_forward_dispatched": (_int, [_vp, _int, _vp, _i64, _vp, _vp, _vp, _vp, _vp,
                                                  _vp, _i64, _i64, _i64, _vp, _vp, _sz, _vp]),
    "moe_mx4_tokens_workspace_bytes": (_sz, [_i64, _i64, _i64, _i64, _int, _int]),
    "moe_mx4_forward_tokens": (_int, [_vp, _vp, _int, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64,
                                      _i64, _i64, _int, _int, _vp, _vp, _vp, _vp, _sz, _vp]),
    "moe_mx8_code_bytes": (_sz, [_i64]),
    "moe_mx8_scale_bytes": (_sz, [_i64]),
    "moe_mx8_quantize": (_int, [_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp]),
    "moe_mx8_dequantize": (_int, [_vp, _vp, _i64, _i64, _vp, _int, _i64, _vp]),
    "moe_mx8_dispatch": (_int, [_vp, _vp, _i64, _i64, _vp, _i64, _int, _vp, _vp, _vp, _vp, _vp, _vp,
                                _sz, _vp]),
    "moe_mx8_product_workspace_bytes": (_sz, []),
    "moe_mx8_product": (_int, [_vp, _vp, _i64, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _int, _vp,
                               _sz, _vp]),
    "moe_mx8_experts_workspace_bytes": (_sz, [_i64, _i64]),
    "moe_mx8_experts_forward_dispatched": (_int, [_vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp,
                                                  _i64, _i64, _i64, _vp, _int, _vp, _sz, _vp]),
    "moe_mx8_forward_workspace_bytes": (_sz, [_i64, _i64, _i64, _i64, _int, _int]),
    "moe_mx8_forward": (_int, [_vp, _vp, _vp, _vp, _int, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64,
                               _i64, _i64, _int, _vp, _int, _vp, _sz, _vp]),
    "moe_rms_norm": (_int, [_vp, _i64, _vp, _i64, _vp, _int, _int, _i64, _i64, _f32, _vp, _i64, _vp,
                            _i64, _vp, _vp, _vp, _vp]),
    "moe_rms_norm_backward_workspace_bytes": (_sz, [_i64, _i64, _int]),
    "moe_rms_norm_backward": (_int, [_vp, _i64, _vp, _i64, _vp, _int, _vp, _vp, _i64, _int, _i64,
                                     _i64, _vp, _i64, _vp, _vp, _sz, _vp]),
    "moe_route_softmax_grouped": (_int, [_vp, _int, _vp, _i64, _i64, _int, _int, _int, _int, _int,
                                         _f32, _vp, _vp, _vp]),
    "moe_forward_softmax_grouped": (_int, [_vp, _vp, _int, _vp, _vp, _vp, _vp, _int, _i64, _i64,
                                           _i64, _i64, _int, _int, _int, _int, _int, _f32, _vp,
                                           _vp, _sz, _vp]),
}

_lib = None


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} "
                         f"({lib().moe_status_string(status).decode()})")


def lib() -> ctypes.CDLL:
    """The loaded libmoe.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m mixture_experts_routing_moe_gb300.build` (needs nvcc)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _lib = L
    return _lib


def header_functions(header: str = HEADER) -> list[str]:
    """Names of the functions a header (include/moe.h) declares."""
    src = open(header).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return sorted(set(re.findall(r"\b(moe_[a-z_0-9]+)\s*\(", src)))


def _check(st: int, where: str):
    if st != 0:
        raise MoeError(st, where)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    # the current stream's handle without a Stream object around it (3 us a call)
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


def _new(shape, dtype, device, stream):
    """Memory for what a call on `stream` (None: the current one) writes.  It is that stream's own:
    torch may hand out a block of another stream whose queued work still uses it.  The current
    stream counts as a user too, for a result that is freed while it is still read there."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(t.device))
    return t


def _new_ws(need: int, device, stream):
    return _new(max(need, 256), torch.uint8, device, stream)


def _no_rows(offsets, stream):
    """The offsets of a call without tokens, for which the library enqueues nothing."""
    with torch.cuda.stream(stream):
        offsets.zero_()


def _cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("libmoe takes contiguous CUDA tensors")


def _code(t) -> int:
    try:
        return DTYPE_CODE[t.dtype]
    except KeyError:
        raise MoeError(3, f"dtype {t.dtype}") from None


# ------------------------------------------------------------------------------ entry points
def moe_route(logits, top_k: int, renormalize: bool = True, idx=None, w=None, stream=None):
    """route(logits, RoutingOptions{top_k, renormalize}) -> (idx uint32 [T,k], w [T,k])."""
    _cuda(logits)
    T, E = logits.shape
    if idx is None:
        idx = _new((T, top_k), torch.uint32, logits.device, stream)
    if w is None:
        w = _new((T, top_k), logits.dtype, logits.device, stream)
    _cuda(idx, w)
    _check(lib().moe_route(_ptr(logits), _code(logits), T, E, top_k, int(bool(renormalize)),
                           _ptr(idx), _ptr(w), _stream(stream)), "moe_route")
    return idx, w


def moe_route_sigmoid_grouped(logits, top_k: int, groups: int, selected_groups: int,
                              group_top_two: bool = True, renormalize: bool = True,
                              scale: float = 1.0, bias=None, idx=None, w=None, stream=None):
    """route_sigmoid_grouped(logits, bias, GroupRoutingOptions) -> (idx uint32 [T,k], w [T,k])."""
    _cuda(logits, bias)
    if bias is not None and bias.dtype != torch.float32:
        raise MoeError(3, "bias must be float32")
    T, E = logits.shape
    if idx is None:
        idx = _new((T, top_k), torch.uint32, logits.device, stream)
    if w is None:
        w = _new((T, top_k), logits.dtype, logits.device, stream)
    _cuda(idx, w)
    _check(lib().moe_route_sigmoid_grouped(
        _ptr(logits), _code(logits), _ptr(bias), T, E, top_k, groups, selected_groups,
        int(bool(group_top_two)), int(bool(renormalize)), float(scale), _ptr(idx), _ptr(w),
        _stream(stream)), "moe_route_sigmoid_grouped")
    return idx, w


INDEX_CODE = {torch.uint32: 0, torch.int32: 1, torch.int64: 2}
SCORING = {"softmax": 0, "sigmoid": 1}


def moe_selected_router_weights(logits, idx, scoring: str = "softmax", renormalize: bool = True,
                                scale: float = 1.0, w=None, stream=None):
    """selected_router_weights(logits, indices, options) -> FP32 weights [T, k]."""
    _cuda(logits, idx)
    T, E = logits.shape
    k = idx.shape[1]
    w = _new((T, k), torch.float32, logits.device, stream) if w is None else w
    _cuda(w)
    _check(lib().moe_selected_router_weights(
        _ptr(logits), _code(logits), _ptr(idx), INDEX_CODE[idx.dtype], T, E, k, SCORING[scoring],
        int(bool(renormalize)), float(scale), _ptr(w), _stream(stream)),
        "moe_selected_router_weights")
    return w


def moe_selected_router_backward(logits, idx, grad_w, scoring: str = "softmax",
                                 renormalize: bool = True, scale: float = 1.0, grad=None,
                                 stream=None):
    """selected_router_backward(logits, indices, grad_weights, options) -> dL/dlogits [T, E]."""
    _cuda(logits, idx, grad_w)
    if grad_w.dtype != torch.float32:
        raise MoeError(3, "grad_weights must be float32")
    T, E = logits.shape
    k = idx.shape[1]
    grad = _new(logits.shape, logits.dtype, logits.device, stream) if grad is None else grad
    _cuda(grad)
    _check(lib().moe_selected_router_backward(
        _ptr(logits), _code(logits), _ptr(idx), INDEX_CODE[idx.dtype], _ptr(grad_w), T, E, k,
        SCORING[scoring], int(bool(renormalize)), float(scale), _ptr(grad), _stream(stream)),
        "moe_selected_router_backward")
    return grad


def dispatch_workspace_bytes(T: int, E: int, top_k: int) -> int:
    return lib().moe_dispatch_workspace_bytes(T, E, top_k)


def moe_dispatch(x, idx, E: int, x_d=None, offsets=None, token_of_row=None, row_of_slot=None,
                 ws=None, stream=None):
    """RoutingPlan::dispatch -> dict(x_d, offsets, token_of_row, row_of_slot, ws)."""
    _cuda(x, idx)
    T, H = x.shape
    k = idx.shape[1]
    R, dev = T * k, x.device
    x_d = _new((R, H), x.dtype, dev, stream) if x_d is None else x_d
    offsets = _new(E + 1, torch.int32, dev, stream) if offsets is None else offsets
    token_of_row = _new(R, torch.uint32, dev, stream) if token_of_row is None else token_of_row
    row_of_slot = _new(R, torch.uint32, dev, stream) if row_of_slot is None else row_of_slot
    if ws is None:
        ws = _new_ws(dispatch_workspace_bytes(T, E, k), dev, stream)
    _cuda(x_d, offsets, token_of_row, row_of_slot, ws)
    _check(lib().moe_dispatch(_ptr(x), _code(x), T, H, _ptr(idx), E, k, _ptr(x_d), _ptr(offsets),
                              _ptr(token_of_row), _ptr(row_of_slot), _ptr(ws), ws.numel(),
                              _stream(stream)), "moe_dispatch")
    if T == 0:
        _no_rows(offsets, stream)
    return {"x_d": x_d, "offsets": offsets, "token_of_row": token_of_row,
            "row_of_slot": row_of_slot, "ws": ws}


def experts_workspace_bytes(rows: int, E: int, H: int, I: int, dtype) -> int:
    return lib().moe_experts_workspace_bytes(rows, E, H, I, DTYPE_CODE[dtype])


def moe_experts_forward_dispatched(x_d, offsets, gate, up, down, y=None, ws=None, stream=None):
    """SwiGluExperts::forward_dispatched -> y [rows, H]."""
    _cuda(x_d, offsets, gate, up, down)
    rows, H = x_d.shape
    E, I, _ = gate.shape
    y = _new((rows, H), x_d.dtype, x_d.device, stream) if y is None else y
    if ws is None:
        ws = _new_ws(experts_workspace_bytes(rows, E, H, I, gate.dtype), x_d.device, stream)
    _cuda(y, ws)
    _check(lib().moe_experts_forward_dispatched(
        _ptr(x_d), _ptr(offsets), rows, _ptr(gate), _ptr(up), _ptr(down), _code(gate), E, H, I,
        _ptr(y), _ptr(ws), ws.numel(), _stream(stream)), "moe_experts_forward_dispatched")
    return y


def moe_combine(y, row_of_slot, w, out=None, stream=None):
    """DispatchedTokens::combine -> out [T, H] in y's dtype."""
    _cuda(y, row_of_slot, w)
    T, k = w.shape
    H = y.shape[1]
    out = _new((T, H), y.dtype, y.device, stream) if out is None else out
    _cuda(out)
    _check(lib().moe_combine(_ptr(y), _code(y), _ptr(row_of_slot), _ptr(w), _code(w), T, H, k,
                             _ptr(out), _stream(stream)), "moe_combine")
    return out


def forward_workspace_bytes(T, E, H, I, top_k, logits_dtype, dtype) -> int:
    return lib().moe_forward_workspace_bytes(T, E, H, I, top_k, DTYPE_CODE[logits_dtype],
                                             DTYPE_CODE[dtype])


def moe_forward(x, logits, gate, up, down, top_k: int, renormalize: bool = True, out=None,
                ws=None, stream=None):
    """SwiGluExperts::forward(input, logits, options) -> out [T, H]."""
    _cuda(x, logits, gate, up, down)
    T, H = x.shape
    E, I, _ = gate.shape
    out = _new(x.shape, x.dtype, x.device, stream) if out is None else out
    if ws is None:
        ws = _new_ws(forward_workspace_bytes(T, E, H, I, top_k, logits.dtype, x.dtype), x.device,
                     stream)
    _cuda(out, ws)
    _check(lib().moe_forward(_ptr(x), _ptr(logits), _code(logits), _ptr(gate), _ptr(up),
                             _ptr(down), _code(gate), T, E, H, I, top_k, int(bool(renormalize)),
                             _ptr(out), _ptr(ws), ws.numel(), _stream(stream)), "moe_forward")
    return out


def moe_forward_sigmoid_grouped(x, logits, gate, up, down, top_k: int, groups: int,
                                selected_groups: int, group_top_two: bool = True,
                                renormalize: bool = True, scale: float = 1.0, bias=None, out=None,
                                ws=None, stream=None):
    """SwiGluExperts::forward_sigmoid_grouped -> out [T, H]."""
    _cuda(x, logits, gate, up, down, bias)
    T, H = x.shape
    E, I, _ = gate.shape
    out = _new(x.shape, x.dtype, x.device, stream) if out is None else out
    if ws is None:
        ws = _new_ws(forward_workspace_bytes(T, E, H, I, top_k, logits.dtype, x.dtype), x.device,
                     stream)
    _cuda(out, ws)
    _check(lib().moe_forward_sigmoid_grouped(
        _ptr(x), _ptr(logits), _code(logits), _ptr(bias), _ptr(gate), _ptr(up), _ptr(down),
        _code(gate), T, E, H, I, top_k, groups, selected_groups, int(bool(group_top_two)),
        int(bool(renormalize)), float(scale), _ptr(out), _ptr(ws), ws.numel(), _stream(stream)),
        "moe_forward_sigmoid_grouped")
    return out


def moe_forward_fused(T: int, E: int, H: int, I: int, top_k: int, logits_dtype, dtype) -> bool:
    """Whether moe_forward runs these sizes as the single fused launch (aligned tensors)."""
    return bool(lib().moe_forward_fused(T, E, H, I, top_k, DTYPE_CODE[logits_dtype], DTYPE_CODE[dtype]))


def moe_forward_with_events(x, logits, gate, up, down, top_k: int, renormalize: bool, out=None,
                            ws=None, events=None, stream=None):
    """The staged moe_forward (separate launches), recording six torch.cuda.Event objects at the
    stage boundaries (before route / after route / after dispatch / after gate-up / after down /
    after combine) when `events` is given."""
    _cuda(x, logits, gate, up, down)
    T, H = x.shape
    E, I, _ = gate.shape
    out = _new(x.shape, x.dtype, x.device, stream) if out is None else out
    if ws is None:
        ws = _new_ws(forward_workspace_bytes(T, E, H, I, top_k, logits.dtype, x.dtype), x.device,
                     stream)
    _cuda(out, ws)
    arr = None
    if events is not None:
        if len(events) != 6:
            raise ValueError("moe_forward_with_events needs six events")
        for ev in events:
            if ev.cuda_event == 0:      # torch creates the CUDA event on its first record
                ev.record(torch.cuda.current_stream() if stream is None else stream)
        arr = (ctypes.c_void_p * 6)(*[ctypes.c_void_p(ev.cuda_event) for ev in events])
    _check(lib().moe_forward_with_events(
        _ptr(x), _ptr(logits), _code(logits), _ptr(gate), _ptr(up), _ptr(down), _code(gate), T, E,
        H, I, top_k, int(bool(renormalize)), _ptr(out), _ptr(ws), ws.numel(), _stream(stream),
        arr), "moe_forward_with_events")
    return out


def moe_combine_backward(y, row_of_slot, w, dout, stream=None):
    """DispatchedTokens::combine_backward -> (dexpert [T*k, H], dweights [T, k] FP32)."""
    _cuda(y, row_of_slot, w, dout)
    T, k = w.shape
    H = y.shape[1]
    dexpert = _new(y.shape, y.dtype, y.device, stream)
    dweights = _new((T, k), torch.float32, y.device, stream)
    _check(lib().moe_combine_backward(_ptr(y), _code(y), _ptr(row_of_slot), _ptr(w), _code(w),
                                      _ptr(dout), T, H, k, _ptr(dexpert), _ptr(dweights),
                                      _stream(stream)), "moe_combine_backward")
    return dexpert, dweights


def moe_experts_backward(x_d, offsets, gate, up, down, dy, ws=None, stream=None):
    """cache.backward(dexpert) -> (dinput [rows, H], dgate, dup [E, I, H], ddown [E, H, I] FP32)."""
    _cuda(x_d, offsets, gate, up, down, dy)
    rows, H = x_d.shape
    E, I, _ = gate.shape
    dev = x_d.device
    dinput = _new(x_d.shape, x_d.dtype, x_d.device, stream)
    dgate = _new((E, I, H), torch.float32, dev, stream)
    dup = _new((E, I, H), torch.float32, dev, stream)
    ddown = _new((E, H, I), torch.float32, dev, stream)
    if ws is None:
        ws = _new_ws(lib().moe_experts_backward_workspace_bytes(rows, I), dev, stream)
    _check(lib().moe_experts_backward(
        _ptr(x_d), _ptr(offsets), rows, _ptr(gate), _ptr(up), _ptr(down), _code(gate), E, H, I,
        _ptr(dy), _ptr(dinput), _ptr(dgate), _ptr(dup), _ptr(ddown), _ptr(ws), ws.numel(),
        _stream(stream)), "moe_experts_backward")
    return dinput, dgate, dup, ddown


def moe_dispatch_backward(dinput, row_of_slot, T: int, top_k: int, stream=None):
    """DispatchedTokens::dispatch_backward -> dx [T, H] (slot rows summed, no weights)."""
    _cuda(dinput, row_of_slot)
    H = dinput.shape[1]
    dx = _new((T, H), dinput.dtype, dinput.device, stream)
    _check(lib().moe_dispatch_backward(_ptr(dinput), _code(dinput), _ptr(row_of_slot), T, H, top_k,
                                       _ptr(dx), _stream(stream)), "moe_dispatch_backward")
    return dx


def moe_wait_selftest(ws, stream=None) -> None:
    """One bounded wait that nothing completes: the timeout lands in ws's status word."""
    _cuda(ws)
    _check(lib().moe_wait_selftest(_ptr(ws), ws.numel(), _stream(stream)), "moe_wait_selftest")


def moe_device_status(ws, stream=None) -> int:
    """Synchronise, read and clear the workspace status word (0 = MOE_OK)."""
    return lib().moe_device_status(_ptr(ws), ws.numel(), _stream(stream))


# ------------------------------------------------------------- microscaled 4-bit (moe_mx4.h)
# Small calls take a few microseconds on the GPU, so the checks below are kept to the attributes
# they need; sizes that follow from other sizes are remembered.
@functools.lru_cache(maxsize=4096)
def _mx4_pitch(K: int):
    """(bytes of codes, bytes of scales) of a row of K values."""
    blocks = -(-K // 32)
    return 16 * blocks, -(-blocks // 4) * 4


@functools.lru_cache(maxsize=4096)
def _mx4_scale_shape(shape, K: int):
    """The shape of the scales that go with codes of a shape; None if those are not rows of K."""
    pc, ps = _mx4_pitch(K)
    return (*shape[:-1], ps) if len(shape) and shape[-1] == pc else None


_u8, _empty = torch.uint8, torch.empty


def _mx4_rows(codes, scales, K: int, where: str):
    """Checks one operand in blocks, [..., rows] rows of K values; returns the shape of codes."""
    if not (codes.is_cuda and scales.is_cuda and codes.is_contiguous() and scales.is_contiguous()):
        raise ValueError("libmoe takes contiguous CUDA tensors")
    if codes.dtype is not _u8 or scales.dtype is not _u8:
        raise MoeError(3, f"{where}: codes and scales are uint8")
    shape = codes.shape
    if scales.shape != _mx4_scale_shape(shape, K):
        raise MoeError(2, f"{where}: rows of {K} values have {_mx4_pitch(K)} bytes of codes and "
                          "scales")
    return shape


def _mx4_leading(t, K: int, where: str) -> int:
    """Elements from one row of K consecutive values to the next."""
    if t.is_cuda:
        if t.is_contiguous():
            return K
        if t.dim() == 2 and t.stride(1) == 1 and t.stride(0) >= K:
            return t.stride(0)
    raise ValueError(f"{where} takes CUDA rows of consecutive values")


def _mx4_dtype(t) -> int:
    code = DTYPE_CODE.get(t.dtype)
    return _code(t) if code is None else code


# Workspaces of calls that were given none, kept from call to call up to a size.  A call makes
# several launches and the GIL is released while it makes them, so two threads' launches may
# interleave on the stream that they share (all threads start on the default one): each thread has
# buffers of its own, one a stream, and the calls of one thread on one stream follow one another.
# A buffer that is outgrown, or belongs to a thread that ended, goes back to torch, which hands it
# out again behind the work of the stream it was made on (as with any tensor, a stream from outside
# torch has to stay alive until then).
class _Mx4Kept(threading.local):
    """(device, stream handle) -> the calling thread's workspace there."""

    def __init__(self):
        self.of = {}

    def __getitem__(self, key):
        return self.of[key]


_mx4_kept = _Mx4Kept()
# Calls that need more take longer on the device than an allocation takes on the host.
_MX4_KEPT_BYTES = 8 << 20
_MX4_KEPT_STREAMS = 4  # of a thread; the oldest buffer makes room


def _mx4_ws(ws, need: int, device, stream, handle: int):
    """The caller's workspace, or one of at least `need` bytes for a call on stream `handle`
    (`stream`, or the current one if that is None)."""
    if ws is not None:
        _cuda(ws)
        return ws
    # A captured call gets its own: the graph may run beside later calls.
    if stream is None and need <= _MX4_KEPT_BYTES and not torch.cuda.is_current_stream_capturing():
        key, of = (device.index, handle), _mx4_kept.of
        ws = of.get(key)
        if ws is None or ws.numel() < need:
            if ws is None and len(of) >= _MX4_KEPT_STREAMS:
                del of[next(iter(of))]
            ws = of[key] = _empty(need, dtype=_u8, device=device)
        return ws
    return _new(need, _u8, device, stream)


def moe_mx4_quantize(x, codes=None, scales=None, stream=None):
    """Rows of x [..., K] to blocks -> (codes uint8 [..., 16 ceil(K/32)], scales uint8
    [..., 4 ceil(K/128)]).  x is contiguous, or two-dimensional with rows a stride apart."""
    shape = x.shape
    K = shape[-1]
    ld = K if x.is_cuda and x.is_contiguous() else _mx4_leading(x, K, "moe_mx4_quantize")
    dt = DTYPE_CODE.get(x.dtype)
    if dt is None:
        dt = _code(x)  # raises
    given = codes is not None or scales is not None
    if codes is None or scales is None:
        pc, ps = _mx4_pitch(K)
        lead = (shape[0],) if len(shape) == 2 else shape[:-1]
        dev = x.device
        codes = _new((*lead, pc), _u8, dev, stream) if codes is None else codes
        scales = _new((*lead, ps), _u8, dev, stream) if scales is None else scales
    if given and _mx4_rows(codes, scales, K, "moe_mx4_quantize")[:-1] != shape[:-1]:
        raise MoeError(2, "moe_mx4_quantize: codes have other rows than x")
    st = (_lib or lib()).moe_mx4_quantize(
        x.data_ptr(), dt, shape[0] if len(shape) == 2 else x.numel() // max(K, 1), K, ld,
        codes.data_ptr(), scales.data_ptr(), _stream(stream))
    if st:
        raise MoeError(st, "moe_mx4_quantize")
    return codes, scales


def moe_mx4_dequantize(codes, scales, K: int, dtype=torch.bfloat16, out=None, stream=None):
    """The values of rows of K values in blocks -> out [..., K] of dtype."""
    shape = _mx4_rows(codes, scales, K, "moe_mx4_dequantize")
    if out is None:
        lead = (shape[0],) if len(shape) == 2 else shape[:-1]
        out = _new((*lead, K), dtype, codes.device, stream)
        ld = K
    else:
        if out.shape != (*shape[:-1], K):
            raise MoeError(2, "moe_mx4_dequantize: out has another shape")
        ld = _mx4_leading(out, K, "moe_mx4_dequantize")
    dt = DTYPE_CODE.get(out.dtype)
    if dt is None:
        dt = _code(out)  # raises
    st = (_lib or lib()).moe_mx4_dequantize(
        codes.data_ptr(), scales.data_ptr(),
        shape[0] if len(shape) == 2 else out.numel() // max(K, 1), K, out.data_ptr(), dt, ld,
        _stream(stream))
    if st:
        raise MoeError(st, "moe_mx4_dequantize")
    return out


def _mx4_offsets(offsets, E: int, where: str):
    _cuda(offsets)
    if offsets.dtype != torch.int32 or offsets.numel() != E + 1:
        raise MoeError(2, f"{where}: offsets are int32 [E + 1]")
    return offsets.data_ptr()


def moe_mx4_product(a_codes, a_scales, b_codes, b_scales, offsets=None, dtype=torch.bfloat16,
                    out=None, ws=None, stream=None):
    """A [rows] times B [E, N] (or [N]) by groups of rows -> out [rows, N] of dtype.  The rows of A
    and B hold the same number of blocks; offsets int32 [E + 1] on the device, or None for one
    group."""
    where = "moe_mx4_product"
    K = 2 * a_codes.shape[-1]
    sa = _mx4_rows(a_codes, a_scales, K, where)
    sb = _mx4_rows(b_codes, b_scales, K, where)
    if len(sa) != 2 or len(sb) not in (2, 3):
        raise MoeError(2, "moe_mx4_product: A is [rows, bytes], B [N, bytes] or [E, N, bytes]")
    rows, N = sa[0], sb[-2]
    E = sb[0] if len(sb) == 3 else 1
    off = None if offsets is None else _mx4_offsets(offsets, E, where)
    if out is None:
        out = _new((rows, N), dtype, a_codes.device, stream)
    elif out.shape != (rows, N):
        raise MoeError(2, "moe_mx4_product: out has another shape")
    else:
        _cuda(out)
    s = _stream(stream)
    ws = _mx4_ws(ws, 256, out.device, stream, s)
    _check(lib().moe_mx4_product(a_codes.data_ptr(), a_scales.data_ptr(), rows,
                                 b_codes.data_ptr(), b_scales.data_ptr(), off, E, N, K,
                                 out.data_ptr(), _mx4_dtype(out), ws.data_ptr(), ws.numel(), s),
           where)
    return out


def _mx4_expert_weights(gate, up, down, H: int, where: str):
    """Checks (codes, scales) of gate, up [E, I] rows of H and down [E, H] rows of I -> (E, I)."""
    sg = _mx4_rows(*gate, H, where)
    if len(sg) != 3:
        raise MoeError(2, f"{where}: expert weights are [E, rows, bytes]")
    E, I = sg[0], sg[1]
    if _mx4_rows(*up, H, where) != sg or _mx4_rows(*down, I, where)[:-1] != (E, H):
        raise MoeError(2, f"{where}: gate, up and down do not belong together")
    return E, I


@functools.lru_cache(maxsize=4096)
def mx4_experts_workspace_bytes(rows: int, H: int, I: int) -> int:
    return lib().moe_mx4_experts_workspace_bytes(rows, H, I)


def moe_mx4_experts_forward_dispatched(x_d, offsets, gate, up, down, y=None, ws=None,
                                       stream=None):
    """SwiGLU experts with weights and activations in blocks -> y [rows, H] in x_d's dtype.
    gate, up, down: (codes, scales) of [E, I, H], [E, I, H] and [E, H, I]."""
    where = "moe_mx4_experts_forward_dispatched"
    _cuda(x_d)
    rows, H = x_d.shape
    E, I = _mx4_expert_weights(gate, up, down, H, where)
    off = _mx4_offsets(offsets, E, where)
    if y is None:
        y = _new(x_d.shape, x_d.dtype, x_d.device, stream)
    elif y.shape != x_d.shape or y.dtype != x_d.dtype:
        raise MoeError(2, f"{where}: y is not like x_d")
    else:
        _cuda(y)
    s = _stream(stream)
    ws = _mx4_ws(ws, max(mx4_experts_workspace_bytes(rows, H, I), 256), x_d.device, stream, s)
    _check(lib().moe_mx4_experts_forward_dispatched(
        x_d.data_ptr(), _mx4_dtype(x_d), off, rows, gate[0].data_ptr(), gate[1].data_ptr(),
        up[0].data_ptr(), up[1].data_ptr(), down[0].data_ptr(), down[1].data_ptr(), E, H, I,
        y.data_ptr(), ws.data_ptr(), ws.numel(), s), where)
    return y


@functools.lru_cache(maxsize=4096)
def mx4_tokens_workspace_bytes(T: int, E: int, H: int, I: int, top_k: int, dtype) -> int:
    return lib().moe_mx4_tokens_workspace_bytes(T, E, H, I, top_k, DTYPE_CODE.get(dtype, -1))


def moe_mx4_forward_tokens(x, router, gate, up, down, top_k: int, renormalize: bool = True,
                           out=None, idx=None, w=None, ws=None, stream=None):
    """A whole layer for a few tokens (router, top-k, experts in blocks, combine) -> out [T, H].
    router [E, H] in x's dtype (f16 / bf16); gate, up, down: (codes, scales).  idx (uint32
    [T, top_k]) and w (float32 [T, top_k]), when given, receive the selection."""
    where = "moe_mx4_forward_tokens"
    _cuda(x, router, idx, w)
    T, H = x.shape
    E, I = _mx4_expert_weights(gate, up, down, H, where)
    if router.shape != (E, H) or router.dtype != x.dtype:
        raise MoeError(2, f"{where}: router is [E, H] in x's dtype")
    if (idx is not None and (idx.dtype != torch.uint32 or idx.shape != (T, top_k))) or (
            w is not None and (w.dtype != torch.float32 or w.shape != (T, top_k))):
        raise MoeError(2, f"{where}: idx is uint32 [T, top_k], w float32 [T, top_k]")
    if out is None:
        out = _new(x.shape, x.dtype, x.device, stream)
    elif out.shape != x.shape or out.dtype != x.dtype:
        raise MoeError(2, f"{where}: out is not like x")
    else:
        _cuda(out)
    s = _stream(stream)
    ws = _mx4_ws(ws, max(mx4_tokens_workspace_bytes(T, E, H, I, top_k, x.dtype), 256), x.device,
                 stream, s)
    _check(lib().moe_mx4_forward_tokens(
        x.data_ptr(), router.data_ptr(), _mx4_dtype(x), gate[0].data_ptr(), gate[1].data_ptr(),
        up[0].data_ptr(), up[1].data_ptr(), down[0].data_ptr(), down[1].data_ptr(), T, E, H, I,
        top_k, int(bool(renormalize)), out.data_ptr(), _ptr(idx), _ptr(w), ws.data_ptr(),
        ws.numel(), s), where)
    return out
