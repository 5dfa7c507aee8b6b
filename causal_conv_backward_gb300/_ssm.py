"""The short convolution and the selective scan on torch tensors: argument
checks and marshalling over the C ABI of ``include/mcc1d_ssm.h``.

Like ``forward`` and ``backward`` of the masked convolution, the calls record
nothing for autograd: results do not require a gradient, whatever the inputs
do, and gradients come from the ``_backward`` calls.
``examples/selective_block.py`` puts the pairs into ``autograd.Function``s.

``stream`` (a torch stream or its handle) takes a call off the current stream.
The caller orders it after what made the inputs, and later users of the results
after it; memory is not reused before both streams are done with it."""
from __future__ import annotations

import ctypes
import struct
from collections import namedtuple

from ._lib import Mcc1dError, load as _load_lib

SILU, SOFTPLUS = 1, 2

_vp, _i64, _i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32


def _struct(name, doc, fields):
    return type(name, (ctypes.Structure,), {"_fields_": fields, "__doc__": doc})


_CONV_SHAPE = [("S", _i64), ("B", _i64), ("H", _i64), ("W", _i64), ("dtype", _i32), ("flags", _i32)]
_SCAN_SHAPE = [("S", _i64), ("B", _i64), ("H", _i64), ("N", _i64), ("G", _i64), ("dtype", _i32), ("flags", _i32)]

ShortConvArgs = _struct("ShortConvArgs", "Mirror of ``mcc1d_short_conv_args``.", [
    ("x", _vp), ("x_strides", _i64 * 2), ("weight", _vp), ("bias", _vp), ("state", _vp), ("lengths", _vp),
    ("y", _vp), ("final_state", _vp)] + _CONV_SHAPE)
ShortConvBwdArgs = _struct("ShortConvBwdArgs", "Mirror of ``mcc1d_short_conv_bwd_args``.", [
    ("grad_y", _vp), ("grad_y_strides", _i64 * 2), ("x", _vp), ("x_strides", _i64 * 2), ("weight", _vp),
    ("bias", _vp), ("state", _vp), ("lengths", _vp), ("grad_final_state", _vp), ("grad_x", _vp),
    ("grad_weight", _vp), ("grad_bias", _vp), ("grad_state", _vp)] + _CONV_SHAPE)
ShortConvStepArgs = _struct("ShortConvStepArgs", "Mirror of ``mcc1d_short_conv_step_args``.", [
    ("x", _vp), ("x_stride", _i64), ("state", _vp), ("weight", _vp), ("bias", _vp), ("slots", _vp), ("y", _vp),
    ("cache_rows", _i64)] + _CONV_SHAPE[1:])
ScanArgs = _struct("ScanArgs", "Mirror of ``mcc1d_scan_args``.", [
    ("u", _vp), ("u_strides", _i64 * 2), ("delta", _vp), ("delta_strides", _i64 * 2), ("z", _vp),
    ("z_strides", _i64 * 2), ("B_", _vp), ("B_strides", _i64 * 3), ("C", _vp), ("C_strides", _i64 * 3), ("A", _vp),
    ("D", _vp), ("delta_bias", _vp), ("state", _vp), ("lengths", _vp), ("y", _vp), ("final_state", _vp)] + _SCAN_SHAPE)
ScanBwdArgs = _struct("ScanBwdArgs", "Mirror of ``mcc1d_scan_bwd_args``.", [
    ("fwd", ScanArgs), ("grad_y", _vp), ("grad_y_strides", _i64 * 2), ("grad_final_state", _vp), ("grad_u", _vp),
    ("grad_delta", _vp), ("grad_z", _vp), ("grad_B", _vp), ("grad_C", _vp), ("grad_A", _vp), ("grad_D", _vp),
    ("grad_delta_bias", _vp), ("grad_state", _vp)])
ScanStepArgs = _struct("ScanStepArgs", "Mirror of ``mcc1d_scan_step_args``.", [
    ("u", _vp), ("u_stride", _i64), ("delta", _vp), ("delta_stride", _i64), ("z", _vp), ("z_stride", _i64),
    ("B_", _vp), ("B_strides", _i64 * 2), ("C", _vp), ("C_strides", _i64 * 2), ("A", _vp), ("D", _vp),
    ("delta_bias", _vp), ("state", _vp), ("slots", _vp), ("y", _vp), ("cache_rows", _i64)] + _SCAN_SHAPE[1:])

ShortConvGrads = namedtuple("ShortConvGrads", "x weight bias state")
SelectiveScanGrads = namedtuple("SelectiveScanGrads", "u delta A B C D z delta_bias state")



def _packer(cls):
    """struct.pack for the fields of ``cls``: the calls build their descriptor
    as one bytes object, several times faster than filling a ctypes structure."""
    def codes(c):
        out = ""
        for _, kind in c._fields_:
            if hasattr(kind, "_fields_"):
                out += codes(kind)
            elif kind is _vp:
                out += "P"
            else:
                n = getattr(kind, "_length_", 1)
                out += ("q" if ctypes.sizeof(kind) // n == 8 else "i") * n
        return out
    s = struct.Struct("@" + codes(cls))
    assert s.size == ctypes.sizeof(cls)
    return s.pack


_pack_conv, _pack_conv_bwd, _pack_conv_step = (_packer(c) for c in (ShortConvArgs, ShortConvBwdArgs, ShortConvStepArgs))
_pack_scan, _pack_scan_bwd, _pack_scan_step = (_packer(c) for c in (ScanArgs, ScanBwdArgs, ScanStepArgs))

_lib = None
_torch = None
_raw_stream = None
_current_device = None


def _load():
    """The library with this module's prototypes, and torch."""
    global _lib, _torch, _raw_stream, _current_device
    if _lib is None:
        import torch
        lib = _load_lib()
        size, u64 = ctypes.POINTER(ctypes.c_uint64), ctypes.c_uint64
        for name, args in (("short_conv", []), ("short_conv_bwd", [_vp, u64]), ("short_conv_step", []),
                           ("scan", [_vp, u64]), ("scan_bwd", [_vp, u64]), ("scan_step", [])):
            f = getattr(lib, "mcc1d_" + name)
            f.argtypes, f.restype = [_vp, *args, _vp], _i32
        for name in ("short_conv_bwd", "scan", "scan_bwd"):
            f = getattr(lib, f"mcc1d_{name}_workspace_size")
            f.argtypes, f.restype = [_vp, size], _i32
        # the current stream's handle without a Stream object around it
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: torch.cuda.current_stream(index).cuda_stream)
        _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        _torch, _lib = torch, lib
    return _lib


# ------------------------------------------------------------------ checks
def _code(t, name):
    if t.dtype is _torch.bfloat16:
        return 0
    if t.dtype is _torch.float16:
        return 1
    raise TypeError(f"{name} must be bfloat16 or float16, not {t.dtype}")


def _refuse(t, name, shape, dtype, index):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{index}")
    raise ValueError(f"{name} must be contiguous")


def _dense(t, name, shape, dtype, index):
    """The address of a dense tensor of this shape, dtype and device."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index or not t.is_contiguous():
        _refuse(t, name, shape, dtype, index)
    return t.data_ptr()


def _optional(t, name, shape, dtype, index):
    return 0 if t is None else _dense(t, name, shape, dtype, index)


def _rows(t, name, shape, dtype, index):
    """The address of a tensor with adjacent elements along its last axis."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index:
        _refuse(t, name, shape, dtype, index)
    if shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have adjacent elements along its last axis (stride 1, not {t.stride(-1)})")
    return t.data_ptr()


def _first(t, name, dims):
    """Shape, dtype code and device of the leading tensor."""
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, not {t.dim()}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    shape = t.shape
    if shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have adjacent elements along its last axis (stride 1, not {t.stride(-1)})")
    index = t.get_device()
    if index != _current_device():
        raise ValueError(f"{name} is on cuda:{index}, the current device is cuda:{_current_device()}")
    return shape, _code(t, name), index


def _flag(activation):
    if activation == "silu":
        return SILU
    if activation is None:
        return 0
    raise ValueError(f"activation must be 'silu' or None, not {activation!r}")


# ------------------------------------------------------------------ streams and workspaces
def _stream(stream, index):
    """The stream's handle, and the torch stream where one was given."""
    if stream is None:
        return _raw_stream(index), None
    if isinstance(stream, int):
        stream = _torch.cuda.ExternalStream(stream, device=index) if stream else _torch.cuda.default_stream(index)
    elif stream.device.index != index:
        raise ValueError(f"stream is on cuda:{stream.device.index}, the tensors on cuda:{index}")
    return stream.cuda_stream, stream


def _empty(shape, dtype, device, stream):
    """Memory for a call on `stream`. A given stream's comes from its own pool:
    the current stream may still be reading or writing what its pool hands out,
    and nothing orders the given stream after that."""
    if stream is None:
        return _torch.empty(shape, dtype=dtype, device=device)
    with _torch.cuda.stream(stream):
        return _torch.empty(shape, dtype=dtype, device=device)


def _record(stream, index, used, made=()):
    """After a call on a given stream: no tensor's memory is reused before that
    stream is done with it, nor the outputs' before the current stream is."""
    current = _torch.cuda.current_stream(index)
    for t in used:
        if t is not None:
            t.record_stream(stream)
    for t in made:
        if t is not None:
            t.record_stream(stream)
            t.record_stream(current)


def _call(name, args, handle):
    st = getattr(_lib, name)(args, handle)
    if st != 0:
        raise Mcc1dError(st, name)


def _call_ws(name, args, handle, stream, device):
    """The two phases: sizes the workspace, takes it from torch, enqueues."""
    n = ctypes.c_uint64()
    st = getattr(_lib, name + "_workspace_size")(args, n)
    if st != 0:
        raise Mcc1dError(st, name + "_workspace_size")
    n = n.value
    ws = _empty(n, _torch.uint8, device, stream) if n else None
    st = getattr(_lib, name)(args, ws.data_ptr() if n else 0, n, handle)
    if st != 0:
        raise Mcc1dError(st, name)


# ------------------------------------------------------------------ short convolution
def short_conv(x, weight, bias=None, *, activation="silu", lengths=None, state=None, return_state=False, y=None,
               stream=None):
    """y = act(bias + causal depthwise conv(x, weight)) on x [S,B,H] (bf16 or
    fp16; any strides with adjacent channels), weight [W,H] (1 <= W <= 8), bias
    [H] or None. ``activation``: "silu" or None. ``state`` [B,W-1,H] holds the
    W-1 rows before the sequence (zeros without it). ``lengths`` (int32 [B])
    ends sequence b after lengths[b] tokens; y is zero past the end, and x is
    not read there. A given ``y`` is dense and overlaps no input. Returns y, or
    (y, final_state) with ``return_state``: the last W-1 rows, which continue
    the sequence in another call or in ``short_conv_step``."""
    _load()
    shape, code, index = _first(x, "x", 3)
    S, B, H = shape
    W, dt, device = weight.shape[0], x.dtype, x.device
    handle, stream = _stream(stream, index)
    if y is None:
        y = _empty(shape, dt, device, stream)
    final = _empty((B, W - 1, H), dt, device, stream) if return_state else None
    args = _pack_conv(x.data_ptr(), x.stride(0), x.stride(1), _dense(weight, "weight", (W, H), dt, index),
                      _optional(bias, "bias", (H,), dt, index), _optional(state, "state", (B, W - 1, H), dt, index),
                      _optional(lengths, "lengths", (B,), _torch.int32, index), _dense(y, "y", shape, dt, index),
                      0 if final is None else final.data_ptr(), S, B, H, W, code, _flag(activation))
    _call("mcc1d_short_conv", args, handle)
    if stream is not None:
        _record(stream, index, (x, weight, bias, state, lengths), (y, final))
    return (y, final) if return_state else y


def short_conv_backward(grad_y, x, weight, bias=None, *, activation="silu", lengths=None, state=None,
                        grad_final_state=None, stream=None):
    """Gradients of ``short_conv`` (same arguments) for grad_y [S,B,H] and, if
    the final state went into the loss, grad_final_state [B,W-1,H]. Returns
    ``ShortConvGrads(x, weight, bias, state)``; bias and state are None where
    the argument was."""
    _load()
    shape, code, index = _first(x, "x", 3)
    S, B, H = shape
    W, dt, device = weight.shape[0], x.dtype, x.device
    handle, stream = _stream(stream, index)
    gx = _empty(shape, dt, device, stream)
    gw = _empty((W, H), dt, device, stream)
    gb = _empty((H,), dt, device, stream) if bias is not None else None
    gs = _empty((B, W - 1, H), dt, device, stream) if state is not None else None
    args = _pack_conv_bwd(_rows(grad_y, "grad_y", shape, dt, index), grad_y.stride(0), grad_y.stride(1), x.data_ptr(),
                          x.stride(0), x.stride(1), _dense(weight, "weight", (W, H), dt, index),
                          _optional(bias, "bias", (H,), dt, index), _optional(state, "state", (B, W - 1, H), dt, index),
                          _optional(lengths, "lengths", (B,), _torch.int32, index),
                          _optional(grad_final_state, "grad_final_state", (B, W - 1, H), dt, index), gx.data_ptr(),
                          gw.data_ptr(), 0 if gb is None else gb.data_ptr(), 0 if gs is None else gs.data_ptr(),
                          S, B, H, W, code, _flag(activation))
    _call_ws("mcc1d_short_conv_bwd", args, handle, stream, device)
    if stream is not None:
        _record(stream, index, (grad_y, x, weight, bias, state, lengths, grad_final_state), (gx, gw, gb, gs))
    return ShortConvGrads(gx, gw, gb, gs)


def _cache(state, tail, dtype, index, B, slots):
    """Address and rows of a cache [rows, *tail] that serves B sequences, and
    the address of the rows' slots."""
    rows = state.shape[0] if state.dim() else 0
    at = _dense(state, "state", (rows, *tail), dtype, index)
    if slots is not None:
        return at, rows, _dense(slots, "slots", (B,), _torch.int32, index)
    if rows < B:
        raise ValueError(f"state has {rows} rows for {B} sequences")
    return at, rows, 0


def short_conv_step(x, state, weight, bias=None, *, activation="silu", slots=None, y=None, stream=None):
    """``short_conv`` of one token per sequence: x [B,H]; ``state`` is a cache
    [rows,W-1,H] whose row b (or slots[b], int32) holds sequence b's window and
    is moved on in place. A slot outside the cache marks a padding row: y is
    zero, no state changes. Two rows must not name one slot. A given ``y`` is
    dense and overlaps nothing else. Returns y [B,H]."""
    _load()
    shape, code, index = _first(x, "x", 2)
    B, H = shape
    W, dt = weight.shape[0], x.dtype
    handle, stream = _stream(stream, index)
    if y is None:
        y = _empty(shape, dt, x.device, stream)
    cache, rows, at = _cache(state, (W - 1, H), dt, index, B, slots)
    args = _pack_conv_step(x.data_ptr(), x.stride(0), cache, _dense(weight, "weight", (W, H), dt, index),
                           _optional(bias, "bias", (H,), dt, index), at, _dense(y, "y", shape, dt, index), rows, B, H,
                           W, code, _flag(activation))
    _call("mcc1d_short_conv_step", args, handle)
    if stream is not None:
        _record(stream, index, (x, state, weight, bias, slots), (y,))
    return y


# ------------------------------------------------------------------ selective scan
def _scan_fields(u, delta, A, B, C, D, z, delta_bias, softplus, lengths, state, y, final):
    """The descriptor's fields, in order."""
    shape, code, index = _first(u, "u", 3)
    S, nb, H = shape
    dt, f32 = u.dtype, _torch.float32
    if A.dim() != 2 or B.dim() != 4:
        raise ValueError("A must be [H,N] and B, C [S,B,G,N]")
    N, G = A.shape[1], B.shape[2]
    bc = (S, nb, G, N)
    return (u.data_ptr(), u.stride(0), u.stride(1), _rows(delta, "delta", shape, dt, index), delta.stride(0),
            delta.stride(1), *((0, 0, 0) if z is None else (_rows(z, "z", shape, dt, index), z.stride(0), z.stride(1))),
            _rows(B, "B", bc, dt, index), B.stride(0), B.stride(1), B.stride(2),
            _rows(C, "C", bc, dt, index), C.stride(0), C.stride(1), C.stride(2), _dense(A, "A", (H, N), f32, index),
            _optional(D, "D", (H,), f32, index), _optional(delta_bias, "delta_bias", (H,), f32, index),
            _optional(state, "state", (nb, H, N), f32, index), _optional(lengths, "lengths", (nb,), _torch.int32, index),
            _optional(y, "y", shape, dt, index), 0 if final is None else final.data_ptr(), S, nb, H, N, G, code,
            SOFTPLUS if softplus else 0)


def selective_scan(u, delta, A, B, C, D=None, z=None, delta_bias=None, *, delta_softplus=False, lengths=None,
                   state=None, return_state=False, y=None, stream=None):
    """h_t = exp(dt_t A) h_{t-1} + dt_t u_t B_t;  y_t = (C_t . h_t + D u_t) * silu(z_t)
    with dt = delta + delta_bias, through softplus if ``delta_softplus``.

    u, delta, z [S,B,H] and B, C [S,B,G,N] are bf16 or fp16 (any strides with
    an adjacent last axis; H/G channels share a group's B and C; N <= 64); A
    [H,N], D [H], delta_bias [H] and ``state`` [B,H,N], the state before the
    sequence, are fp32. ``lengths`` (int32 [B]) ends sequence b after
    lengths[b] tokens: y is zero past the end, nothing is read there. A given
    ``y`` is dense and overlaps no input. Returns y, or (y, final_state) with
    ``return_state``."""
    _load()
    (S, nb, H), _, index = _first(u, "u", 3)
    device = u.device
    handle, stream = _stream(stream, index)
    if y is None:
        y = _empty((S, nb, H), u.dtype, device, stream)
    final = _empty((nb, H, A.shape[-1]), _torch.float32, device, stream) if return_state else None
    args = _pack_scan(*_scan_fields(u, delta, A, B, C, D, z, delta_bias, delta_softplus, lengths, state, y, final))
    _call_ws("mcc1d_scan", args, handle, stream, device)
    if stream is not None:
        _record(stream, index, (u, delta, A, B, C, D, z, delta_bias, lengths, state), (y, final))
    return (y, final) if return_state else y


def selective_scan_backward(grad_y, u, delta, A, B, C, D=None, z=None, delta_bias=None, *, delta_softplus=False,
                            lengths=None, state=None, grad_final_state=None, stream=None):
    """Gradients of ``selective_scan`` (same arguments) for grad_y [S,B,H] and,
    if the final state went into the loss, grad_final_state [B,H,N]. Returns
    ``SelectiveScanGrads(u, delta, A, B, C, D, z, delta_bias, state)`` with None
    where the argument was None; A, D, delta_bias and state are fp32."""
    _load()
    fwd = _scan_fields(u, delta, A, B, C, D, z, delta_bias, delta_softplus, lengths, state, None, None)
    shape, device, index, dt, f32 = u.shape, u.device, u.get_device(), u.dtype, _torch.float32
    S, nb, H = shape
    G, N = B.shape[2:]
    handle, stream = _stream(stream, index)

    def out(like, shape, dtype):
        return _empty(shape, dtype, device, stream) if like is not None else None

    g = SelectiveScanGrads(out(u, shape, dt), out(u, shape, dt), out(A, (H, N), f32), out(B, (S, nb, G, N), dt),
                           out(C, (S, nb, G, N), dt), out(D, (H,), f32), out(z, shape, dt),
                           out(delta_bias, (H,), f32), out(state, (nb, H, N), f32))
    at = SelectiveScanGrads(*[0 if t is None else t.data_ptr() for t in g])
    args = _pack_scan_bwd(*fwd, _rows(grad_y, "grad_y", shape, dt, index), grad_y.stride(0), grad_y.stride(1),
                          _optional(grad_final_state, "grad_final_state", (nb, H, N), f32, index), at.u, at.delta,
                          at.z, at.B, at.C, at.A, at.D, at.delta_bias, at.state)
    _call_ws("mcc1d_scan_bwd", args, handle, stream, device)
    if stream is not None:
        _record(stream, index, (grad_y, u, delta, A, B, C, D, z, delta_bias, lengths, state, grad_final_state), g)
    return g


def selective_scan_step(u, delta, state, A, B, C, D=None, z=None, delta_bias=None, *, delta_softplus=False,
                        slots=None, y=None, stream=None):
    """``selective_scan`` of one token per sequence: u, delta, z [B,H], B, C
    [B,G,N]; ``state`` is an fp32 cache [rows,H,N] whose row b (or slots[b],
    int32) holds sequence b's state and is moved on in place. A slot outside
    the cache marks a padding row: y is zero, no state changes. Two rows must
    not name one slot. A given ``y`` is dense and overlaps nothing else. Returns
    y [B,H]."""
    _load()
    shape, code, index = _first(u, "u", 2)
    nb, H = shape
    dt, f32 = u.dtype, _torch.float32
    if A.dim() != 2 or B.dim() != 3:
        raise ValueError("A must be [H,N] and B, C [B,G,N]")
    N, G = A.shape[1], B.shape[1]
    bc = (nb, G, N)
    handle, stream = _stream(stream, index)
    if y is None:
        y = _empty(shape, dt, u.device, stream)
    cache, rows, at = _cache(state, (H, N), f32, index, nb, slots)
    args = _pack_scan_step(u.data_ptr(), u.stride(0), _rows(delta, "delta", shape, dt, index), delta.stride(0),
                           *((0, 0) if z is None else (_rows(z, "z", shape, dt, index), z.stride(0))),
                           _rows(B, "B", bc, dt, index), B.stride(0), B.stride(1), _rows(C, "C", bc, dt, index),
                           C.stride(0), C.stride(1), _dense(A, "A", (H, N), f32, index),
                           _optional(D, "D", (H,), f32, index), _optional(delta_bias, "delta_bias", (H,), f32, index),
                           cache, at, _dense(y, "y", shape, dt, index), rows, nb, H, N, G, code,
                           SOFTPLUS if delta_softplus else 0)
    _call("mcc1d_scan_step", args, handle)
    if stream is not None:
        _record(stream, index, (u, delta, state, A, B, C, D, z, delta_bias, slots), (y,))
    return y
