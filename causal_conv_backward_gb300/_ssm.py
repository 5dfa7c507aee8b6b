"""The short convolution and the selective scan on torch tensors: argument
checks and marshalling over the C ABI of ``include/mcc1d_ssm.h``."""
from __future__ import annotations

import ctypes
from collections import namedtuple

from ._lib import Mcc1dError, load as _load_lib

SILU, SOFTPLUS = 1, 2
MAX_W, MAX_N = 8, 64

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

_lib = None
_torch = None


def _load():
    """The library with this module's prototypes, and torch."""
    global _lib, _torch
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
        _torch, _lib = torch, lib
    return _lib


# ------------------------------------------------------------------ checks
def _code(t, name):
    if t.dtype is _torch.bfloat16:
        return 0
    if t.dtype is _torch.float16:
        return 1
    raise TypeError(f"{name} must be bfloat16 or float16, not {t.dtype}")


def _check(t, name, shape, dtype, device, dense=True):
    """`t` has this shape, dtype and device, and is dense (or at least has
    adjacent elements along its last axis)."""
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, not {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if dense:
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    elif shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have adjacent elements along its last axis (stride 1, not {t.stride(-1)})")


def _first(t, name, dims):
    """Dims, dtype code and device of the leading tensor."""
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, not {t.dim()}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have adjacent elements along its last axis (stride 1, not {t.stride(-1)})")
    return t.shape, _code(t, name), t.device


def _ptr(t):
    return None if t is None else t.data_ptr()


def _flag(activation):
    if activation == "silu":
        return SILU
    if activation is None:
        return 0
    raise ValueError(f"activation must be 'silu' or None, not {activation!r}")


def _optional(t, name, shape, dtype, device):
    if t is not None:
        _check(t, name, shape, dtype, device)


# ------------------------------------------------------------------ streams and workspaces
def _stream(stream, device):
    """The stream's handle, and the torch stream to record tensors on where it
    is not the current one (their memory must not be reused before it is done)."""
    if stream is None:
        return _torch.cuda.current_stream(device).cuda_stream, None
    if isinstance(stream, int):
        stream = _torch.cuda.ExternalStream(stream, device=device) if stream else _torch.cuda.default_stream(device)
    return stream.cuda_stream, stream


def _record(stream, *tensors):
    if stream is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def _call(name, args, handle):
    st = getattr(_lib, name)(ctypes.byref(args), handle or None)
    if st != 0:
        raise Mcc1dError(st, name)


def _call_ws(name, args, handle, stream, device):
    """The two phases: sizes the workspace, takes it from torch, enqueues."""
    n = ctypes.c_uint64(0)
    st = getattr(_lib, name + "_workspace_size")(ctypes.byref(args), ctypes.byref(n))
    if st != 0:
        raise Mcc1dError(st, name + "_workspace_size")
    ws = _torch.empty(n.value, dtype=_torch.uint8, device=device) if n.value else None
    st = getattr(_lib, name)(ctypes.byref(args), _ptr(ws), n.value, handle or None)
    if st != 0:
        raise Mcc1dError(st, name)
    _record(stream, ws)


def _strides(t, dims):
    """Strides of the leading axes; those of axes of one element do not matter."""
    st, sh = t.stride(), t.shape
    return tuple(st[i] if sh[i] > 1 else 0 for i in range(dims))


# ------------------------------------------------------------------ short convolution
def short_conv(x, weight, bias=None, *, activation="silu", lengths=None, state=None, return_state=False, y=None,
               stream=None):
    """y = act(bias + causal depthwise conv(x, weight)) on x [S,B,H] (bf16 or
    fp16; any strides with adjacent channels), weight [W,H] (1 <= W <= 8), bias
    [H] or None. ``activation``: "silu" or None. ``state`` [B,W-1,H] holds the
    W-1 rows before the sequence (zeros without it). ``lengths`` (int32 [B])
    ends sequence b after lengths[b] tokens; y is zero past the end, and x is
    not read there. Returns y, or (y, final_state) with ``return_state``: the
    last W-1 rows, which continue the sequence in another call or in
    ``short_conv_step``."""
    _load()
    (S, B, H), code, dev = _first(x, "x", 3)
    W, dt = weight.shape[0], x.dtype
    _check(weight, "weight", (W, H), dt, dev)
    _optional(bias, "bias", (H,), dt, dev)
    _optional(state, "state", (B, W - 1, H), dt, dev)
    _optional(lengths, "lengths", (B,), _torch.int32, dev)
    _optional(y, "y", (S, B, H), dt, dev)
    flags = _flag(activation)
    handle, stream = _stream(stream, dev)
    if y is None:
        y = _torch.empty((S, B, H), dtype=dt, device=dev)
    final = _torch.empty((B, W - 1, H), dtype=dt, device=dev) if return_state else None
    args = ShortConvArgs(x.data_ptr(), _strides(x, 2), weight.data_ptr(), _ptr(bias), _ptr(state), _ptr(lengths),
                         y.data_ptr(), _ptr(final), S, B, H, W, code, flags)
    _call("mcc1d_short_conv", args, handle)
    _record(stream, x, weight, bias, state, lengths, y, final)
    return (y, final) if return_state else y


def short_conv_backward(grad_y, x, weight, bias=None, *, activation="silu", lengths=None, state=None,
                        grad_final_state=None, stream=None):
    """Gradients of ``short_conv`` (same arguments) for grad_y [S,B,H] and, if
    the final state went into the loss, grad_final_state [B,W-1,H]. Returns
    ``ShortConvGrads(x, weight, bias, state)``; bias and state are None where
    the argument was."""
    _load()
    (S, B, H), code, dev = _first(x, "x", 3)
    W, dt = weight.shape[0], x.dtype
    _check(weight, "weight", (W, H), dt, dev)
    _check(grad_y, "grad_y", (S, B, H), dt, dev, dense=False)
    _optional(bias, "bias", (H,), dt, dev)
    _optional(state, "state", (B, W - 1, H), dt, dev)
    _optional(lengths, "lengths", (B,), _torch.int32, dev)
    _optional(grad_final_state, "grad_final_state", (B, W - 1, H), dt, dev)
    flags = _flag(activation)
    handle, stream = _stream(stream, dev)
    gx = _torch.empty((S, B, H), dtype=dt, device=dev)
    gw = _torch.empty((W, H), dtype=dt, device=dev)
    gb = _torch.empty((H,), dtype=dt, device=dev) if bias is not None else None
    gs = _torch.empty((B, W - 1, H), dtype=dt, device=dev) if state is not None else None
    args = ShortConvBwdArgs(grad_y.data_ptr(), _strides(grad_y, 2), x.data_ptr(), _strides(x, 2), weight.data_ptr(),
                            _ptr(bias), _ptr(state), _ptr(lengths), _ptr(grad_final_state), gx.data_ptr(),
                            gw.data_ptr(), _ptr(gb), _ptr(gs), S, B, H, W, code, flags)
    _call_ws("mcc1d_short_conv_bwd", args, handle, stream, dev)
    _record(stream, grad_y, x, weight, bias, state, lengths, grad_final_state, gx, gw, gb, gs)
    return ShortConvGrads(gx, gw, gb, gs)


def _cache(state, name, tail, dtype, device, B, slots):
    """Rows of a cache [rows, *tail] that serves B sequences."""
    rows = state.shape[0] if state.dim() else 0
    _check(state, name, (rows, *tail), dtype, device)
    if slots is not None:
        _check(slots, "slots", (B,), _torch.int32, device)
    elif rows < B:
        raise ValueError(f"{name} has {rows} rows for {B} sequences")
    return rows


def short_conv_step(x, state, weight, bias=None, *, activation="silu", slots=None, y=None, stream=None):
    """``short_conv`` of one token per sequence: x [B,H]; ``state`` is a cache
    [rows,W-1,H] whose row b (or slots[b], int32) holds sequence b's window and
    is moved on in place. A slot outside the cache marks a padding row: y is
    zero, no state changes. Two rows must not name one slot. Returns y [B,H]."""
    _load()
    (B, H), code, dev = _first(x, "x", 2)
    W, dt = weight.shape[0], x.dtype
    _check(weight, "weight", (W, H), dt, dev)
    _optional(bias, "bias", (H,), dt, dev)
    _optional(y, "y", (B, H), dt, dev)
    rows = _cache(state, "state", (W - 1, H), dt, dev, B, slots)
    flags = _flag(activation)
    handle, stream = _stream(stream, dev)
    if y is None:
        y = _torch.empty((B, H), dtype=dt, device=dev)
    args = ShortConvStepArgs(x.data_ptr(), _strides(x, 1)[0], _ptr(state), weight.data_ptr(), _ptr(bias), _ptr(slots),
                             y.data_ptr(), rows, B, H, W, code, flags)
    _call("mcc1d_short_conv_step", args, handle)
    _record(stream, x, state, weight, bias, slots, y)
    return y


# ------------------------------------------------------------------ selective scan
def _scan_args(u, delta, A, B, C, D, z, delta_bias, softplus, lengths, state, y, final):
    (S, nb, H), code, dev = _first(u, "u", 3)
    dt, f32 = u.dtype, _torch.float32
    if A.dim() != 2 or B.dim() != 4:
        raise ValueError("A must be [H,N] and B, C [S,B,G,N]")
    N, G = A.shape[1], B.shape[2]
    _check(A, "A", (H, N), f32, dev)
    _check(delta, "delta", (S, nb, H), dt, dev, dense=False)
    _check(B, "B", (S, nb, G, N), dt, dev, dense=False)
    _check(C, "C", (S, nb, G, N), dt, dev, dense=False)
    if z is not None:
        _check(z, "z", (S, nb, H), dt, dev, dense=False)
    _optional(D, "D", (H,), f32, dev)
    _optional(delta_bias, "delta_bias", (H,), f32, dev)
    _optional(lengths, "lengths", (nb,), _torch.int32, dev)
    _optional(state, "state", (nb, H, N), f32, dev)
    return ScanArgs(u.data_ptr(), _strides(u, 2), delta.data_ptr(), _strides(delta, 2), _ptr(z),
                    _strides(z, 2) if z is not None else (0, 0), B.data_ptr(), _strides(B, 3), C.data_ptr(),
                    _strides(C, 3), A.data_ptr(), _ptr(D), _ptr(delta_bias), _ptr(state), _ptr(lengths), _ptr(y),
                    _ptr(final), S, nb, H, N, G, code, SOFTPLUS if softplus else 0)


def selective_scan(u, delta, A, B, C, D=None, z=None, delta_bias=None, *, delta_softplus=False, lengths=None,
                   state=None, return_state=False, y=None, stream=None):
    """h_t = exp(dt_t A) h_{t-1} + dt_t u_t B_t;  y_t = (C_t . h_t + D u_t) * silu(z_t)
    with dt = delta + delta_bias, through softplus if ``delta_softplus``.

    u, delta, z [S,B,H] and B, C [S,B,G,N] are bf16 or fp16 (any strides with
    an adjacent last axis; H/G channels share a group's B and C; N <= 64); A
    [H,N], D [H], delta_bias [H] and ``state`` [B,H,N], the state before the
    sequence, are fp32. ``lengths`` (int32 [B]) ends sequence b after
    lengths[b] tokens: y is zero past the end, nothing is read there. Returns
    y, or (y, final_state) with ``return_state``."""
    _load()
    S, nb, H = u.shape if u.dim() == 3 else (0, 0, 0)
    _optional(y, "y", (S, nb, H), u.dtype, u.device)
    if y is None and u.is_cuda:
        y = _torch.empty((S, nb, H), dtype=u.dtype, device=u.device)
    final = _torch.empty((nb, H, A.shape[-1]), dtype=_torch.float32, device=u.device) if return_state else None
    args = _scan_args(u, delta, A, B, C, D, z, delta_bias, delta_softplus, lengths, state, y, final)
    handle, stream = _stream(stream, u.device)
    _call_ws("mcc1d_scan", args, handle, stream, u.device)
    _record(stream, u, delta, A, B, C, D, z, delta_bias, lengths, state, y, final)
    return (y, final) if return_state else y


def selective_scan_backward(grad_y, u, delta, A, B, C, D=None, z=None, delta_bias=None, *, delta_softplus=False,
                            lengths=None, state=None, grad_final_state=None, stream=None):
    """Gradients of ``selective_scan`` (same arguments) for grad_y [S,B,H] and,
    if the final state went into the loss, grad_final_state [B,H,N]. Returns
    ``SelectiveScanGrads(u, delta, A, B, C, D, z, delta_bias, state)`` with None
    where the argument was None; A, D, delta_bias and state are fp32."""
    _load()
    fwd = _scan_args(u, delta, A, B, C, D, z, delta_bias, delta_softplus, lengths, state, None, None)
    (S, nb, H), dev, dt, f32 = u.shape, u.device, u.dtype, _torch.float32
    G, N = B.shape[2:]
    _check(grad_y, "grad_y", (S, nb, H), dt, dev, dense=False)
    _optional(grad_final_state, "grad_final_state", (nb, H, N), f32, dev)
    handle, stream = _stream(stream, dev)

    def out(like, shape, dtype):
        return _torch.empty(shape, dtype=dtype, device=dev) if like is not None else None

    g = SelectiveScanGrads(out(u, (S, nb, H), dt), out(u, (S, nb, H), dt), out(A, (H, N), f32),
                           out(B, (S, nb, G, N), dt), out(C, (S, nb, G, N), dt), out(D, (H,), f32),
                           out(z, (S, nb, H), dt), out(delta_bias, (H,), f32), out(state, (nb, H, N), f32))
    args = ScanBwdArgs(fwd, grad_y.data_ptr(), _strides(grad_y, 2), _ptr(grad_final_state), _ptr(g.u), _ptr(g.delta),
                       _ptr(g.z), _ptr(g.B), _ptr(g.C), _ptr(g.A), _ptr(g.D), _ptr(g.delta_bias), _ptr(g.state))
    _call_ws("mcc1d_scan_bwd", args, handle, stream, dev)
    _record(stream, grad_y, u, delta, A, B, C, D, z, delta_bias, lengths, state, grad_final_state, *g)
    return g


def selective_scan_step(u, delta, state, A, B, C, D=None, z=None, delta_bias=None, *, delta_softplus=False,
                        slots=None, y=None, stream=None):
    """``selective_scan`` of one token per sequence: u, delta, z [B,H], B, C
    [B,G,N]; ``state`` is an fp32 cache [rows,H,N] whose row b (or slots[b],
    int32) holds sequence b's state and is moved on in place. A slot outside
    the cache marks a padding row: y is zero, no state changes. Two rows must
    not name one slot. Returns y [B,H]."""
    _load()
    (nb, H), code, dev = _first(u, "u", 2)
    dt, f32 = u.dtype, _torch.float32
    if A.dim() != 2 or B.dim() != 3:
        raise ValueError("A must be [H,N] and B, C [B,G,N]")
    N, G = A.shape[1], B.shape[1]
    _check(A, "A", (H, N), f32, dev)
    _check(delta, "delta", (nb, H), dt, dev, dense=False)
    _check(B, "B", (nb, G, N), dt, dev, dense=False)
    _check(C, "C", (nb, G, N), dt, dev, dense=False)
    if z is not None:
        _check(z, "z", (nb, H), dt, dev, dense=False)
    _optional(D, "D", (H,), f32, dev)
    _optional(delta_bias, "delta_bias", (H,), f32, dev)
    _optional(y, "y", (nb, H), dt, dev)
    rows = _cache(state, "state", (H, N), f32, dev, nb, slots)
    handle, stream = _stream(stream, dev)
    if y is None:
        y = _torch.empty((nb, H), dtype=dt, device=dev)
    args = ScanStepArgs(u.data_ptr(), _strides(u, 1)[0], delta.data_ptr(), _strides(delta, 1)[0], _ptr(z),
                        _strides(z, 1)[0] if z is not None else 0, B.data_ptr(), _strides(B, 2), C.data_ptr(),
                        _strides(C, 2), A.data_ptr(), _ptr(D), _ptr(delta_bias), state.data_ptr(), _ptr(slots),
                        y.data_ptr(), rows, nb, H, N, G, code, SOFTPLUS if delta_softplus else 0)
    _call("mcc1d_scan_step", args, handle)
    _record(stream, u, delta, state, A, B, C, D, z, delta_bias, slots, y)
    return y
