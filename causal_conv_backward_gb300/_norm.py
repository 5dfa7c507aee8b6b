"""The norms of a block on torch tensors, behind its mixer and behind the
residual sum: argument checks and marshalling over the C ABI of
``include/mcc1d_norm.h``. As with the short convolution and the scan, the calls
record nothing for autograd (``examples/gated_delta_block.py`` has the
``autograd.Function``s), and ``stream`` takes a call off the current stream."""
from __future__ import annotations

import ctypes
from collections import namedtuple

from . import _ssm as _base
from ._ssm import (_call, _call_ws, _dense, _empty, _first, _i32, _i64, _optional, _packer, _record, _rows,
                   _stream, _struct, _vp)

WIDE = 4

GatedNormArgs = _struct("GatedNormArgs", "Mirror of ``mcc1d_gated_norm_args``.", [
    ("x", _vp), ("x_strides", _i64 * 3), ("z", _vp), ("z_strides", _i64 * 3), ("weight", _vp), ("y", _vp), ("S", _i64),
    ("B", _i64), ("H", _i64), ("D", _i64), ("eps", ctypes.c_double), ("dtype", _i32), ("flags", _i32)])
GatedNormBwdArgs = _struct("GatedNormBwdArgs", "Mirror of ``mcc1d_gated_norm_bwd_args``.", [
    ("fwd", GatedNormArgs), ("grad_y", _vp), ("grad_y_strides", _i64 * 3), ("grad_x", _vp), ("grad_z", _vp),
    ("grad_weight", _vp)])
ResidualNormArgs = _struct("ResidualNormArgs", "Mirror of ``mcc1d_residual_norm_args``.", [
    ("x", _vp), ("x_strides", _i64 * 2), ("residual", _vp), ("residual_strides", _i64 * 2), ("weight", _vp),
    ("post_weight", _vp), ("scale", _vp), ("y", _vp), ("h", _vp), ("S", _i64), ("B", _i64), ("H", _i64),
    ("eps", ctypes.c_double), ("dtype", _i32), ("flags", _i32)])
ResidualNormBwdArgs = _struct("ResidualNormBwdArgs", "Mirror of ``mcc1d_residual_norm_bwd_args``.", [
    ("fwd", ResidualNormArgs), ("grad_y", _vp), ("grad_y_strides", _i64 * 2), ("grad_h", _vp),
    ("grad_h_strides", _i64 * 2), ("grad_x", _vp), ("grad_residual", _vp), ("grad_weight", _vp),
    ("grad_post_weight", _vp), ("grad_scale", _vp)])

GatedNormGrads = namedtuple("GatedNormGrads", "x z weight")
ResidualNormGrads = namedtuple("ResidualNormGrads", "x residual weight post_weight scale")

_pack_gated, _pack_gated_bwd = _packer(GatedNormArgs), _packer(GatedNormBwdArgs)
_pack_residual, _pack_residual_bwd = _packer(ResidualNormArgs), _packer(ResidualNormBwdArgs)

_ready = None


def _load():
    """The library with this module's prototypes."""
    global _ready
    lib = _base._lib if _base._lib is not None else _base._load()
    if _ready is not lib:
        size, u64 = ctypes.POINTER(ctypes.c_uint64), ctypes.c_uint64
        for name, args in (("gated_norm", []), ("gated_norm_bwd", [_vp, u64]), ("residual_norm", []),
                           ("residual_norm_bwd", [_vp, u64])):
            f = getattr(lib, "mcc1d_" + name)
            f.argtypes, f.restype = [_vp, *args, _vp], _i32
        for name in ("gated_norm_bwd", "residual_norm_bwd"):
            f = getattr(lib, f"mcc1d_{name}_workspace_size")
            f.argtypes, f.restype = [_vp, size], _i32
        _ready = lib


def _leading(t, name, least, most):
    """Shape, the same filled up on the left with ones, dtype code and device of the leading tensor."""
    n = t.dim()
    if not least <= n <= most:
        raise ValueError(f"{name} must have {least} to {most} dimensions, not {n}")
    shape, code, index = _first(t, name, n)
    return shape, (1,) * (most - n) + tuple(shape), code, index


def _steps(t, most):
    """The strides of all axes but the last, filled up on the left with zeros."""
    s = t.stride()
    return (0,) * (most - len(s)) + s[:-1]


# ------------------------------------------------------------------ behind the mixer
def _gated_fields(x, z, weight, y, eps, lead):
    shape, (S, B, H, D), code, index = lead
    dt = x.dtype
    return (x.data_ptr(), *_steps(x, 4), *((0, 0, 0, 0) if z is None else (_rows(z, "z", shape, dt, index), *_steps(z, 4))),
            _dense(weight, "weight", (D,), dt, index), 0 if y is None else _dense(y, "y", shape, dt, index), S, B, H, D, eps, code, 0)


def gated_norm(x, z, weight, *, eps=1e-6, y=None, stream=None):
    """y = x / sqrt(mean(x^2) + eps) * weight * silu(z) over the last axis of x
    [S,B,H,D] (or [B,H,D], [H,D]; bf16 or fp16; any strides with an adjacent last
    axis), with weight [D]; z like x, or None for no gate. A given ``y`` is dense
    and overlaps no input. Returns y."""
    _load()
    lead = _leading(x, "x", 2, 4)
    handle, stream = _stream(stream, lead[3])
    if y is None:
        y = _empty(lead[0], x.dtype, x.device, stream)
    _call("mcc1d_gated_norm", _pack_gated(*_gated_fields(x, z, weight, y, eps, lead)), handle)
    if stream is not None:
        _record(stream, lead[3], (x, z, weight), (y,))
    return y


def gated_norm_backward(grad_y, x, z, weight, *, eps=1e-6, stream=None):
    """Gradients of ``gated_norm`` (same arguments) for grad_y like x. Returns
    ``GatedNormGrads(x, z, weight)``; z is None where the argument was."""
    _load()
    lead = _leading(x, "x", 2, 4)
    fwd = _gated_fields(x, z, weight, None, eps, lead)
    shape, device, index, dt = lead[0], x.device, lead[3], x.dtype
    handle, stream = _stream(stream, index)
    at = _rows(grad_y, "grad_y", shape, dt, index)
    gx = _empty(shape, dt, device, stream)
    gz = _empty(shape, dt, device, stream) if z is not None else None
    gw = _empty(weight.shape, dt, device, stream)
    args = _pack_gated_bwd(*fwd, at, *_steps(grad_y, 4), gx.data_ptr(), 0 if gz is None else gz.data_ptr(), gw.data_ptr())
    _call_ws("mcc1d_gated_norm_bwd", args, handle, stream, device)
    if stream is not None:
        _record(stream, index, (grad_y, x, z, weight), (gx, gz, gw))
    return GatedNormGrads(gx, gz, gw)


# ------------------------------------------------------------------ behind the residual sum
def _stream_type(residual, dt):
    """The residual stream's dtype and flag."""
    if residual.dtype is _base._torch.float32:
        return residual.dtype, WIDE
    if residual.dtype is not dt:
        raise TypeError(f"residual must be {dt} or torch.float32, not {residual.dtype}")
    return dt, 0


def _residual_fields(x, residual, weight, post_weight, scale, y, h, eps, lead, rt, flag):
    shape, (S, B, H), code, index = lead
    dt, row = x.dtype, (H,)
    return (x.data_ptr(), *_steps(x, 3), _rows(residual, "residual", shape, rt, index), *_steps(residual, 3),
            _dense(weight, "weight", row, dt, index), _optional(post_weight, "post_weight", row, dt, index),
            _optional(scale, "scale", row, _base._torch.float32, index), _optional(y, "y", shape, dt, index),
            _optional(h, "h", shape, rt, index), S, B, H, eps, code, flag)


def residual_norm(x, residual, weight, *, post_weight=None, scale=None, eps=1e-6, y=None, h=None, stream=None):
    """h = residual + scale * m,  y = h / sqrt(mean(h^2) + eps) * weight, where m is
    the branch's output x, or x / sqrt(mean(x^2) + eps) * post_weight where that
    is given. x [S,B,H] (or [B,H]; any strides with adjacent channels) and the
    weights [H] are bf16 or fp16, residual (and so h) has that dtype or fp32,
    scale [H] is fp32. Given ``y`` and ``h`` are dense and overlap no input.
    Returns (y, h): what the next block reads, and the residual behind it."""
    _load()
    lead = _leading(x, "x", 2, 3)
    rt, flag = _stream_type(residual, x.dtype)
    handle, stream = _stream(stream, lead[3])
    if y is None:
        y = _empty(lead[0], x.dtype, x.device, stream)
    if h is None:
        h = _empty(lead[0], rt, x.device, stream)
    _call("mcc1d_residual_norm", _pack_residual(*_residual_fields(x, residual, weight, post_weight, scale, y, h, eps, lead, rt, flag)),
          handle)
    if stream is not None:
        _record(stream, lead[3], (x, residual, weight, post_weight, scale), (y, h))
    return y, h


def residual_norm_backward(grad_y, grad_h, x, residual, weight, *, post_weight=None, scale=None, eps=1e-6, stream=None):
    """Gradients of ``residual_norm`` (same arguments) for grad_y like x and, if h
    went into the loss, grad_h like residual (or None). Returns
    ``ResidualNormGrads(x, residual, weight, post_weight, scale)`` with None where
    the argument was None."""
    _load()
    lead = _leading(x, "x", 2, 3)
    rt, flag = _stream_type(residual, x.dtype)
    fwd = _residual_fields(x, residual, weight, post_weight, scale, None, None, eps, lead, rt, flag)
    shape, device, index, dt = lead[0], x.device, lead[3], x.dtype
    handle, stream = _stream(stream, index)
    at = _rows(grad_y, "grad_y", shape, dt, index), *_steps(grad_y, 3)
    at_h = (0, 0, 0) if grad_h is None else (_rows(grad_h, "grad_h", shape, rt, index), *_steps(grad_h, 3))
    gx, gr = _empty(shape, dt, device, stream), _empty(shape, rt, device, stream)
    gw = _empty(weight.shape, dt, device, stream)
    gp = _empty(weight.shape, dt, device, stream) if post_weight is not None else None
    gs = _empty(weight.shape, _base._torch.float32, device, stream) if scale is not None else None
    args = _pack_residual_bwd(*fwd, *at, *at_h, gx.data_ptr(), gr.data_ptr(), gw.data_ptr(), 0 if gp is None else gp.data_ptr(),
                              0 if gs is None else gs.data_ptr())
    _call_ws("mcc1d_residual_norm_bwd", args, handle, stream, device)
    if stream is not None:
        _record(stream, index, (grad_y, grad_h, x, residual, weight, post_weight, scale), (gx, gr, gw, gp, gs))
    return ResidualNormGrads(gx, gr, gw, gp, gs)
