"""The gated delta rule on torch tensors: argument checks and marshalling over
the C ABI of ``include/mcc1d_delta.h``. As with the short convolution and the
scan, the calls record nothing for autograd (``examples/gated_delta_block.py``
has the ``autograd.Function``s), and ``stream`` takes a call off the current
stream."""
from __future__ import annotations

import ctypes
from collections import namedtuple

from . import _ssm as _base
from ._ssm import (SOFTPLUS, _cache, _call, _call_ws, _dense, _empty, _first, _i32, _i64, _optional, _packer, _record, _rows,
                   _stream, _struct, _vp)

SIGMOID, QK_NORM = 8, 16

_SHAPE = [("B", _i64), ("H", _i64), ("G", _i64), ("K", _i64), ("V", _i64), ("scale", ctypes.c_double), ("dtype", _i32), ("flags", _i32)]

DeltaArgs = _struct("DeltaArgs", "Mirror of ``mcc1d_delta_args``.", [
    ("q", _vp), ("q_strides", _i64 * 3), ("k", _vp), ("k_strides", _i64 * 3), ("v", _vp), ("v_strides", _i64 * 3),
    ("delta", _vp), ("delta_strides", _i64 * 2), ("beta", _vp), ("beta_strides", _i64 * 2), ("A", _vp), ("delta_bias", _vp),
    ("state", _vp), ("lengths", _vp), ("y", _vp), ("final_state", _vp), ("S", _i64)] + _SHAPE)
DeltaBwdArgs = _struct("DeltaBwdArgs", "Mirror of ``mcc1d_delta_bwd_args``.", [
    ("fwd", DeltaArgs), ("grad_y", _vp), ("grad_y_strides", _i64 * 3), ("grad_final_state", _vp), ("grad_q", _vp),
    ("grad_k", _vp), ("grad_v", _vp), ("grad_delta", _vp), ("grad_beta", _vp), ("grad_A", _vp), ("grad_delta_bias", _vp),
    ("grad_state", _vp)])
DeltaStepArgs = _struct("DeltaStepArgs", "Mirror of ``mcc1d_delta_step_args``.", [
    ("q", _vp), ("q_strides", _i64 * 2), ("k", _vp), ("k_strides", _i64 * 2), ("v", _vp), ("v_strides", _i64 * 2),
    ("delta", _vp), ("delta_stride", _i64), ("beta", _vp), ("beta_stride", _i64), ("A", _vp), ("delta_bias", _vp),
    ("state", _vp), ("slots", _vp), ("y", _vp), ("cache_rows", _i64)] + _SHAPE)

GatedDeltaGrads = namedtuple("GatedDeltaGrads", "q k v delta beta A delta_bias state")

_pack, _pack_bwd, _pack_step = _packer(DeltaArgs), _packer(DeltaBwdArgs), _packer(DeltaStepArgs)

_ready = None


def _load():
    """The library with this module's prototypes."""
    global _ready
    lib = _base._lib if _base._lib is not None else _base._load()
    if _ready is not lib:
        size, u64 = ctypes.POINTER(ctypes.c_uint64), ctypes.c_uint64
        for name, args in (("delta", [_vp, u64]), ("delta_bwd", [_vp, u64]), ("delta_step", [])):
            f = getattr(lib, "mcc1d_" + name)
            f.argtypes, f.restype = [_vp, *args, _vp], _i32
        for name in ("delta", "delta_bwd"):
            f = getattr(lib, f"mcc1d_{name}_workspace_size")
            f.argtypes, f.restype = [_vp, size], _i32
        _ready = lib


def _flags(delta_softplus, beta_sigmoid, qk_norm):
    return (SOFTPLUS if delta_softplus else 0) | (SIGMOID if beta_sigmoid else 0) | (QK_NORM if qk_norm else 0)


def _scale(K, scale):
    return scale if scale is not None else K ** -0.5 if K else 1.0      # no keys: refused below


def _leading(q, v, dims):
    """The sizes S, B (of prompts), G, K, H, V in front, and q's dtype code and device."""
    shape, code, index = _first(q, "q", dims)
    if v.dim() != dims:
        raise ValueError(f"v must have {dims} dimensions, not {v.dim()}")
    return tuple(shape[:-2]), *shape[-2:], *v.shape[-2:], code, index


def _fields(q, k, v, delta, beta, A, delta_bias, softplus, sigmoid, norm, scale, lengths, state, y, final):
    """The descriptor's fields, in order."""
    (S, B), G, K, H, V, code, index = _leading(q, v, 4)
    dt, f32 = q.dtype, _base._torch.float32
    if delta is not None and A is None:
        raise ValueError("delta needs A")
    return (q.data_ptr(), *q.stride()[:3], _rows(k, "k", q.shape, dt, index), *k.stride()[:3], _rows(v, "v", (S, B, H, V), dt, index), *v.stride()[:3],
            *((0, 0, 0) if delta is None else (_rows(delta, "delta", (S, B, H), dt, index), delta.stride(0), delta.stride(1))),
            _rows(beta, "beta", (S, B, H), dt, index), beta.stride(0), beta.stride(1), _optional(A, "A", (H,), f32, index),
            _optional(delta_bias, "delta_bias", (H,), f32, index), _optional(state, "state", (B, H, V, K), f32, index),
            _optional(lengths, "lengths", (B,), _base._torch.int32, index), _optional(y, "y", (S, B, H, V), dt, index),
            0 if final is None else final.data_ptr(), S, B, H, G, K, V, _scale(K, scale), code,
            _flags(softplus, sigmoid, norm))


def gated_delta(q, k, v, delta, beta, A=None, delta_bias=None, *, delta_softplus=False, beta_sigmoid=False, qk_norm=False,
                scale=None, lengths=None, state=None, return_state=False, y=None, stream=None):
    """S_t = a_t S_{t-1} + u_t k_t^T,  u_t = b_t (v_t - a_t S_{t-1} k_t),  y_t = S_t (scale q_t)
    with a = exp(A dt), dt = delta + delta_bias, through softplus if
    ``delta_softplus`` (without delta a = 1, whatever A and delta_bias), b = beta, through a sigmoid if
    ``beta_sigmoid``, and with ``qk_norm`` q / sqrt(|q|^2 + 1e-6) and
    k / sqrt(|k|^2 + 1e-6) for q and k. ``scale`` is K ** -0.5 unless given.

    q, k [S,B,G,K], v [S,B,H,V] and delta, beta [S,B,H] are bf16 or fp16 (any
    strides with an adjacent last axis; H/G heads of v share one of q and k;
    K <= 128, V <= 1024); A, delta_bias [H] and ``state`` [B,H,V,K], the state
    before the sequence, are fp32. ``lengths`` (int32 [B]) ends sequence b after
    lengths[b] tokens: y is zero past the end, nothing is read there. A given
    ``y`` is dense and overlaps no input. Returns y [S,B,H,V], or (y,
    final_state) with ``return_state``."""
    _load()
    (S, B), G, K, H, V, _, index = _leading(q, v, 4)
    device = q.device
    handle, stream = _stream(stream, index)
    if y is None:
        y = _empty((S, B, H, V), q.dtype, device, stream)
    final = _empty((B, H, V, K), _base._torch.float32, device, stream) if return_state else None
    args = _pack(*_fields(q, k, v, delta, beta, A, delta_bias, delta_softplus, beta_sigmoid, qk_norm, scale, lengths, state,
                          y, final))
    _call_ws("mcc1d_delta", args, handle, stream, device)
    if stream is not None:
        _record(stream, index, (q, k, v, delta, beta, A, delta_bias, lengths, state), (y, final))
    return (y, final) if return_state else y


def gated_delta_backward(grad_y, q, k, v, delta, beta, A=None, delta_bias=None, *, delta_softplus=False, beta_sigmoid=False,
                         qk_norm=False, scale=None, lengths=None, state=None, grad_final_state=None, stream=None):
    """Gradients of ``gated_delta`` (same arguments) for grad_y [S,B,H,V] and, if
    the final state went into the loss, grad_final_state [B,H,V,K]. Returns
    ``GatedDeltaGrads(q, k, v, delta, beta, A, delta_bias, state)`` with None
    where the argument was None; A, delta_bias and state are fp32. Without delta
    nothing depends on A and delta_bias: zeros."""
    _load()
    fwd = _fields(q, k, v, delta, beta, A, delta_bias, delta_softplus, beta_sigmoid, qk_norm, scale, lengths, state, None, None)
    (S, B), G, K, H, V, _, index = _leading(q, v, 4)
    device, dt, f32 = q.device, q.dtype, _base._torch.float32
    handle, stream = _stream(stream, index)
    at = _rows(grad_y, "grad_y", (S, B, H, V), dt, index), *grad_y.stride()[:3]
    at_final = _optional(grad_final_state, "grad_final_state", (B, H, V, K), f32, index)

    def out(like, shape, dtype):
        return _empty(shape, dtype, device, stream) if like is not None else None

    g = GatedDeltaGrads(out(q, (S, B, G, K), dt), out(k, (S, B, G, K), dt), out(v, (S, B, H, V), dt), out(delta, (S, B, H), dt),
                        out(beta, (S, B, H), dt), out(A, (H,), f32), out(delta_bias, (H,), f32), out(state, (B, H, V, K), f32))
    made = g if delta is not None else g._replace(A=None, delta_bias=None)      # without delta nothing depends on them
    args = _pack_bwd(*fwd, *at, at_final, *[0 if t is None else t.data_ptr() for t in made])
    _call_ws("mcc1d_delta_bwd", args, handle, stream, device)
    if delta is None and (A is not None or delta_bias is not None):
        with _base._torch.cuda.stream(stream):      # None: the current one
            for t in (g.A, g.delta_bias):
                if t is not None:
                    t.zero_()
    if stream is not None:
        _record(stream, index, (grad_y, q, k, v, delta, beta, A, delta_bias, lengths, state, grad_final_state), g)
    return g


def gated_delta_step(q, k, v, delta, beta, state, A=None, delta_bias=None, *, delta_softplus=False, beta_sigmoid=False,
                     qk_norm=False, scale=None, slots=None, y=None, stream=None):
    """``gated_delta`` of one token per sequence: q, k [B,G,K], v [B,H,V], delta,
    beta [B,H]; ``state`` is an fp32 cache [rows,H,V,K] whose row b (or slots[b],
    int32) holds sequence b's state and is moved on in place. A slot outside the
    cache marks a padding row: y is zero, no state changes. Two rows must not
    name one slot. A given ``y`` is dense and overlaps nothing else. Returns y
    [B,H,V]."""
    _load()
    (B,), G, K, H, V, code, index = _leading(q, v, 3)
    dt, f32 = q.dtype, _base._torch.float32
    if delta is not None and A is None:
        raise ValueError("delta needs A")
    handle, stream = _stream(stream, index)
    cache, rows, at = _cache(state, (H, V, K), f32, index, B, slots)
    if y is None:
        y = _empty((B, H, V), dt, q.device, stream)
    args = _pack_step(q.data_ptr(), *q.stride()[:2], _rows(k, "k", q.shape, dt, index), *k.stride()[:2],
                      _rows(v, "v", (B, H, V), dt, index), *v.stride()[:2],
                      *((0, 0) if delta is None else (_rows(delta, "delta", (B, H), dt, index), delta.stride(0))),
                      _rows(beta, "beta", (B, H), dt, index), beta.stride(0), _optional(A, "A", (H,), f32, index),
                      _optional(delta_bias, "delta_bias", (H,), f32, index), cache, at, _dense(y, "y", (B, H, V), dt, index),
                      rows, B, H, G, K, V, _scale(K, scale), code, _flags(delta_softplus, beta_sigmoid, qk_norm))
    _call("mcc1d_delta_step", args, handle)
    if stream is not None:
        _record(stream, index, (q, k, v, delta, beta, state, A, delta_bias, slots), (y,))
    return y
