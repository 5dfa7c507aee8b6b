"""The host contracts of include/mcc1d_delta.h and include/mcc1d_norm.h: the
binding's structures mirror the headers', bad arguments and overlapping outputs
are refused with their status before a device is touched, workspace sizes are
functions of the shape (no GPU needed)."""
import ctypes
import os
import shutil
import subprocess

import pytest

import causal_conv_backward_gb300 as m
from causal_conv_backward_gb300 import _delta, _norm, _ssm
from causal_conv_backward_gb300 import build as cbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULLPTR, INVALID, SHAPE, WORKSPACE = 0, 161001, 161002, 561002, 561003
STRUCTS = {"mcc1d_delta_args": m.DeltaArgs, "mcc1d_delta_bwd_args": m.DeltaBwdArgs, "mcc1d_delta_step_args": m.DeltaStepArgs,
           "mcc1d_gated_norm_args": m.GatedNormArgs, "mcc1d_gated_norm_bwd_args": m.GatedNormBwdArgs,
           "mcc1d_residual_norm_args": m.ResidualNormArgs, "mcc1d_residual_norm_bwd_args": m.ResidualNormBwdArgs}
AREA = 1 << 24      # every pointer in an area of its own


@pytest.fixture(scope="module", autouse=True)
def lib():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("made-up addresses")
    cbuild.build()
    _delta._load(), _norm._load()


def test_structures_mirror_the_headers(tmp_path):
    gcc = shutil.which("gcc") or pytest.skip("no gcc")
    lines = ['#include <stddef.h>', '#include <stdio.h>', '#include "mcc1d_delta.h"', '#include "mcc1d_norm.h"', "int main(void) {"]
    for c, py in STRUCTS.items():
        lines.append(f'printf("{c} %zu", sizeof({c}));')
        for f in py._fields_:
            lines.append(f'printf(" %zu", offsetof({c}, {f[0]}));')
        lines.append('printf("\\n");')
    lines.append("return 0; }")
    src, exe = tmp_path / "sizes.c", tmp_path / "sizes"
    src.write_text("\n".join(lines))
    subprocess.run([gcc, "-std=c99", "-Wall", "-Werror", "-pedantic", f"-I{os.path.join(ROOT, 'include')}", str(src), "-o", str(exe)], check=True)
    for line in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines():
        name, size, *offsets = line.split()
        py = STRUCTS[name]
        assert ctypes.sizeof(py) == int(size), name
        assert [getattr(py, f[0]).offset for f in py._fields_] == [int(o) for o in offsets], name


S, B, H, G, K, V, D = 70, 2, 4, 2, 16, 24, 32
QK, VS, GATES = (B * G * K, G * K, K), (B * H * V, H * V, V), (B * H, H)


def make(cls, strides, base=0, **kw):
    """All pointers of `cls`, each in its own area."""
    a = cls(**strides, **kw)
    for i, (name, kind) in enumerate(cls._fields_):
        if kind is _ssm._vp:
            setattr(a, name, (base + i + 1) * AREA)
    return a


def delta_fwd():
    return make(m.DeltaArgs, dict(q_strides=QK, k_strides=QK, v_strides=VS, delta_strides=GATES, beta_strides=GATES), S=S, B=B, H=H, G=G,
                K=K, V=V, scale=0.25, flags=2 | 8 | 16)


def delta_bwd():
    a = make(m.DeltaBwdArgs, dict(grad_y_strides=VS), base=100)
    a.fwd = delta_fwd()
    return a


def delta_step():
    return make(m.DeltaStepArgs, dict(q_strides=QK[1:], k_strides=QK[1:], v_strides=VS[1:]), delta_stride=H, beta_stride=H, cache_rows=3, B=B,
                H=H, G=G, K=K, V=V, scale=0.25, flags=2)


NORM = (B * H * D, H * D, D)


def gated_fwd():
    return make(m.GatedNormArgs, dict(x_strides=NORM, z_strides=NORM), S=S, B=B, H=H, D=D, eps=1e-6)


def gated_bwd():
    a = make(m.GatedNormBwdArgs, dict(grad_y_strides=NORM), base=100)
    a.fwd = gated_fwd()
    return a


def residual_fwd():
    return make(m.ResidualNormArgs, dict(x_strides=GATES, residual_strides=GATES), S=S, B=B, H=H, eps=1e-6, flags=4)


def residual_bwd():
    a = make(m.ResidualNormBwdArgs, dict(grad_y_strides=GATES, grad_h_strides=GATES), base=100)
    a.fwd = residual_fwd()
    return a


CALLS = {"delta": delta_fwd, "delta_bwd": delta_bwd, "delta_step": delta_step, "gated_norm": gated_fwd, "gated_norm_bwd": gated_bwd,
         "residual_norm": residual_fwd, "residual_norm_bwd": residual_bwd}
PHASED = ("delta", "delta_bwd", "gated_norm_bwd", "residual_norm_bwd")
OUT = {"delta": ["y", "final_state"],
       "delta_bwd": ["grad_q", "grad_k", "grad_v", "grad_delta", "grad_beta", "grad_A", "grad_delta_bias", "grad_state"],
       "delta_step": ["y", "state"], "gated_norm": ["y"], "gated_norm_bwd": ["grad_x", "grad_z", "grad_weight"],
       "residual_norm": ["y", "h"],
       "residual_norm_bwd": ["grad_x", "grad_residual", "grad_weight", "grad_post_weight", "grad_scale"]}
IGNORED = {"delta": ("y", "final_state"), "gated_norm": ("y",), "residual_norm": ("y", "h")}     # of a backward's `fwd`


def lib_call(name, a, ws=1000 * AREA, n=1 << 40):
    f = getattr(_ssm._lib, "mcc1d_" + name)
    return f(ctypes.byref(a), ws, n, None) if name in PHASED else f(ctypes.byref(a), None)


def size(name, a):
    n = ctypes.c_uint64(12345)
    return getattr(_ssm._lib, f"mcc1d_{name}_workspace_size")(ctypes.byref(a), ctypes.byref(n)), n.value


def put(a, field, value):
    part, _, last = field.rpartition(".")
    setattr(getattr(a, part) if part else a, last, value)


def put_all(a, kw):
    for k, v in kw.items():
        if isinstance(v, tuple):
            part, _, last = k.rpartition(".")
            at = getattr(getattr(a, part) if part else a, last)
            for i, x in enumerate(v):
                at[i] = x
        else:
            put(a, k, v)
    return a


def pointers(name):
    own = [f for f, kind in type(CALLS[name]())._fields_ if kind is _ssm._vp]
    if name.endswith("_bwd"):
        fwd = name[:-4]
        own += ["fwd." + f for f, kind in type(CALLS[fwd]())._fields_ if kind is _ssm._vp and f not in IGNORED[fwd]]
    return own


@pytest.mark.parametrize("name", CALLS)
def test_separate_memory_is_not_refused(name):
    assert lib_call(name, CALLS[name]()) not in (NULLPTR, INVALID, SHAPE, WORKSPACE)


@pytest.mark.parametrize("name,out", [(n, o) for n in CALLS for o in OUT[n]])
def test_an_output_on_anything_else_is_refused(name, out):
    for field in pointers(name):
        if field != out:
            a = CALLS[name]()
            put(a, field, getattr(a, out))
            assert lib_call(name, a) == INVALID, field
    if name in PHASED:
        assert lib_call(name, CALLS[name](), ws=getattr(CALLS[name](), out)) == INVALID


def test_between_the_rows_of_an_input_there_is_room():
    """y in the other half of the projection that q, k, v are a part of."""
    a = delta_fwd()
    wide = 4 * B * H * V
    put_all(a, {"v_strides": (wide, wide // B, V)})
    a.y = a.v + 2 * (wide // B // 2)
    a.S, a.B = 1, 1
    assert lib_call("delta", a) != INVALID
    a.y = a.v + 2 * (H * V - 1)
    assert lib_call("delta", a) == INVALID


@pytest.mark.parametrize("name", CALLS)
def test_what_is_required(name):
    optional = {"delta": ["delta", "delta_bias", "state", "lengths", "final_state"],
                "delta_bwd": ["grad_final_state", "grad_delta_bias", "grad_state", "fwd.delta_bias", "fwd.state", "fwd.lengths"],
                "delta_step": ["delta", "delta_bias", "slots"], "gated_norm": ["z"], "gated_norm_bwd": ["grad_z"],
                "residual_norm": ["post_weight", "scale"], "residual_norm_bwd": ["grad_h", "grad_post_weight", "grad_scale"]}[name]
    for field in pointers(name):
        a = CALLS[name]()
        put(a, field, None)
        if field == "fwd.delta_bias":
            a.grad_delta_bias = None
        if field in optional:
            assert lib_call(name, a) not in (NULLPTR, INVALID), field
        else:
            assert lib_call(name, a) == NULLPTR, field


COMMON = [("dtype", 2, INVALID), ("flags", 64, INVALID), ("B", 0, SHAPE), ("H", 0, SHAPE), ("B", 65536, SHAPE), ("H", (1 << 20) + 4, SHAPE)]
DELTA = COMMON + [("K", 0, SHAPE), ("K", 129, SHAPE), ("V", 0, SHAPE), ("V", 1025, SHAPE), ("G", 3, SHAPE), ("G", 0, SHAPE),
                  ("scale", float("nan"), INVALID), ("scale", float("inf"), INVALID)]
PROMPT = [("S", 0, SHAPE), ("S", 1 << 31, SHAPE), ("q_strides", (-1, 0, 0), INVALID), ("v_strides", (0, 0, -1), INVALID),
          ("beta_strides", (0, -1), INVALID), ("delta_strides", (-1, 0), INVALID), ("A", AREA + 2, INVALID), ("state", AREA + 2, INVALID),
          ("lengths", AREA + 1, INVALID), ("k", AREA + 1, INVALID)]


@pytest.mark.parametrize("field,value,code", DELTA + PROMPT)
def test_delta_refuses(field, value, code):
    a = put_all(delta_fwd(), {field: value})
    assert size("delta", a) == (code, 12345) and lib_call("delta", a) == code
    a = put_all(delta_bwd(), {"fwd." + field: value})
    assert size("delta_bwd", a) == (code, 12345) and lib_call("delta_bwd", a) == code


@pytest.mark.parametrize("kw,code", [({"grad_y_strides": (0, -1, 0)}, INVALID), ({"grad_y": AREA + 1}, INVALID), ({"grad_A": AREA + 2}, INVALID),
                                     ({"fwd.delta_bias": None}, NULLPTR), ({"fwd.delta": None}, NULLPTR)])
def test_delta_bwd_refuses(kw, code):
    assert lib_call("delta_bwd", put_all(delta_bwd(), kw)) == code


@pytest.mark.parametrize("field,value,code", DELTA + [("cache_rows", 0, SHAPE), ("q_strides", (-1, 0), INVALID), ("beta_stride", -1, INVALID),
                                                      ("delta_stride", -1, INVALID), ("state", AREA + 2, INVALID), ("slots", AREA + 2, INVALID)])
def test_delta_step_refuses(field, value, code):
    assert lib_call("delta_step", put_all(delta_step(), {field: value})) == code


@pytest.mark.parametrize("name", ["delta", "delta_step"])
def test_states_stay_below_2_to_the_31(name):
    for V, code in ((63, OK), (64, SHAPE)):          # 2 * 2^17 * 128 * 64 = 2^31
        a = put_all(CALLS[name](), {"H": 1 << 17, "K": 128, "V": V, "B": 2})
        assert (size(name, a)[0] if name in PHASED else lib_call(name, a)) in ((SHAPE,) if code else (OK, INVALID, 561100, 561102)), V


def test_delta_step_needs_rows_or_slots():
    assert lib_call("delta_step", put_all(delta_step(), {"cache_rows": 1, "slots": None})) == SHAPE


EPS = [("eps", -1.0, INVALID), ("eps", float("nan"), INVALID), ("eps", float("inf"), INVALID)]


@pytest.mark.parametrize("field,value,code", [c for c in COMMON if c[0] != "H" or c[1] == 0] + EPS + [
    ("D", 0, SHAPE), ("D", 16385, SHAPE), ("S", 0, SHAPE), ("S", (1 << 31) - 4096, SHAPE), ("x_strides", (0, 0, -1), INVALID), ("z", AREA + 1, INVALID)])
def test_gated_norm_refuses(field, value, code):
    assert lib_call("gated_norm", put_all(gated_fwd(), {field: value})) == code
    assert lib_call("gated_norm_bwd", put_all(gated_bwd(), {"fwd." + field: value})) == code


@pytest.mark.parametrize("field,value,code", COMMON + EPS + [
    ("H", 16385, SHAPE), ("S", 0, SHAPE), ("x_strides", (0, -1), INVALID), ("residual", AREA + 2, INVALID), ("scale", AREA + 2, INVALID)])
def test_residual_norm_refuses(field, value, code):
    assert lib_call("residual_norm", put_all(residual_fwd(), {field: value})) == code
    assert lib_call("residual_norm_bwd", put_all(residual_bwd(), {"fwd." + field: value})) == code


@pytest.mark.parametrize("name,kw", [("gated_norm_bwd", {"fwd.z": None}), ("residual_norm_bwd", {"fwd.scale": None}),
                                     ("residual_norm_bwd", {"fwd.post_weight": None})])
def test_gradients_of_what_is_not_there(name, kw):
    assert lib_call(name, put_all(CALLS[name](), kw)) == NULLPTR


def test_null_descriptors_and_sizes():
    for name in CALLS:
        f = getattr(_ssm._lib, "mcc1d_" + name)
        assert (f(None, None, 0, None) if name in PHASED else f(None, None)) == NULLPTR
    for name in PHASED:
        a = CALLS[name]()
        f = getattr(_ssm._lib, f"mcc1d_{name}_workspace_size")
        assert f(ctypes.byref(a), None) == NULLPTR
        st, n = size(name, a)
        assert st == OK and n > 0 and size(name, a) == (OK, n)
        assert lib_call(name, a, ws=None) == NULLPTR
        assert lib_call(name, a, ws=1000 * AREA + 4) == INVALID
        assert lib_call(name, a, n=n - 1) == WORKSPACE
    a = delta_fwd()
    a.S = 31         # token by token
    assert size("delta", a) == (OK, 0)


def test_cpu_tensors_and_shapes_are_refused():
    torch = pytest.importorskip("torch")
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    q, v, g, A = bf(5, 2, 2, 8), bf(5, 2, 4, 8), bf(5, 2, 4), torch.zeros(4)
    for call in (lambda: m.gated_delta(q, q, v, g, g, A), lambda: m.gated_delta_backward(v, q, q, v, g, g, A),
                 lambda: m.gated_delta_step(q[0], q[0], v[0], g[0], g[0], torch.zeros(2, 4, 8, 8), A), lambda: m.gated_norm(v, v, bf(8)),
                 lambda: m.gated_norm_backward(v, v, v, bf(8)), lambda: m.residual_norm(g, g, bf(4)),
                 lambda: m.residual_norm_backward(g, None, g, g, bf(4)), lambda: m.gated_norm(bf(8), None, bf(8)),
                 lambda: m.gated_delta(q[0], q, v, g, g, A)):
        with pytest.raises(ValueError):
            call()
