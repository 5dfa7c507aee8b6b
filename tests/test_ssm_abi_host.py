"""The host contract of include/mcc1d_ssm.h: the binding's structures mirror the
header's, bad arguments are refused with their status before a device is
touched, workspace sizes are functions of the shape (no GPU needed)."""
import ctypes
import os
import shutil
import subprocess

import pytest

import causal_conv_backward_gb300 as m
from causal_conv_backward_gb300 import _ssm
from causal_conv_backward_gb300 import build as cbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULLPTR, INVALID, SHAPE, WORKSPACE = 0, 161001, 161002, 561002, 561003
STRUCTS = {"mcc1d_short_conv_args": m.ShortConvArgs, "mcc1d_short_conv_bwd_args": m.ShortConvBwdArgs,
           "mcc1d_short_conv_step_args": m.ShortConvStepArgs, "mcc1d_scan_args": m.ScanArgs,
           "mcc1d_scan_bwd_args": m.ScanBwdArgs, "mcc1d_scan_step_args": m.ScanStepArgs}


@pytest.fixture(scope="module", autouse=True)
def lib():
    cbuild.build()
    return _ssm._load()


def test_structures_mirror_the_header(tmp_path):
    gcc = shutil.which("gcc") or pytest.skip("no gcc")
    lines = ['#include <stddef.h>', '#include <stdio.h>', '#include "mcc1d_ssm.h"', "int main(void) {"]
    for c, py in STRUCTS.items():
        lines.append(f'printf("{c} %zu", sizeof({c}));')
        for f in py._fields_:
            lines.append(f'printf(" %zu", offsetof({c}, {f[0]}));')
        lines.append('printf("\\n");')
    lines.append("return 0; }")
    src = tmp_path / "sizes.c"
    src.write_text("\n".join(lines))
    exe = tmp_path / "sizes"
    subprocess.run([gcc, "-std=c99", "-Wall", "-Werror", "-pedantic", f"-I{os.path.join(ROOT, 'include')}", str(src), "-o", str(exe)], check=True)
    for line in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines():
        name, size, *offsets = line.split()
        py = STRUCTS[name]
        assert ctypes.sizeof(py) == int(size), name
        assert [getattr(py, f[0]).offset for f in py._fields_] == [int(o) for o in offsets], name


P = 0x10000


def conv_args(**kw):
    d = dict(x=P, x_strides=(64, 32), weight=P, y=P, S=5, B=2, H=32, W=4, dtype=0, flags=1)
    return m.ShortConvArgs(**{**d, **kw})


def conv_bwd_args(**kw):
    d = dict(grad_y=P, grad_y_strides=(64, 32), x=P, x_strides=(64, 32), weight=P, grad_x=P, grad_weight=P, S=5, B=2,
             H=32, W=4, dtype=0, flags=1)
    return m.ShortConvBwdArgs(**{**d, **kw})


def conv_step_args(**kw):
    d = dict(x=P, x_stride=32, state=P, weight=P, y=P, cache_rows=2, B=2, H=32, W=4, dtype=0, flags=1)
    return m.ShortConvStepArgs(**{**d, **kw})


def scan_args(**kw):
    d = dict(u=P, u_strides=(64, 32), delta=P, delta_strides=(64, 32), B_=P, B_strides=(32, 16, 16), C=P,
             C_strides=(32, 16, 16), A=P, y=P, S=5, B=2, H=32, N=16, G=1, dtype=0, flags=2)
    return m.ScanArgs(**{**d, **kw})


def scan_bwd_args(fwd=None, **kw):
    d = dict(fwd=fwd or scan_args(y=None), grad_y=P, grad_y_strides=(64, 32), grad_u=P, grad_delta=P, grad_B=P, grad_C=P,
             grad_A=P)
    return m.ScanBwdArgs(**{**d, **kw})


def scan_step_args(**kw):
    d = dict(u=P, u_stride=32, delta=P, delta_stride=32, B_=P, B_strides=(16, 16), C=P, C_strides=(16, 16), A=P, state=P,
             y=P, cache_rows=2, B=2, H=32, N=16, G=1, dtype=0, flags=2)
    return m.ScanStepArgs(**{**d, **kw})


def size(name, a):
    n = ctypes.c_uint64(12345)
    st = getattr(_ssm._load(), f"mcc1d_{name}_workspace_size")(ctypes.byref(a), ctypes.byref(n))
    return st, n.value


def direct(name, a):
    return getattr(_ssm._load(), "mcc1d_" + name)(ctypes.byref(a), None)


def in_phase(name, a, ws=P, n=1 << 40):
    return getattr(_ssm._load(), "mcc1d_" + name)(ctypes.byref(a), ws, n, None)


COMMON = [(dict(dtype=2), INVALID), (dict(flags=64), INVALID), (dict(B=0), SHAPE), (dict(H=0), SHAPE),
          (dict(B=65536), SHAPE), (dict(H=(1 << 20) + 1), SHAPE)]
CONV_BAD = COMMON + [(dict(S=0), SHAPE), (dict(S=1 << 31), SHAPE), (dict(W=0), SHAPE), (dict(W=9), SHAPE),
                     (dict(x=P + 1), INVALID), (dict(lengths=P + 2), INVALID), (dict(x_strides=(-64, 32)), INVALID),
                     (dict(x=None), NULLPTR), (dict(weight=None), NULLPTR)]
SCAN_BAD = COMMON + [(dict(S=0), SHAPE), (dict(N=0), SHAPE), (dict(N=65), SHAPE), (dict(G=5), SHAPE), (dict(G=0), SHAPE),
                     (dict(u_strides=(64, -1)), INVALID), (dict(B_strides=(32, 16, -16)), INVALID),
                     (dict(u=P + 1), INVALID), (dict(A=P + 2), INVALID), (dict(state=P + 2), INVALID),
                     (dict(C=None), NULLPTR), (dict(A=None), NULLPTR), (dict(B=65535, H=1 << 20), SHAPE)]


@pytest.mark.parametrize("kw,code", CONV_BAD + [(dict(y=None), NULLPTR), (dict(final_state=P + 1), INVALID)])
def test_short_conv_refuses(kw, code):
    assert direct("short_conv", conv_args(**kw)) == code


@pytest.mark.parametrize("kw,code", CONV_BAD + [(dict(grad_x=None), NULLPTR), (dict(grad_bias=P), NULLPTR),
                                                (dict(grad_state=P), NULLPTR), (dict(grad_y=P + 1), INVALID)])
def test_short_conv_bwd_refuses(kw, code):
    a = conv_bwd_args(**kw)
    assert size("short_conv_bwd", a) == (code, 12345)
    assert in_phase("short_conv_bwd", a) == code


@pytest.mark.parametrize("kw,code", COMMON + [(dict(W=9), SHAPE), (dict(cache_rows=1), SHAPE), (dict(cache_rows=0, slots=P), SHAPE),
                                              (dict(state=None), NULLPTR), (dict(x_stride=-1), INVALID)])
def test_short_conv_step_refuses(kw, code):
    assert direct("short_conv_step", conv_step_args(**kw)) == code


@pytest.mark.parametrize("kw,code", SCAN_BAD + [(dict(y=None), NULLPTR), (dict(final_state=P + 1), INVALID)])
def test_scan_refuses(kw, code):
    a = scan_args(**kw)
    assert size("scan", a) == (code, 12345)
    assert in_phase("scan", a) == code


@pytest.mark.parametrize("kw,code", SCAN_BAD)
def test_scan_bwd_refuses_bad_inputs(kw, code):
    a = scan_bwd_args(scan_args(**{"y": None, **kw}))
    assert size("scan_bwd", a) == (code, 12345)
    assert in_phase("scan_bwd", a) == code


@pytest.mark.parametrize("kw,code", [(dict(grad_A=None), NULLPTR), (dict(grad_z=P), NULLPTR), (dict(grad_D=P), NULLPTR),
                                     (dict(grad_delta_bias=P), NULLPTR), (dict(grad_y=P + 1), INVALID),
                                     (dict(grad_state=P + 2), INVALID), (dict(grad_y_strides=(-1, 0)), INVALID)])
def test_scan_bwd_refuses(kw, code):
    assert size("scan_bwd", scan_bwd_args(**kw)) == (code, 12345)


@pytest.mark.parametrize("kw,code", COMMON + [(dict(N=65), SHAPE), (dict(G=3), SHAPE), (dict(cache_rows=1), SHAPE),
                                              (dict(state=None), NULLPTR), (dict(u_stride=-1), INVALID),
                                              (dict(state=P + 2), INVALID), (dict(slots=P + 1), INVALID)])
def test_scan_step_refuses(kw, code):
    assert direct("scan_step", scan_step_args(**kw)) == code


def test_null_descriptors_and_sizes():
    lib = _ssm._load()
    for name in ("short_conv", "short_conv_step", "scan_step"):
        assert getattr(lib, "mcc1d_" + name)(None, None) == NULLPTR
    for name, a in (("short_conv_bwd", conv_bwd_args()), ("scan", scan_args()), ("scan_bwd", scan_bwd_args())):
        assert getattr(lib, "mcc1d_" + name)(None, None, 0, None) == NULLPTR
        f = getattr(lib, f"mcc1d_{name}_workspace_size")
        assert f(ctypes.byref(a), None) == NULLPTR
        st, n = size(name, a)
        assert st == OK and size(name, a) == (OK, n)
        if n:
            assert in_phase(name, a, ws=None) == NULLPTR
            assert in_phase(name, a, ws=P + 4) == INVALID
            assert in_phase(name, a, n=n - 1) == WORKSPACE


def test_cpu_tensors_are_refused():
    torch = pytest.importorskip("torch")
    x, w = torch.zeros(4, 2, 8, dtype=torch.bfloat16), torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        m.short_conv(x, w)
    with pytest.raises(ValueError):
        m.short_conv_step(x[0], torch.zeros(2, 3, 8, dtype=torch.bfloat16), w)
    A, B = torch.zeros(8, 4), torch.zeros(4, 2, 1, 4, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        m.selective_scan(x, x, A, B, B)
    with pytest.raises(ValueError):
        m.selective_scan_backward(x, x, x, A, B, B)
    with pytest.raises(ValueError):
        m.selective_scan_step(x[0], x[0], torch.zeros(2, 8, 4), A, B[0], B[0])
