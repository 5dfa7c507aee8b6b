"""Outputs that overlap an input or another output are refused before a device
is touched; memory that only lies between an input's rows is not. Made-up
addresses, so only where no device could be handed them (no GPU needed)."""
import random

import pytest

import causal_conv_backward_gb300 as m
from causal_conv_backward_gb300 import _ssm
from causal_conv_backward_gb300 import build as cbuild
from test_ssm_abi_host import INVALID, direct, in_phase

AREA = 1 << 24      # every pointer in an area of its own


@pytest.fixture(scope="module", autouse=True)
def lib():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("made-up addresses")
    cbuild.build()
    return _ssm._load()


S, B, H, W, N, G = 5, 2, 32, 4, 16, 2
ACT, BC, ONE = (B * H, H), (B * G * N, G * N, N), (G * N, N)


def make(cls, strides, **kw):
    """All pointers of `cls`, each in its own area."""
    a = cls(**strides, **kw)
    for i, (name, kind) in enumerate(cls._fields_):
        if kind is _ssm._vp:
            setattr(a, name, (i + 1) * AREA)
    return a


def scan_fwd():
    return make(m.ScanArgs, dict(u_strides=ACT, delta_strides=ACT, z_strides=ACT, B_strides=BC, C_strides=BC),
                S=S, B=B, H=H, N=N, G=G, flags=2)


def scan_bwd():
    a = make(m.ScanBwdArgs, dict(grad_y_strides=ACT))
    a.fwd = scan_fwd()
    for name, kind in m.ScanBwdArgs._fields_:
        if kind is _ssm._vp:
            setattr(a, name, getattr(a, name) + 100 * AREA)
    return a


CALLS = {
    "short_conv": lambda: make(m.ShortConvArgs, dict(x_strides=ACT), S=S, B=B, H=H, W=W),
    "short_conv_bwd": lambda: make(m.ShortConvBwdArgs, dict(grad_y_strides=ACT, x_strides=ACT), S=S, B=B, H=H, W=W),
    "short_conv_step": lambda: make(m.ShortConvStepArgs, {}, x_stride=H, cache_rows=3, B=B, H=H, W=W),
    "scan": scan_fwd,
    "scan_bwd": scan_bwd,
    "scan_step": lambda: make(m.ScanStepArgs, dict(B_strides=ONE, C_strides=ONE), u_stride=H, delta_stride=H, z_stride=H,
                              cache_rows=3, B=B, H=H, N=N, G=G),
}
OUT = {"short_conv": ["y", "final_state"], "short_conv_bwd": ["grad_x", "grad_weight", "grad_bias", "grad_state"],
       "short_conv_step": ["y", "state"], "scan": ["y", "final_state"],
       "scan_bwd": ["grad_u", "grad_delta", "grad_z", "grad_B", "grad_C", "grad_A", "grad_D", "grad_delta_bias", "grad_state"],
       "scan_step": ["y", "state"]}
PHASED = ("short_conv_bwd", "scan", "scan_bwd")


def status(name, a, ws=1000 * AREA):
    return in_phase(name, a, ws=ws) if name in PHASED else direct(name, a)


def pointers(name):
    own = [f for f, kind in type(CALLS[name]())._fields_ if kind is _ssm._vp]
    return own + (["fwd." + f for f, kind in m.ScanArgs._fields_ if kind is _ssm._vp and f not in ("y", "final_state")]
                  if name == "scan_bwd" else [])


def put(a, field, value):
    if field.startswith("fwd."):
        setattr(a.fwd, field[4:], value)
    else:
        setattr(a, field, value)


@pytest.mark.parametrize("name", CALLS)
def test_separate_memory_is_not_refused(name):
    assert status(name, CALLS[name]()) != INVALID


@pytest.mark.parametrize("name,out", [(n, o) for n in CALLS for o in OUT[n]])
def test_an_output_on_anything_else_is_refused(name, out):
    for field in pointers(name):
        if field == out:
            continue
        a = CALLS[name]()
        put(a, field, getattr(a, out))
        assert status(name, a) == INVALID, field
    if name in PHASED and name != "scan":       # this size of scan needs no workspace
        assert status(name, CALLS[name](), ws=getattr(CALLS[name](), out)) == INVALID


def test_the_backward_ignores_the_forwards_outputs():
    a = scan_bwd()
    a.fwd.y, a.fwd.final_state = a.grad_u, a.grad_state
    assert status("scan_bwd", a) != INVALID


def test_missing_tensors_overlap_nothing():
    a = CALLS["scan"]()
    a.z, a.z_strides[0], a.z_strides[1] = None, 1, 1
    a.D = a.delta_bias = a.state = a.lengths = a.final_state = None
    a.flags = 0
    assert status("scan", a) != INVALID
    a.y = a.u
    assert status("scan", a) == INVALID


@pytest.mark.parametrize("seed", range(8))
def test_rows_against_their_bytes(seed):
    """Random strides and places against the bytes themselves: between rows, at
    their ends, under zero strides."""
    r = random.Random(seed)
    for _ in range(200):
        S, B, H = r.randint(1, 5), r.randint(1, 4), r.randint(1, 6)
        s = [r.choice((0, 1, H, H + 3, B * H, 4 * B * H, r.randint(0, 40))) for _ in range(2)]
        x, y = AREA, AREA + 2 * r.randint(-2 * S * B * H, 4 * 4 * B * H)
        read = {x + 2 * (t * s[0] + b * s[1] + h) for t in range(S) for b in range(B) for h in range(H)}
        written = {y + 2 * i for i in range(S * B * H)}
        a = m.ShortConvArgs(x=x, x_strides=tuple(s), weight=2 * AREA, y=y, S=S, B=B, H=H, W=2)
        assert (direct("short_conv", a) == INVALID) == bool(read & written), (S, B, H, s, y - x)


@pytest.mark.parametrize("seed", range(4))
def test_groups_against_their_bytes(seed):
    r = random.Random(100 + seed)
    for _ in range(200):
        S, B, G, N = r.randint(1, 4), r.randint(1, 3), r.randint(1, 3), r.randint(1, 4)
        H = G * r.randint(1, 3)
        s = [r.choice((0, N, G * N, B * G * N, 3 * B * G * N, r.randint(0, 30))) for _ in range(3)]
        at, y = AREA, AREA + 2 * r.randint(-2 * S * B * H, 12 * B * G * N)
        read = {at + 2 * (t * s[0] + b * s[1] + g * s[2] + n) for t in range(S) for b in range(B) for g in range(G) for n in range(N)}
        written = {y + 2 * i for i in range(S * B * H)}
        a = m.ScanArgs(u=2 * AREA, u_strides=(B * H, H), delta=3 * AREA, delta_strides=(B * H, H), B_=at, B_strides=tuple(s),
                       C=4 * AREA, C_strides=(B * G * N, G * N, N), A=5 * AREA, y=y, S=S, B=B, H=H, N=N, G=G)
        assert (status("scan", a) == INVALID) == bool(read & written), (S, B, G, N, H, s, y - at)
