"""NaN and infinity in the gated delta rule's inputs: they come out of every
token that depends on them, by whichever path, and out of no other's."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import causal_conv_backward_gb300 as m  # noqa: E402
import delta_reference as ref  # noqa: E402
from ssm_reference import check, to64  # noqa: E402
from test_delta_gpu import FORMS, NAN, cuda_ready, inputs, lens  # noqa: E402,F401

INF = float("inf")
TOKENS = ("q", "k", "v", "delta", "beta")
SHAPE = dict(B=2, H=4, G=2, K=32, V=24)


def run(t, lengths=None):
    args = [t[k] for k in TOKENS + ("A", "delta_bias")]
    return m.gated_delta(*args, lengths=lens(lengths), state=t["state"], return_state=True, **FORMS)


def exact(t, lengths=None, grad=False):
    d = {k: to64(v, grad=grad) for k, v in t.items()}
    return d, *ref.delta_rule(*[d[k] for k in TOKENS + ("A", "delta_bias")], lengths=lengths, state=d["state"])


def same_where_finite(got, bad, clean, what):
    """Not finite exactly where the definition is not; `clean`, without the value, elsewhere."""
    bad = bad.detach()
    assert torch.equal(torch.isfinite(got.cpu()), torch.isfinite(bad)), what
    check(torch.where(torch.isfinite(bad).cuda(), got, 0), torch.where(torch.isfinite(bad), clean, 0), 32 + 256, what)


def spoil(t, name, at, value):
    t = dict(t, **{name: t[name].clone()})
    t[name][at] = value
    return t


# a token on each side of 16 and of a chunk, in the token path (S < 32) and in chunks
PLACES = [(16, 5), (31, 0), (32, 0), (64, 20), (64, 63), (130, 64), (200, 17), (200, 70)]


@pytest.mark.parametrize("S,at", PLACES)
@pytest.mark.parametrize("name", ["delta", "A", "delta_bias"])
def test_a_gate_that_is_nan(S, at, name):
    t, _, gy, gf = inputs(S, **SHAPE)
    bad = spoil(t, name, (at, 0, 1) if name == "delta" else 1, NAN)
    y, final = run(bad)
    first = at if name == "delta" else 0
    seq = slice(0, 1) if name == "delta" else slice(None)
    assert torch.isnan(y[first:, seq, 1]).all() and torch.isnan(final[seq, 1]).all()
    clean, state = run(t)
    others = [0, 2, 3]
    assert torch.equal(y[:, :, others], clean[:, :, others]) and torch.equal(final[:, others], state[:, others])
    if name == "delta":
        assert torch.equal(y[:, 1], clean[:, 1]) and torch.equal(final[1], state[1])
    got = m.gated_delta_backward(gy, *[bad[k] for k in TOKENS + ("A", "delta_bias")], state=bad["state"], grad_final_state=gf, **FORMS)
    d, ry, rf = exact(bad, grad=True)
    names = [k for k in got._fields]
    for k, want in zip(names, torch.autograd.grad((ry * to64(gy)).sum() + (rf * to64(gf)).sum(), [d[k] for k in names])):
        assert not torch.isfinite(getattr(got, k).cpu())[~torch.isfinite(want)].any(), k


@pytest.mark.parametrize("S,at", PLACES)
@pytest.mark.parametrize("value", [NAN, INF])
@pytest.mark.parametrize("name", ["q", "k", "v", "beta", "delta"])
def test_earlier_tokens_and_other_rows_keep_their_values(S, at, name, value):
    if name in ("beta", "delta") and value == INF:
        value = NAN             # a gate of one, or no state left: finite
    t, _, _, _ = inputs(S, **SHAPE)
    bad = spoil(t, name, (at, 0, 1) if name in ("beta", "delta") else (at, 0, 1, 3), value)
    y, final = run(bad)
    _, ry, rf = exact(bad)
    _, cy, cf = exact(t)
    same_where_finite(y, ry, cy, "y")
    same_where_finite(final, rf, cf, "final state")


@pytest.mark.parametrize("S", [16, 100])
def test_what_a_length_leaves_out_spoils_nothing(S):
    """The first value that is not finite is the first one behind the end."""
    t, _, _, _ = inputs(S, **SHAPE)
    n = [S // 2, S]
    bad = t
    for name in TOKENS:
        bad = spoil(bad, name, (slice(n[0], None), 0), NAN)
    y, final = run(bad, n)
    clean, state = run(t, n)
    assert torch.equal(y, clean) and torch.equal(final, state)


@pytest.mark.parametrize("name", TOKENS + ("state",))
def test_long_prompts_in_segments(name):
    """One head, its time axis cut into segments: a value that is not finite
    reaches all tokens after it, and none before."""
    S, at = 2600, 1000
    t, _, _, _ = inputs(S, 1, 1, 1, 16, 8, what="dbs")
    where = {"q": (at, 0, 0, 3), "k": (at, 0, 0, 3), "v": (at, 0, 0, 3), "delta": (at, 0, 0), "beta": (at, 0, 0), "state": (0, 0, 3)}[name]
    bad = spoil(t, name, where, NAN)
    y, final = run(bad)
    _, ry, rf = exact(bad)
    _, cy, cf = exact(t)
    same_where_finite(y, ry, cy, "y")
    same_where_finite(final, rf, cf, "final state")


@pytest.mark.parametrize("name", ["q", "k", "v", "beta"])
@pytest.mark.parametrize("S,at", [(16, 5), (64, 20), (200, 70)])
def test_gradients_do_not_hide_it(S, at, name):
    t, _, gy, gf = inputs(S, **SHAPE)
    bad = spoil(t, name, (at, 0, 1) if name == "beta" else (at, 0, 1, 3), NAN)
    got = m.gated_delta_backward(gy, *[bad[k] for k in TOKENS + ("A", "delta_bias")], state=bad["state"], grad_final_state=gf, **FORMS)
    d, ry, rf = exact(bad, grad=True)
    names = [k for k in got._fields]
    for k, want in zip(names, torch.autograd.grad((ry * to64(gy)).sum() + (rf * to64(gf)).sum(), [d[k] for k in names])):
        g = getattr(got, k).cpu()
        assert not torch.isfinite(g)[~torch.isfinite(want)].any(), k
        if k in TOKENS:         # the other sequence has nothing to do with it
            assert torch.isfinite(g[:, 1]).all(), k
