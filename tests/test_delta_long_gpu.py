"""The gated delta rule over long prompts of few heads, whose time axis is cut
into segments: against float64, and against the same prompt in parts short
enough to stay whole."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import causal_conv_backward_gb300 as m  # noqa: E402
from ssm_reference import check  # noqa: E402
from test_delta_gpu import F32, FORMS, FP16, cuda_ready, inputs, lens, rand, run  # noqa: E402,F401


@pytest.mark.parametrize("S,H,G,K,V", [(2500, 1, 1, 16, 8), (2304, 2, 1, 100, 130), (3000, 1, 1, 128, 64)])
@pytest.mark.parametrize("what", ["db", "dbsf"])
def test_segments(S, H, G, K, V, what):
    run(S, 1, H, G, K, V, what=what)


@pytest.mark.parametrize("lengths", [[2500, 0], [1, 2499], [700, 1300], [64, 2048]])
def test_segments_of_sequences_that_end_early(lengths):
    run(2500, 2, 1, 1, 24, 16, FP16, lengths=lengths)


def check_both(got, want, terms, what):
    """Two computed results: each is off the exact value by what `check` allows
    (there `want` is exact), so their difference is by twice that, in halves."""
    middle = (got.double() + want.double()) / 2          # |got - middle| = |got - want| / 2
    check(got, middle, terms, what)


def test_parts_of_a_long_prompt():
    """100 K tokens at once, and 1000 at a time with the state handed on."""
    S, H, G, K, V, part = 100_000, 2, 1, 64, 64, 1000
    t, _, gy, gf = inputs(S, 1, H, G, K, V)
    toks, rest = ("q", "k", "v", "delta", "beta"), ("A", "delta_bias")
    y, final = m.gated_delta(*[t[k] for k in toks + rest], state=t["state"], return_state=True, **FORMS)
    state, ys, starts = t["state"], [], []
    for i in range(0, S, part):
        starts.append(state)
        a, state = m.gated_delta(*[t[k][i:i + part] for k in toks], *[t[k] for k in rest], state=state, return_state=True, **FORMS)
        ys.append(a)
    check_both(y, torch.cat(ys), 4 * K + 512, "y")
    check_both(final, state, 4 * K + 512, "state")
    # the gradients of both, the state's handed back
    got = m.gated_delta_backward(gy, *[t[k] for k in toks + rest], state=t["state"], grad_final_state=gf, **FORMS)
    g, parts = gf, []
    for n, i in reversed(list(enumerate(range(0, S, part)))):
        r = m.gated_delta_backward(gy[i:i + part], *[t[k][i:i + part] for k in toks], *[t[k] for k in rest], state=starts[n], grad_final_state=g, **FORMS)
        g = r.state
        parts.insert(0, r)
    for k in toks:
        check_both(getattr(got, k), torch.cat([getattr(r, k) for r in parts]), 4 * V * H + 512, k)
    check_both(got.state, g, 4 * K + 512, "state")
    for k in rest:
        want = sum(getattr(r, k).double() for r in parts)
        check(getattr(got, k), want, S * 64, k)
