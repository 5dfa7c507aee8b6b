"""The gated delta rule and the norms on a stream of their own while the current
stream is busy, two calls at once, in graphs beside eager calls, and over more
than 2^31 elements."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import causal_conv_backward_gb300 as m  # noqa: E402
from ssm_reference import check  # noqa: E402
from test_delta_gpu import BF16, F32, FORMS, cuda_ready, inputs, lens, rand  # noqa: E402,F401

CYCLES = 100_000_000      # some 50 ms


def calls():
    S, B, H, G, K, V = 300, 2, 4, 2, 64, 64
    t, _, gy, gf = inputs(S, B, H, G, K, V)
    toks = [t[k] for k in ("q", "k", "v", "delta", "beta")]
    w, z, r = rand(V, seed=20), rand(S, B, H, V, seed=21), rand(S, B, 512, dtype=F32, seed=22)
    x, wr, post, scale, gr = rand(S, B, 512, seed=23), rand(512, seed=24), rand(512, seed=25), rand(512, dtype=F32, seed=26), rand(S, B, 512, seed=27)
    ln, kw = lens([S, 211]), dict(post_weight=post, scale=scale)
    return {
        "gated_delta": (m.gated_delta, (*toks, t["A"], t["delta_bias"]), dict(FORMS, state=t["state"], lengths=ln, return_state=True)),
        "gated_delta_backward": (m.gated_delta_backward, (gy, *toks, t["A"], t["delta_bias"]),
                                 dict(FORMS, state=t["state"], lengths=ln, grad_final_state=gf)),
        "gated_delta_step": (m.gated_delta_step, (*[v[0].contiguous() for v in toks], t["state"], t["A"], t["delta_bias"]), FORMS),
        "gated_norm": (m.gated_norm, (t["v"], z, w), {}),
        "gated_norm_backward": (m.gated_norm_backward, (gy, t["v"], z, w), {}),
        "residual_norm": (m.residual_norm, (x, r, wr), kw),
        "residual_norm_backward": (m.residual_norm_backward, (gr, rand(S, B, 512, dtype=F32, seed=28), x, r, wr), kw),
    }


NAMES = ("gated_delta", "gated_delta_backward", "gated_delta_step", "gated_norm", "gated_norm_backward", "residual_norm", "residual_norm_backward")


def call(name, c, **kw):
    """The outputs, the state that a step moves on among them."""
    f, args, own = c[name]
    out = f(*args, **own, **kw)
    out = list(out) if isinstance(out, tuple) else [out]
    return [t for t in out if t is not None] + ([args[5]] if name.endswith("step") else [])


def same(got, want):
    return all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", NAMES)
def test_current_stream_still_writes_freed_memory(name):
    want = [t.clone() for t in call(name, calls())]
    c, side = calls(), torch.cuda.Stream()
    torch.cuda.synchronize()
    old = [torch.empty_like(t) for t in want for _ in range(4)]
    torch.cuda._sleep(CYCLES)
    for t in old:
        t.fill_(float("nan"))
    del t, old                          # free for the current stream, which has yet to write them
    got = call(name, c, stream=side)
    torch.cuda.synchronize()
    assert same(got, want)


@pytest.mark.parametrize("name", NAMES)
def test_inputs_freed_while_the_stream_works(name):
    want = [t.clone() for t in call(name, calls())]
    c, side = calls(), torch.cuda.Stream()
    torch.cuda.synchronize()
    f, args, kw = c[name]
    sizes = [(t.shape, t.dtype) for t in (*args, *kw.values()) if isinstance(t, torch.Tensor)]
    with torch.cuda.stream(side):
        torch.cuda._sleep(CYCLES)
    got = call(name, c, stream=side)
    c.clear()
    del args, kw
    new = [torch.full(shape, 1, dtype=dtype, device="cuda") for shape, dtype in sizes for _ in range(4)]
    torch.cuda.synchronize()
    assert same(got, want) and len(new) > 0


def test_two_calls_at_once():
    """The same call on two streams, and others between: no state of the library's own."""
    c = calls()
    want = {n: [t.clone() for t in call(n, calls())] for n in NAMES}
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for n in NAMES:
        if n.endswith("step"):
            continue
        for s in streams:
            got.append((n, call(n, c, stream=s)))
    torch.cuda.synchronize()
    assert all(same(g, want[n]) for n, g in got)


def test_captured_beside_an_eager_graph_of_the_same_leaves():
    """Backward calls captured while gradients of the same tensors are pending."""
    c = calls()
    want = [t.clone() for t in call("gated_delta_backward", c)]
    leaf = c["gated_delta"][1][2].detach().clone().requires_grad_()
    eager = (leaf.float() ** 2).sum()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call("gated_delta_backward", c)
    eager.backward()
    for t in got:
        t.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    assert same(got, want)


def test_two_graphs_with_their_own_workspaces():
    a, b = calls(), calls()
    for t in b["gated_delta"][1][:3]:
        t.mul_(0.5)
    want = [[t.clone() for t in call("gated_delta_backward", c)] for c in (a, b)]
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for g, c in zip(graphs, (a, b)):
        with torch.cuda.graph(g):
            outs.append(call("gated_delta_backward", c))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert same(outs[0], want[0]) and same(outs[1], want[1])


def test_more_than_2_to_the_31_values():
    """Heads and sequences past 2^31 elements of v, against themselves alone."""
    S, B, H, G, K, V = 8300, 16, 128, 128, 16, 128
    assert S * B * H * V > 1 << 31

    def big(*shape, seed, dtype=BF16):
        g = torch.Generator(device="cuda").manual_seed(seed)
        return torch.empty(shape, device="cuda", dtype=dtype).normal_(generator=g)

    q, k, v, gy = (big(S, B, n, d, seed=i) for i, (n, d) in enumerate(((G, K), (G, K), (H, V), (H, V))))
    delta, beta, A = big(S, B, H, seed=5), big(S, B, H, seed=6), -torch.exp(big(H, seed=7, dtype=F32))
    y, state = m.gated_delta(q, k, v, delta, beta, A, return_state=True, **FORMS)
    g = m.gated_delta_backward(gy, q, k, v, delta, beta, A, **FORMS)
    w = rand(V, seed=8)
    n, gn = m.gated_norm(y, v, w), m.gated_norm_backward(gy, y, v, w)
    for b, h in ((0, 0), (B - 1, H - 1), (7, 63)):
        one = [t[:, b:b + 1, h:h + 1] for t in (q, k, v, delta, beta)]
        y1, s1 = m.gated_delta(*one, A[h:h + 1], return_state=True, **FORMS)
        # both are rounded: the difference of two, by halves
        both = lambda got, want, terms, what: check(got, (got.double() + want.double()) / 2, terms, what)  # noqa: E731
        both(y[:, b:b + 1, h:h + 1], y1, 512, "y")
        both(state[b:b + 1, h:h + 1], s1, 512, "state")
        g1 = m.gated_delta_backward(gy[:, b:b + 1, h:h + 1], *one, A[h:h + 1], **FORMS)
        for name in ("q", "k", "v", "delta", "beta"):
            both(getattr(g, name)[:, b:b + 1, h:h + 1], getattr(g1, name), 2048, name)
        part = [t[-64:, b:b + 1, h:h + 1] for t in (y, v, gy)]
        assert torch.equal(n[-64:, b:b + 1, h:h + 1], m.gated_norm(part[0], part[1], w))
        g2 = m.gated_norm_backward(part[2], part[0], part[1], w)
        assert torch.equal(gn.x[-64:, b:b + 1, h:h + 1], g2.x) and torch.equal(gn.z[-64:, b:b + 1, h:h + 1], g2.z)
