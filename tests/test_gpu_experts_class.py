"""ExpertFFN on the GPU: the whole step closely, decoding, graphs whose routing changes (what it keeps: test_experts_class.py)."""
import pytest
import torch

import _experts_plain
import scaled_quantize_gemm_gb300 as sq
from _experts_ref import routing
from _ffn_ref import gen, randn
from scaled_quantize_gemm_gb300.experts import ExpertFFN

pytestmark = pytest.mark.gpu
DEV, BF = "cuda", torch.bfloat16


def _block(K, F, E, k, act, seed):
    g = gen(seed)
    w_gu = (randn(g, E, 2 * F, K) * K ** -0.5).to(BF)
    w_down = (randn(g, E, K, F) * F ** -0.5).to(BF)
    return ExpertFFN(randn(g, K) * 0.2 + 1, w_gu, w_down, k, act=act), g


def _route(g, T, k, E, how="masked"):
    return routing(g, T, k, E, how), torch.softmax(randn(g, T, k), 1)


def _step(b, x, way, dy):
    b.calibrate(x, *way)
    for _ in range(2):
        y = b.forward(x, *way)
        grads = b.backward(dy)
        b.update_scales()
    return [t.clone() for t in (y, *grads)], b.states.clone()


@pytest.mark.parametrize("act", [sq.ACT_SILU, sq.ACT_GELU])
@pytest.mark.parametrize("T,K,F,E,k,how", [(50, 256, 400, 6, 2, "masked"), (9, 544, 272, 33, 3, "spread"), (1500, 1056, 528, 4, 2, "skewed")])
def test_training_step_against_plain_arithmetic(T, K, F, E, k, how, act, monkeypatch):
    """The same class over plain fp32 forms of the entry points: the same casts, so the results differ where a value
    lies within fp32 rounding of a border between two codes, and by the rounding of bf16 outputs.  At most one code in
    a thousand a step (2^-3) off, sqrt(1e-3) 2^-3 = 0.4 % in norm for each of the seven operands that are cast, and
    2^-8 for each bf16 value (g and u, the rows, drows, dn, dx): below 1.5 % together."""
    b, g = _block(K, F, E, k, act, 7)
    x, dy, way = (randn(g, T, K) * 1.5).to(BF), (randn(g, T, K) * 1e-3).to(BF), _route(g, T, k, E, how)
    got, states = _step(b, x, way, dy)
    torch.cuda.synchronize()
    with monkeypatch.context() as mp:
        _experts_plain.install(mp)
        p = ExpertFFN(b.gamma, b.w_gate_up, b.w_down, k, act=act)
        want, plain_states = _step(p, x, way, dy)
    for name, a, w in zip(("y", "dx", "dweights", "dgamma", "dw_gate_up", "dw_down"), got, want):
        ref = (w - x if name == "y" else w - dy if name == "dx" else w).double()      # without the residual branch
        rest = 2.0 ** -8 * float(w.double().norm()) if a.dtype == BF else 0.0         # the output's own rounding
        assert float((a.double() - w.double()).norm()) <= 0.015 * float(ref.norm()) + rest, name
    assert float((states - plain_states).abs().max() / plain_states.abs().max()) <= 0.02
    assert sq.fp8_device_status(True) == sq.OK


def test_the_same_step_twice():
    outs = []
    for _ in range(2):
        b, g = _block(512, 256, 8, 2, sq.ACT_SILU, 3)
        x, dy, way = randn(g, 333, 512).to(BF), (randn(g, 333, 512) * 1e-3).to(BF), _route(g, 333, 2, 8)
        outs.append(_step(b, x, way, dy))
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(outs[0][0], outs[1][0])) and torch.equal(outs[0][1], outs[1][1])


K, F, E, k = 2048, 784, 24, 4


def _ready(seed):
    b, g = _block(K, F, E, k, sq.ACT_SILU, seed)
    b.calibrate(randn(g, 64, K).to(BF), *_route(g, 64, k, E, "spread"))
    b.freeze()
    return b, g


@pytest.mark.parametrize("warm", [True, False])
def test_graphs_of_several_batch_sizes_and_routings(warm):
    """Graphs of 1, 40 and 300 tokens, replayed after calls of other sizes, with the ids in place at the replay."""
    b, g = _ready(1)
    inputs = {n: (randn(g, n, K).to(BF), *_route(g, n, k, E, "spread")) for n in (1, 40, 300)}
    other = {n: routing(g, n, k, E, "masked") for n in inputs}
    want = {n: b.decode(*v) for n, v in inputs.items()}
    want_other = {n: b.decode(v[0], other[n], v[2]) for n, v in inputs.items()}
    fresh, _ = _ready(1)
    graphs, ys = {}, {}
    for n, v in inputs.items():
        ys[n] = torch.empty_like(v[0])
        if warm:
            fresh.decode(*v, ys[n])
        torch.cuda.synchronize()
        graphs[n] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[n]):
            fresh.decode(*v, ys[n])
    for wanted, ids in ((want, {n: v[1].clone() for n, v in inputs.items()}), (want_other, other), (want, {n: v[1].clone() for n, v in inputs.items()})):
        fresh.decode(randn(g, 77, K).to(BF), *_route(g, 77, k, E))
        for n in graphs:
            inputs[n][1].copy_(ids[n])
            ys[n].zero_()
            graphs[n].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(ys[n], wanted[n]) for n in graphs)
    assert sq.fp8_device_status(True) == sq.OK


def test_a_captured_training_step():
    """Forward and backward in one graph give what the calls give, for the routing at the replay."""
    b, g = _block(256, 208, 6, 2, sq.ACT_SILU, 5)
    T = 90
    x, dy, way = randn(g, T, 256).to(BF), (randn(g, T, 256) * 1e-3).to(BF), _route(g, T, 2, 6)
    b.calibrate(x, *way)
    b.forward(x, *way)
    b.backward(dy)
    b.update_scales()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = b.forward(x, *way)
        grads = b.backward(dy)
    for how in ("masked", "one", "spread"):
        way[0].copy_(routing(g, T, 2, 6, how))
        before = b.states.clone()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, *grads)]
        b.states = before
        want = [b.forward(x, *way), *b.backward(dy)]
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want)), how


@pytest.mark.parametrize("T", [1, 40, 300])
def test_decode_in_place_and_beside_a_step(T):
    b, g = _ready(6)
    x, way = randn(g, T, K).to(BF), _route(g, T, k, E)
    want = b.decode(x, *way)
    xt, dy, wt = randn(g, 48, K).to(BF), (randn(g, 48, K) * 1e-3).to(BF), _route(g, 48, k, E)
    b.forward(xt, *wt)
    grads = b.backward(dy)
    b.forward(xt, *wt)
    b.decode(randn(g, T, K).to(BF), *way)
    again = b.backward(dy)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(grads, again))
    b2, _ = _ready(6)
    y = x.clone()
    b2.decode(y, *way, y)
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_decode_after_a_wait_that_ran_out():
    b, g = _ready(8)
    x, way = randn(g, 3, K).to(BF), _route(g, 3, k, E, "spread")
    want = b.decode(x, *way).clone()
    waited = torch.zeros(1, dtype=torch.int32, device=DEV)
    assert sq.fp8_device_status(True) == sq.OK
    side = torch.cuda.Stream()
    for i in range(8):
        sq.fp8_selftest_wait_timeout(30 + 20 * i, waited, stream=side)
        for _ in range(20):
            b.decode(x, *way)
        torch.cuda.synchronize()
        assert sq.fp8_device_status(True) == sq.ERR_TIMEOUT
        b.reset_workspaces()
        assert torch.equal(b.decode(x, *way), want)
        assert sq.fp8_device_status(True) == sq.OK
