"""GatedFFN's calls beside each other on the GPU: graphs of several batch sizes, decoding during a training step, and
scales that move (on the CPU, over plain forms of the entry points: test_ffn_class.py)."""
import pytest
import torch

import _ffn_plain
import scaled_quantize_gemm_gb300 as sq
from _ffn_ref import randn
from scaled_quantize_gemm_gb300.ffn import GatedFFN
from test_gpu_ffn_block import BF, DEV, _block

pytestmark = pytest.mark.gpu
K, F = 4112, 5200                            # the up projection of a few tokens splits K through the workspace


def _ready(seed):
    b, g = _block(K, F, sq.ACT_SILU, seed)
    b.calibrate(randn(g, 64, K).to(BF))
    b.freeze()
    return b, g


@pytest.mark.parametrize("warm", [True, False])
def test_graphs_of_several_batch_sizes(warm):
    """Graphs of 3 and 40 tokens, with and without a call before the capture, replayed after calls of other sizes and
    after the memory that was free then has been written."""
    b, g = _ready(1)
    xs = {n: randn(g, n, K).to(BF) for n in (3, 40)}
    ys, graphs = {}, {}
    want = {n: _ready(1)[0].decode(x).clone() for n, x in xs.items()}
    torch.cuda.synchronize()
    for n, x in xs.items():
        ys[n] = torch.empty_like(x)
        if warm:
            b.decode(x, ys[n])
        torch.cuda.synchronize()
        graphs[n] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[n]):
            b.decode(x, ys[n])
    for round_ in range(2):
        for n in (5, 200, 1):
            b.decode(randn(g, n, K).to(BF))
        torch.cuda.synchronize()
        junk = [torch.full((s,), 0x7F, dtype=torch.uint8, device=DEV) for s in (1 << 12, 1 << 16, 1 << 20, 1 << 24) for _ in range(8)]
        torch.cuda.synchronize()
        for n in graphs:
            ys[n].zero_()
            graphs[n].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(ys[n], want[n]) for n in graphs)
        assert all(bool((j == 0x7F).all()) for j in junk)
        del junk
    assert sq.fp8_device_status(True) == sq.OK


@pytest.mark.parametrize("tokens", [48, 3, 200])
def test_decode_between_forward_and_backward(tokens):
    b, g = _ready(2)
    x, dy, x2 = randn(g, 48, K).to(BF), (randn(g, 48, K) * 1e-3).to(BF), randn(g, tokens, K).to(BF)
    for _ in range(2):
        b.forward(x)
        b.backward(dy)
        b.update_scales()
    b.forward(x)
    want = [t.clone() for t in b.backward(dy)]
    b.forward(x)
    b.decode(x2)
    got = b.backward(dy)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def _move(b):
    for i in range(6):
        b._state(i)[0] = 7.0 + i
    b.update_scales()


def test_scales_updated_within_a_step():
    b, g = _ready(3)
    x, dy = randn(g, 48, K).to(BF), (randn(g, 48, K) * 1e-3).to(BF)
    for _ in range(2):
        b.forward(x)
        b.backward(dy)
        b.update_scales()
    b.forward(x)
    want = [t.clone() for t in b.backward(dy)]
    b.forward(x)
    gradients = b.states[4 * (b.H + 2):].clone()
    _move(b)
    b.states[4 * (b.H + 2):] = gradients
    got = b.backward(dy)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_a_graph_follows_the_weights_that_are_frozen():
    """A graph of decode reads the codes and the scales where freeze writes them."""
    b, g = _ready(4)
    x = randn(g, 3, K).to(BF)
    y = torch.empty_like(x)
    b.decode(x, y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.decode(x, y)
    before = y.clone()
    _move(b)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, before)
    b.w_down.mul_(-2)
    b.freeze()
    graph.replay()
    torch.cuda.synchronize()
    replayed = y.clone()
    assert torch.equal(b.decode(x), replayed) and not torch.equal(replayed, before)


@pytest.mark.parametrize("M", [1, 40, 300])
def test_decode_in_place(M):
    b, g = _ready(6)
    x = randn(g, M, K).to(BF)
    want = b.decode(x)
    b.decode(x, x)
    torch.cuda.synchronize()
    assert torch.equal(x, want)


def test_decode_after_a_wait_that_ran_out():
    """The status is read and cleared, the workspaces zeroed, and decode is right again."""
    b, g = _ready(5)
    x = randn(g, 3, K).to(BF)
    want = b.decode(x).clone()
    waited = torch.zeros(1, dtype=torch.int32, device=DEV)
    assert sq.fp8_device_status(True) == sq.OK
    side = torch.cuda.Stream()
    for i in range(8):
        sq.fp8_selftest_wait_timeout(30 + 20 * i, waited, stream=side)
        for _ in range(20):
            b.decode(x)
        torch.cuda.synchronize()
        assert sq.fp8_device_status(True) == sq.ERR_TIMEOUT
        b.reset_workspaces()
        assert torch.equal(b.decode(x), want)
        assert sq.fp8_device_status(True) == sq.OK


# ---------------------------------------------------------------- the whole step, closely
def _step(b, x, dy):
    b.calibrate(x)
    for _ in range(2):
        y = b.forward(x)
        grads = b.backward(dy)
        b.update_scales()
    return [t.clone() for t in (y, *grads)], b.states.clone()


@pytest.mark.parametrize("act", [sq.ACT_SILU, sq.ACT_GELU])
@pytest.mark.parametrize("M,K,F", [(48, 256, 400), (272, 528, 1040), (2304, 1040, 2064)])
def test_training_step_against_plain_arithmetic(M, K, F, act, monkeypatch):
    """The same class over plain fp32 forms of the entry points: the same casts, so the results differ where a value
    lies within fp32 rounding of a border between two codes, and by the rounding of bf16 outputs.  At most one code in
    a thousand a step (2^-3) off, sqrt(1e-3) 2^-3 = 0.4 % in norm for each of the seven operands that are cast, and
    2^-8 for each bf16 value (g and u, dn, dx): below 1.5 % together.  A gradient that is 10 % off, or has lost one of its
    terms, is not."""
    b, g = _block(K, F, act, 7)
    x, dy = (randn(g, M, K) * 1.5).to(BF), (randn(g, M, K) * 1e-3).to(BF)
    got, states = _step(b, x, dy)
    torch.cuda.synchronize()
    with monkeypatch.context() as mp:
        _ffn_plain.install(mp)
        p = GatedFFN(b.gamma, b.beta, b.w_gate_up, b.w_down, act=act)
        want, plain_states = _step(p, x, dy)
    for name, a, w in zip(("y", "dx", "dgamma", "dbeta", "dw_gate_up", "dw_down"), got, want):
        ref = (w - x if name == "y" else w - dy if name == "dx" else w).double()      # without the residual branch
        rest = 2.0 ** -8 * float(w.double().norm()) if a.dtype == BF else 0.0         # the output's own rounding
        assert float((a.double() - w.double()).norm()) <= 0.015 * float(ref.norm()) + rest, name
    assert float((states - plain_states).abs().max() / plain_states.abs().max()) <= 0.02
    assert sq.fp8_device_status(True) == sq.OK
