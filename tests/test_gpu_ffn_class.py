"""GatedFFN's calls beside each other on the GPU: graphs of several batch sizes, decoding during a training step, and
scales that move (on the CPU, over plain forms of the entry points: test_ffn_class.py)."""
import pytest
import torch

import scaled_quantize_gemm_gb300 as sq
from _ffn_ref import randn
from test_gpu_ffn_block import BF, DEV, _block

pytestmark = pytest.mark.gpu
K, F = 1040, 5200                            # the up projection splits K through the workspace for a few tokens


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
