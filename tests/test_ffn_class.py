"""What GatedFFN keeps between its calls, on the CPU (entry points: _ffn_plain.py)."""
import weakref

import pytest
import torch

import _ffn_plain
import scaled_quantize_gemm_gb300 as sq
from _ffn_ref import gen, randn
from scaled_quantize_gemm_gb300 import ffn
from scaled_quantize_gemm_gb300.ffn import GatedFFN

BF = torch.bfloat16
K, F, M = 32, 48, 16


@pytest.fixture
def block(monkeypatch):
    _ffn_plain.install(monkeypatch)
    g = gen(1, "cpu")
    r = lambda *s: randn(g, *s, device="cpu")                                                     # noqa: E731
    b = GatedFFN(r(K) * 0.2 + 1, r(K), (r(2 * F, K) * K ** -0.5).to(BF), (r(K, F) * F ** -0.5).to(BF))
    b.calibrate(r(64, K).to(BF))
    for _ in range(2):                       # scales of the gradients
        b.forward(r(M, K).to(BF))
        b.backward(r(M, K).to(BF))
        b.update_scales()
    return b, r


def _same(p, q):
    return all(torch.equal(a, b) for a, b in zip(p, q))


# ---------------------------------------------------------------- decode beside a training step
@pytest.mark.parametrize("tokens", [M, 5, 64])
def test_decode_between_forward_and_backward(block, tokens):
    """Generating during a training step leaves the step's gradients alone, whatever its number of tokens."""
    b, r = block
    x, dy, x2 = r(M, K).to(BF), r(M, K).to(BF), r(tokens, K).to(BF)
    b.forward(x)
    want = b.backward(dy)
    b.forward(x)
    b.decode(x2)
    assert _same(b.backward(dy), want)


def test_a_refused_backward_keeps_the_forward(block):
    """A number of tokens that the weight gradients do not take is refused before anything is dropped."""
    b, r = block
    b.forward(r(5, K).to(BF))
    for _ in range(2):
        with pytest.raises(ValueError, match="multiple of 16"):
            b.backward(r(5, K).to(BF))


# ---------------------------------------------------------------- buffers that a captured graph may hold
@pytest.fixture
def made(monkeypatch):
    """weak references to every tensor that torch.empty and torch.zeros make, in order"""
    refs = []
    for name in ("empty", "zeros"):
        def make(*a, _f=getattr(torch, name), **kw):
            t = _f(*a, **kw)
            refs.append(weakref.ref(t))
            return t
        monkeypatch.setattr(torch, name, make)
    return refs


def test_buffers_outlive_other_batch_sizes(made, block):
    """What a call of 100 tokens uses (and a graph of it replays on) still exists after calls of 105, 300 and 1."""
    b, r = block
    x, y = r(100, K).to(BF), torch.empty(100, K, dtype=BF)
    before = len(made)
    b.decode(x, y)
    mine = made[before:]
    assert len(mine) == 4                    # the codes of n and h, two workspaces
    for tokens in (105, 300, 1):
        b.decode(r(tokens, K).to(BF))
    assert all(w() is not None for w in mine)


def test_training_buffers_outlive_other_batch_sizes(made, block):
    b, r = block

    def step(tokens):
        b.forward(r(tokens, K).to(BF))
        return b.backward(r(tokens, K).to(BF))

    before = len(made)
    grads = step(8 * M)                      # larger than the fixture's: new buffers
    mine = [w for w in made[before:] if not any(w() is t for t in grads)]
    mine = [w for w in mine if w() is not None]           # (the output y is the caller's)
    assert len(mine) >= 7
    step(M)
    step(17 * M)
    assert all(w() is not None for w in mine)


def test_growing_batches_keep_little(made, block):
    """The buffers grow by doubling: what is kept of all the smaller ones is no more than the largest."""
    b, r = block
    before = len(made)
    for tokens in range(1, 65):
        b.decode(r(tokens, K).to(BF))
    alive = [w() for w in made[before:] if w() is not None]
    assert sum(t.numel() for t in alive) <= 4 * 64 * (K + F + 64 + 64)


def test_a_call_without_tokens(block):
    b, r = block
    assert b.decode(r(0, K).to(BF)).shape == (0, K)


def test_a_buffer_made_during_a_capture_stays_with_the_graph(made, block, monkeypatch):
    """Its memory and its zeros come with the replay: calls outside the graph get others."""
    b, r = block
    x = r(100, K).to(BF)
    before = len(made)
    with monkeypatch.context() as mp:
        mp.setattr(ffn, "_capturing", lambda: True)
        b.decode(x, torch.empty_like(x))
    graph = made[before:]
    assert len(graph) == 4 and all(w() is not None for w in graph)
    before = len(made)
    b.decode(x, torch.empty_like(x))
    assert len(made) == before + 4
    b.decode(x, torch.empty_like(x))
    assert len(made) == before + 4


# ---------------------------------------------------------------- scales that move
def _move(b):
    """what an update does once the maxima have moved"""
    for i in range(6):
        b._state(i)[0] = 7.0 + i
    b.update_scales()


def test_scales_updated_between_forward_and_backward(block):
    """The backward pass takes the forward's codes back with the steps that they were cast with."""
    b, r = block
    x, dy = r(M, K).to(BF), r(M, K).to(BF)
    b.forward(x)
    want = b.backward(dy)
    b.forward(x)
    gradients = b.states[4 * (b.H + 2):].clone()
    _move(b)
    b.states[4 * (b.H + 2):] = gradients     # dY and [dg | du] are cast in the backward pass, with the newest
    assert _same(b.backward(dy), want)


def test_scales_updated_between_freeze_and_decode(block):
    b, r = block
    x = r(7, K).to(BF)
    b.freeze()
    want = b.decode(x)
    _move(b)
    assert torch.equal(b.decode(x), want)
    b.freeze()
    moved = b.decode(x)
    assert not torch.equal(moved, want)
    assert float((moved.float() - want.float()).norm()) <= 0.3 * float((want.float() - x.float()).norm())


def test_freeze_between_forward_and_backward(block):
    """The weights' codes and their step change together."""
    b, r = block
    x, dy = r(M, K).to(BF), r(M, K).to(BF)
    b.forward(x)
    want = b.backward(dy)
    b.forward(x)
    gradients = b.states[4 * (b.H + 2):].clone()
    _move(b)
    b.freeze()
    b.states[4 * (b.H + 2):] = gradients
    for p, q in zip(b.backward(dy), want):
        assert float((p.float() - q.float()).norm()) <= 0.3 * float(q.float().norm())


def test_decode_leaves_the_training_statistics(block):
    """Serving a sequence with large values does not move the scales of the training step."""
    b, r = block
    b.freeze()
    states = b.states.clone()
    b.decode((r(9, K) * 1000).to(BF))
    assert torch.equal(b.states, states)


def test_decode_needs_codes(monkeypatch):
    """Weights that were never cast are refused, not read."""
    _ffn_plain.install(monkeypatch)
    g = gen(2, "cpu")
    b = GatedFFN(torch.ones(K), None, randn(g, 2 * F, K, device="cpu").to(BF), randn(g, K, F, device="cpu").to(BF))
    with pytest.raises(RuntimeError, match="freeze"):
        b.decode(torch.zeros(3, K, dtype=BF))
    b.freeze()
    b.decode(torch.zeros(3, K, dtype=BF))


# ---------------------------------------------------------------- after a wait that ran out
def test_workspaces_can_be_zeroed_again(block, monkeypatch):
    """A kernel that gave up leaves counters behind; the plain forms refuse a workspace that is not zero."""
    b, r = block
    b.freeze()
    x = r(100, K).to(BF)
    want = b.decode(x)
    with monkeypatch.context() as mp:        # a workspace of a captured graph
        mp.setattr(ffn, "_capturing", lambda: True)
        b.decode(r(300, K).to(BF))
    b.decode(r(120, K).to(BF))               # ... and one that a larger one has replaced
    spaces = list(b._spaces)
    assert len(spaces) >= 4
    for t in spaces:
        t[3] = 1
    with pytest.raises(AssertionError, match="not zero"):
        b.decode(x)
    b.reset_workspaces()
    assert torch.equal(b.decode(x), want)
    assert not any(bool(t.any()) for t in spaces)


def test_states_of_a_checkpoint(block):
    """Assigned or copied, they are what the next step and the next freeze take."""
    b, r = block
    x, saved = r(7, K).to(BF), b.states.clone()
    b.freeze()
    want = b.decode(x)
    where = b.states.data_ptr()
    _move(b)
    b.states = saved
    assert b.states.data_ptr() == where and torch.equal(b.states, saved)
    b.freeze()
    assert torch.equal(b.decode(x), want)


# ---------------------------------------------------------------- refusals
def test_a_gradient_of_another_form_is_refused_before_anything_runs(block):
    b, r = block
    x, dy = r(M, K).to(BF), r(M, K).to(BF)
    b.forward(x)
    want = b.backward(dy)
    b.forward(x)
    states = b.states.clone()
    for bad in (r(M - 1, K).to(BF), r(M, K), r(K, M).to(BF).T, r(M * K).to(BF)):
        with pytest.raises(ValueError, match="dy"):
            b.backward(bad)
    assert torch.equal(b.states, states)
    assert _same(b.backward(dy), want)
