"""What ExpertFFN keeps between its calls, on the CPU (entry points: _experts_plain.py)."""
import pytest
import torch

import _experts_plain
import scaled_quantize_gemm_gb300 as sq
from _experts_ref import routing
from _ffn_ref import gen, randn
from scaled_quantize_gemm_gb300.experts import DY, ExpertFFN

BF = torch.bfloat16
K, F, E, k, T = 32, 48, 5, 2, 20


@pytest.fixture
def block(monkeypatch):
    _experts_plain.install(monkeypatch)
    g = gen(1, "cpu")
    r = lambda *s: randn(g, *s, device="cpu")                                                     # noqa: E731
    route = lambda n, how="masked": (routing(g, n, k, E, how, "cpu"), torch.rand((n, k), generator=g))    # noqa: E731
    b = ExpertFFN(r(K) * 0.2 + 1, (r(E, 2 * F, K) * K ** -0.5).to(BF), (r(E, K, F) * F ** -0.5).to(BF), k)
    b.calibrate(r(64, K).to(BF), *route(64, "spread"))
    for _ in range(2):                       # scales of the gradients
        b.forward(r(T, K).to(BF), *route(T))
        b.backward(r(T, K).to(BF))
        b.update_scales()
    return b, r, route


def _same(p, q):
    return all(torch.equal(a, b) for a, b in zip(p, q))


@pytest.mark.parametrize("tokens", [T, 5, 64])
def test_decode_between_forward_and_backward(block, tokens):
    b, r, route = block
    x, dy, x2, way = r(T, K).to(BF), r(T, K).to(BF), r(tokens, K).to(BF), route(T)
    b.forward(x, *way)
    want = b.backward(dy)
    b.forward(x, *way)
    b.decode(x2, *route(tokens))
    assert _same(b.backward(dy), want)


def test_scales_updated_within_a_step(block):
    """Codes are turned back with the steps they were cast with."""
    b, r, route = block
    x, dy, way = r(T, K).to(BF), r(T, K).to(BF), route(T)
    b.forward(x, *way)
    want = b.backward(dy)
    b.forward(x, *way)
    n = b.H + 2
    gradients = b.states[DY * n:(DY + 2) * n].clone()
    for s in b._live[0]:
        s[0] = 9.0
    b.update_scales()
    b.states[DY * n:(DY + 2) * n] = gradients
    assert _same(b.backward(dy), want)


def test_decode_on_frozen_weights(block):
    b, r, route = block
    x, way = r(7, K).to(BF), route(7)
    b.freeze()
    want = b.decode(x, *way)
    b.w_down.mul_(2)
    b.update_scales()
    assert torch.equal(b.decode(x, *way), want)
    y = x.clone()
    assert b.decode(y, *way, y) is y and torch.equal(y, want)
    b.freeze()
    assert not torch.equal(b.decode(x, *way), want)


def test_experts_have_scales_of_their_own(block):
    b, r, route = block
    b.w_gate_up[3].mul_(1000)
    for _ in range(2):
        b.freeze()
        b.update_scales()
    b.freeze()
    steps = b._w_steps[:E]
    assert bool((steps[3] > 100 * steps[[0, 1, 2, 4]]).all())


def test_no_tokens_and_no_experts(block):
    b, r, route = block
    x, way = r(T, K).to(BF), route(T, "none")
    assert torch.equal(b.forward(x, *way), x)
    dy = r(T, K).to(BF)
    dx, dw, dgamma, dgu, dd = b.backward(dy)
    assert torch.equal(dx, dy) and not any(bool(t.any()) for t in (dw, dgamma, dgu, dd))
    assert b.decode(x[:0], way[0][:0], way[1][:0]).shape == (0, K)


def test_many_states_are_updated_in_parts(monkeypatch):
    _experts_plain.install(monkeypatch)
    seen = []
    update = _experts_plain.update_scale
    monkeypatch.setattr(sq, "fp8_update_scale", lambda s, n, H, f: (seen.append((n, len(f))), update(s, n, H, f)))
    b = ExpertFFN(torch.ones(32), torch.zeros((600, 32, 32), dtype=BF), torch.zeros((600, 32, 16), dtype=BF), 1)
    b.update_scales()
    assert seen == [(1024, 1024), (180, 180)]


def test_refusals(block):
    b, r, route = block
    x, way = r(T, K).to(BF), route(T)
    with pytest.raises(RuntimeError, match="without a forward"):
        b.backward(x)
    with pytest.raises(ValueError, match="ids"):
        b.forward(x, way[0][1:], way[1])
    with pytest.raises(ValueError, match="ids"):
        b.decode(x, way[0], way[1][:, :1])
    b.forward(x, *way)
    with pytest.raises(ValueError, match="dy"):
        b.backward(x.float())
    b.backward(x)                            # (a refused call keeps the forward)
    fresh = ExpertFFN(b.gamma, b.w_gate_up, b.w_down, k)
    with pytest.raises(RuntimeError, match="freeze"):
        fresh.decode(x, *way)
    for bad in (dict(top_k=0), dict(top_k=65), dict(w_down=b.w_down[:4]), dict(w_gate_up=b.w_gate_up[:, :, :16])):
        with pytest.raises(ValueError):
            ExpertFFN(**{**dict(gamma=b.gamma, w_gate_up=b.w_gate_up, w_down=b.w_down, top_k=k), **bad})
