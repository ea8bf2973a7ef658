"""What GatedFFN keeps between its calls, on the CPU (entry points: _ffn_plain.py)."""
import pytest
import torch

import _ffn_plain
import scaled_quantize_gemm_gb300 as sq
from _ffn_ref import gen, randn
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
