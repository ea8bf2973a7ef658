"""GatedFFN: the operators together, against the sublayer in 64 bits.

Bounds: a code is within half a step, 2^-4 of its value in E4M3 and 2^-3 in
E5M2 (values below the normal range, a small share of each tensor here, less
in absolute terms).  An output that goes through n casted operands is then off
by at most about the sum of their relative errors in norm: y's branch passes n,
W_gu twice (g and u), h and W_down, 6 x 2^-4 at the very worst, and errors of
independent signs add in squares: sqrt(6) 2^-4 = 0.153.  A gradient adds dY (and
dg | du) in E5M2: sqrt(6 x 2^-8 + 2 x 2^-6) = 0.234.
"""
import pytest
import torch

import scaled_quantize_gemm_gb300 as sq
from _ffn_ref import act64, gen, randn
from scaled_quantize_gemm_gb300.ffn import GatedFFN

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def _block(K, F, act, seed):
    g = gen(seed)
    gamma, beta = randn(g, K) * 0.2 + 1, randn(g, K) * 0.1
    w_gu = (randn(g, 2 * F, K) * K ** -0.5).to(BF)
    w_d = (randn(g, K, F) * F ** -0.5).to(BF)
    return GatedFFN(gamma, beta, w_gu, w_d, act=act), g


def _block64(b, x):
    """(output, parameters) of the sublayer in 64 bits, for autograd"""
    p = [t.double().requires_grad_() for t in (x, b.gamma, b.beta, b.w_gate_up, b.w_down)]
    x64, gamma, beta, w_gu, w_d = p
    mu = x64.mean(1, keepdim=True)
    n = (x64 - mu) * ((x64 - mu).square().mean(1, keepdim=True) + b.eps).rsqrt() * gamma + beta
    z = n @ w_gu.T
    g, u = z[:, :b.F], z[:, b.F:]
    return x64 + (act64(g, b.act)[0] * u) @ w_d.T, p


def _off(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("act", [sq.ACT_SILU, sq.ACT_GELU_TANH, sq.ACT_GELU])
@pytest.mark.parametrize("M,K,F", [(48, 256, 400), (272, 528, 1040), (512, 1024, 2064)])
def test_training_step(M, K, F, act):
    b, g = _block(K, F, act, M + act)
    x, dy = (randn(g, M, K) * 1.5).to(BF), (randn(g, M, K) * 1e-3).to(BF)
    b.calibrate(x)
    for _ in range(2):                       # the gradients' scales come from the first step's history
        y = b.forward(x)
        grads = b.backward(dy)
        b.update_scales()
    torch.cuda.synchronize()
    y64, p = _block64(b, x)
    y64.backward(dy.double())
    y64 = y64.detach()
    assert _off(y.double() - x.double(), y64 - x.double()) <= 0.153 + 2.0 ** -8 * float(y64.norm() / (y64 - x.double()).norm())
    for name, got, ref in zip(("dx", "dgamma", "dbeta", "dw_gate_up", "dw_down"), grads, p):
        assert _off(got, ref.grad) <= 0.234, name
    assert sq.fp8_device_status(True) == sq.OK


@pytest.mark.parametrize("M", [1, 5, 33, 64, 200])
def test_decode_agrees_with_the_training_forward(M):
    """The few-rows kernels and the tiled ones take the same codes of the input; their sums differ in order only, so
    codes of h may differ where a value lies within that rounding of a border between two codes."""
    K, F = 1024, 2064
    b, g = _block(K, F, sq.ACT_SILU, 3)
    x = (randn(g, 208, K) * 1.5).to(BF)
    b.calibrate(x)
    y = b.forward(x)
    b.freeze()
    got = b.decode(x[:M].contiguous())
    torch.cuda.synchronize()
    branch = (y[:M].double() - x[:M].double())
    # half a step of bf16 on each side, and a code step (2^-3) on at most one h in a thousand
    assert float((got.double() - y[:M].double()).norm()) <= 2.0 ** -7 * float(y[:M].double().norm()) + \
        2.0 ** -3 * 1e-3 ** 0.5 * float(branch.norm())


def test_decode_in_a_graph():
    K, F = 528, 784
    b, g = _block(K, F, sq.ACT_SILU, 4)
    b.calibrate((randn(g, 64, K)).to(BF))
    b.freeze()
    x = randn(g, 3, K).to(BF)
    y = torch.empty_like(x)
    b.decode(x, y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.decode(x, y)
    x.copy_(randn(g, 3, K))
    graph.replay()
    torch.cuda.synchronize()
    replayed = y.clone()
    b.decode(x, y)
    torch.cuda.synchronize()
    assert torch.equal(replayed, y)


def test_refusals():
    z = lambda *s: torch.zeros(s, dtype=BF, device=DEV)                                          # noqa: E731
    one = torch.ones(32, device=DEV)
    with pytest.raises(ValueError, match="gated block"):
        GatedFFN(one, None, z(64, 32), z(32, 48))
    with pytest.raises(ValueError, match="gated block"):
        GatedFFN(one, None, z(72, 32), z(32, 36))
    b = GatedFFN(one, None, z(64, 32), z(32, 32))
    with pytest.raises(RuntimeError, match="without a forward"):
        b.backward(z(16, 32))
    b.forward(z(5, 32))
    with pytest.raises(ValueError, match="multiple of 16"):
        b.backward(z(5, 32))
