"""fp8_glu_bwd's codes, element by element, against central differences of the block's own formula.  The loss
sum(dh h(g, u)) is separable, so a difference in one g or u gives that element's gradient alone, and nothing cancels:
a wrong sign, a lost term or a permuted row is as large as the gradient itself."""
import pytest
import torch

import scaled_quantize_gemm_gb300 as sq
from _ffn_ref import GELU, GELU_TANH, NONE, SILU, act64, values
from test_gpu_ffn import _glu_bwd_case

pytestmark = pytest.mark.gpu
EPS = 1e-5               # central differences: EPS^2 / 6 of the third derivative (below 4) is 1e-10, rounding 1e-11


def _share_off(grad, want, m):
    """share of the elements farther off than the codes' rounding: half a step of E5M2, 2^-3 of the value (2^-17 of
    the scaled one below the normal range), and 2^-14 of it for the sums and the activation in fp32"""
    tol = (2.0 ** -3 + 2.0 ** -14) * torch.maximum(grad.abs(), want.abs()) + 2.0 ** -17 / m + 1e-9
    return float(((grad - want).abs() > tol).double().mean())


# one, few and many token tiles, a K that ends inside a block, more than one column tile
@pytest.mark.parametrize("M,F,K", [(1, 272, 144), (64, 272, 144), (300, 528, 1040)])
@pytest.mark.parametrize("act", [GELU, GELU_TANH, SILU, NONE])
def test_against_differences(M, F, K, act):
    dh, g, u, Q, m = _glu_bwd_case(M, F, K, act, 111)
    h = lambda g, u: act64(g, act)[0] * u                                                        # noqa: E731
    want = torch.cat([dh * (h(g + EPS, u) - h(g - EPS, u)), dh * (h(g, u + EPS) - h(g, u - EPS))], 1) / (2 * EPS)
    assert float(want.abs().max()) * m < 57344 and float(want.abs().median()) * m > 2.0 ** -10
    grad = values(Q, sq.E5M2) / m
    assert _share_off(grad, want, m) == 0.0
    # what the comparison has to see
    dg, du = grad[:, :F], grad[:, F:]
    wrong = {"negated": -grad, "without dg": torch.cat([0 * dg, du], 1), "without du": torch.cat([dg, 0 * du], 1),
             "dg and du exchanged": torch.cat([du, dg], 1), "too large": grad * 1.4}
    if M > 1:
        wrong["rows moved"] = grad.roll(1, 0)
    for name, bad in wrong.items():
        assert _share_off(bad, want, m) > 0.3, name
