"""The activations over their whole range, relative to their own value: the tails, where act(x) is far smaller than x,
as an fp32 output gives them.

Bound.  kappa = |x act'(x) / act(x)| says by how many relative units act moves for one of its argument's; an fp32
argument carries half a unit (2^-24) anyhow.  The exponential's argument is rounded two or three times (2^-24 of
it each), which is worth at most 2 kappa 2^-23 of the result; beside that 12 x 2^-23: 2 for the hardware exponential, 3
for the reciprocal with its argument and its use, 4 for the polynomial (its fit and its roundings), 3 for products."""
import pytest
import torch

import scaled_quantize_gemm_gb300 as sq
from _ffn_kernels import KSPLIT, PAIR, ROWS, expected
from _ffn_ref import ACTS, GELU, GELU_TANH, NONE, RELU, SILU, act64
from test_gpu_ffn import BF, DEV, F32, _empty

pytestmark = pytest.mark.gpu
V = 2.0 ** -23
FLOOR = 2.0 ** -115            # of the results looked at relatively; below, exp leaves fp32's normal range


def _arguments(n):
    x = torch.cat([-torch.linspace(0, 14, n // 4, device=DEV), torch.linspace(0, 14, n // 4, device=DEV),
                   -torch.logspace(-30, 2, n // 4, device=DEV), torch.logspace(-30, 2, n - 3 * (n // 4), device=DEV)])
    return x.contiguous()


# the epilogues of all three kernels: the sums are zero, the bias is the argument
@pytest.mark.parametrize("kernel,M,N,K", [(ROWS, 2, 20480, 128), (KSPLIT, 2, 4096, 2048), (PAIR, 2300, 5440, 2064)])
@pytest.mark.parametrize("act", [a for a in ACTS if a != NONE])
def test_values_in_the_tails(kernel, M, N, K, act):
    A, B = torch.zeros((M, K), dtype=torch.uint8, device=DEV), torch.zeros((N, K), dtype=torch.uint8, device=DEV)
    one, x, D = torch.ones(1, device=DEV), _arguments(N), _empty(M, N, dtype=F32)
    with expected(kernel, "fp8_gemm_act"):
        sq.fp8_gemm_act(A, 0, one, B, 0, one, act, D=D, bias=x)
    torch.cuda.synchronize()
    f, d = act64(x.double(), act)
    if act == GELU:
        f = 0.5 * x.double() * torch.special.erfc(-x.double() / 2 ** 0.5)         # (1 + erf cancels in the tail)
        d = 0.5 * torch.special.erfc(-x.double() / 2 ** 0.5) + x.double() * torch.exp(-0.5 * x.double() ** 2) / (2 * torch.pi) ** 0.5
    elif act == GELU_TANH:
        u = 2 * (2 / torch.pi) ** 0.5 * x.double() * (1 + 0.044715 * x.double() ** 2)
        s = torch.sigmoid(u)
        f = x.double() * s
        d = s + f * torch.sigmoid(-u) * 2 * (2 / torch.pi) ** 0.5 * (1 + 3 * 0.044715 * x.double() ** 2)
    tol = V * (12 * f.abs() + 2 * (x.double() * d).abs())
    if act == RELU:
        tol = 0 * tol
    err = (D[M - 1].double() - f).abs()
    seen = f.abs() > FLOOR
    assert int(seen.sum()) > 0.7 * N or act == RELU
    over = (err > tol) & seen
    i = int((err / (tol + 1e-300) * seen).argmax())
    assert not bool(over.any()), f"{int(over.sum())} of {N}, worst at {float(x[i])}: {float(D[M - 1, i])} against {float(f[i])}"
    assert bool((err[~seen] <= 2.0 ** -110).all())
    assert torch.equal(D[0], D[M - 1])


@pytest.mark.parametrize("act", [GELU, GELU_TANH, SILU])
def test_derivatives_in_the_tails(act):
    """dz = act'(z) in bf16: half a step of it beside the bound, with the derivative's two terms for its magnitude."""
    z = _arguments(32768).to(BF).view(8, 4096)
    dz = _empty(8, 4096, dtype=BF)
    sq.fp8_act_bwd(torch.ones_like(z), z, act, dz=dz)
    torch.cuda.synchronize()
    x = z.double()
    if act == GELU:
        a, b = 0.5 * torch.special.erfc(-x / 2 ** 0.5), x * torch.exp(-0.5 * x * x) / (2 * torch.pi) ** 0.5
        k = x * x
    else:
        c, q = (1.0, 0.0) if act == SILU else (2 * (2 / torch.pi) ** 0.5, 0.044715)
        u = c * x * (1 + q * x * x)
        a, b = torch.sigmoid(u), x * torch.sigmoid(u) * torch.sigmoid(-u) * c * (1 + 3 * q * x * x)
        k = (x * c * (1 + 3 * q * x * x)).abs()
    want = a + b
    tol = V * (12 + 2 * k) * (a.abs() + b.abs()) + 2.0 ** -8 * want.abs()
    seen = want.abs() > FLOOR
    over = ((dz.double() - want).abs() > tol) & seen
    assert not bool(over.any()), f"{int(over.sum())}: at {x[over][:4].tolist()} {dz[over][:4].tolist()} against {want[over][:4].tolist()}"
