"""Outputs over other buffers of a call: refused on the host, but for the residual stream in place, which gives what
separate buffers give."""
import pytest
import torch

import scaled_quantize_gemm_gb300 as sq
from _ffn_kernels import KSPLIT, PAIR, ROWS, expected
from _ffn_ref import GELU, NONE, SILU, gen, new_state, randn, to_codes
from test_gpu_ffn import BF, DEV, F32, H, _workspace

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kernel,M,N,K", [(PAIR, 2300, 5440, 1616), (ROWS, 5, 10256, 8208), (ROWS, 64, 20496, 2064),
                                          (KSPLIT, 70, 4096, 4096)])
def test_product_over_its_residual(kernel, M, N, K, dtype):
    g = gen(M)
    A, sa = to_codes(randn(g, M, K), 0)
    B, sb = to_codes(randn(g, N, K), 0)
    R, bias, D = randn(g, M, N).to(dtype), randn(g, N), torch.empty(M, N, dtype=dtype, device=DEV)
    ws = _workspace(sq.fp8_gemm_act_workspace_bytes(M, N, K))
    with expected(kernel, "fp8_gemm_act"):
        sq.fp8_gemm_act(A, 0, sa, B, 0, sb, SILU, D=D, bias=bias, residual=R, workspace=ws)
    sq.fp8_gemm_act(A, 0, sa, B, 0, sb, SILU, D=R, bias=bias, residual=R, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(D, R)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,K", [(1000, 4096), (700, 1535), (300, 2050), (333, 7), (40, 20001)])
@pytest.mark.parametrize("over", ["residual", "x"])
def test_layernorm_sum_in_place(M, K, dtype, over):
    g = gen(M + K)
    x, r = randn(g, M, K).to(dtype), randn(g, M, K).to(dtype)
    gamma, beta = randn(g, K), randn(g, K)
    outs = []
    for in_place in (False, True):
        y, mu, rstd = torch.empty_like(x), torch.empty(M, device=DEV), torch.empty(M, device=DEV)
        a, b = x.clone(), r.clone()
        s = (b if over == "residual" else a) if in_place else torch.empty_like(x)
        sq.fp8_layernorm_fwd(a, gamma, beta, 1e-5, y, mu=mu, rstd=rstd, residual=b, sum_out=s)
        outs.append((y, mu, rstd, s))
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(*outs))


def _refused(call, *names):
    with pytest.raises(sq.Fp8Error, match="overlaps") as e:
        call()
    assert e.value.code == sq.ERR_INVALID_ARG and all(n in str(e.value) for n in names), str(e.value)


def test_refusals():
    """(Every one of these runs nothing: the buffers keep their values.)"""
    M, N, K = 64, 64, 64
    b = lambda *s, dtype=BF: torch.full(s, 3, dtype=dtype, device=DEV)                            # noqa: E731
    u8 = torch.uint8
    x, y, z, v, w = b(M, K), b(M, K), b(M, K), b(K, dtype=F32), b(M, dtype=F32)
    long = b(2 * M, K)                       # overlapping, but not in place
    sq.fp8_device_status(True)
    ln = lambda **kw: sq.fp8_layernorm_fwd(**{**dict(x=x, gamma=v, beta=None, eps=1e-5, y=y), **kw})  # noqa: E731
    _refused(lambda: ln(y=x), "y", "x")
    _refused(lambda: ln(mu=w, rstd=w), "mu_out", "rstd_out")
    _refused(lambda: ln(residual=z, sum_out=y), "sum_out", "y")
    _refused(lambda: ln(x=long[:M], residual=z, sum_out=long[1:M + 1]), "sum_out", "x")
    _refused(lambda: ln(residual=z, sum_out=b(M, K), y=z), "y", "residual")
    ws = torch.full((sq.fp8_layernorm_bwd_workspace_bytes(M, K),), 3, dtype=u8, device=DEV)
    lb = lambda **kw: sq.fp8_layernorm_bwd(**{**dict(dy=y, x=x, gamma=v, mu=w, rstd=w, dx=z, dgamma=b(K, dtype=F32), dbeta=b(K, dtype=F32), workspace=ws), **kw})  # noqa: E731,E501
    _refused(lambda: lb(dx=y), "dx", "dy")
    _refused(lambda: lb(dres=z), "dx", "dres")
    _refused(lambda: lb(dgamma=v), "dgamma", "gamma")
    A, B, one = b(M, K, dtype=u8), b(N, K, dtype=u8), torch.ones(1, device=DEV)
    D = b(M, N)
    ga = lambda **kw: sq.fp8_gemm_act(A, 0, one, B, 0, one, NONE, **{**dict(D=D), **kw})          # noqa: E731
    _refused(lambda: ga(D=None, q_out=A, q_state=new_state(H, 1.0), history_len=H), "q_out", "A")
    _refused(lambda: ga(z_out=D), "z_out", "D")
    _refused(lambda: ga(D=long[:M], residual=long[1:M + 1]), "D", "residual")
    both = b(2 * M, N)
    _refused(lambda: ga(D=both[:M], residual=both.view(-1).view(F32).view(M, N)), "D", "residual")    # another type
    W = b(2 * N, K, dtype=u8)
    _refused(lambda: sq.fp8_glu_fwd(A, 0, one, W, 0, one, SILU, h_out=W.view(-1).view(BF)[:M * N].view(M, N)), "h_out", "W")
    gu = b(M, 2 * N)
    _refused(lambda: sq.fp8_glu_bwd(A, 1, one, B.view(K, N), 0, one, gu, SILU, gu.view(-1).view(u8)[:2 * M * N].view(M, 2 * N),
                                    1, new_state(H, 1.0), H), "q_dgu", "gu")
    _refused(lambda: sq.fp8_act_bwd(x, y, GELU, dz=x), "dz_out", "dy")
    torch.cuda.synchronize()
    for t in (x, y, z, v, w, long, A, B, D, W, gu, ws, both):
        assert bool((t.float() == 3).all())
