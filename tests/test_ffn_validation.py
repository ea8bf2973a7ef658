"""Refusals of the feed-forward operators, on the host before anything runs:
the C entry points with pointers that are never read, and the binding."""
import ctypes

import pytest
import torch

import scaled_quantize_gemm_gb300 as sq
from scaled_quantize_gemm_gb300 import build as sqbuild

P, c = ctypes.c_void_p, ctypes
F = P(4096)              # aligned, never dereferenced
bf16, f32, u8 = torch.bfloat16, torch.float32, torch.uint8


@pytest.fixture(scope="module")
def L():
    sqbuild.build()
    return sq.lib()


def test_layernorm_fwd(L):
    def call(x=F, res=None, dtype=0, gamma=F, beta=F, eps=1e-5, M=4, K=10, total=None, y=F, mu=F, rstd=F, q=None, qf=0,
             st=None, H=0):
        return L.fp8_layernorm_fwd(x, res, dtype, gamma, beta, c.c_float(eps), M, K, total, y, mu, rstd, q, qf, st, H, None)

    for bad in (dict(x=None), dict(gamma=None), dict(y=None), dict(dtype=2), dict(M=-1), dict(K=-1), dict(res=F),
                dict(total=F), dict(eps=-1.0), dict(eps=float("nan")), dict(q=F), dict(q=F, st=F, H=0),
                dict(q=F, st=F, H=4, qf=5)):
        assert call(**bad) == sq.ERR_INVALID_ARG, bad
    for bad in (dict(x=P(4104)), dict(gamma=P(4100)), dict(beta=P(4100)), dict(y=P(4098)), dict(mu=P(4098)),
                dict(res=P(4104), total=F)):
        assert call(**bad) == sq.ERR_MISALIGNED, bad
    assert call(K=0) == sq.ERR_UNSUPPORTED
    assert call(M=1 << 31) == sq.ERR_UNSUPPORTED


def test_layernorm_bwd(L):
    need = sq.fp8_layernorm_bwd_workspace_bytes(100, 48)
    assert need >= 2 * 48 * 4 and sq.fp8_layernorm_bwd_workspace_bytes(0, 48) == 0

    def call(dy=F, x=F, dres=None, dtype=1, gamma=F, mu=F, rstd=F, M=100, K=48, dx=F, dg=F, db=F, ws=F, n=need):
        return L.fp8_layernorm_bwd(dy, x, dres, dtype, gamma, mu, rstd, M, K, dx, dg, db, ws, n, None)

    for bad in (dict(dy=None), dict(x=None), dict(gamma=None), dict(mu=None), dict(rstd=None), dict(dx=None),
                dict(dg=None), dict(db=None), dict(ws=None), dict(n=need - 1), dict(dtype=-1), dict(M=-5)):
        assert call(**bad) == sq.ERR_INVALID_ARG, bad
    for bad in (dict(dy=P(4104)), dict(dres=P(4104)), dict(dg=P(4097)), dict(ws=P(4104))):
        assert call(**bad) == sq.ERR_MISALIGNED, bad
    assert call(K=0) == sq.ERR_UNSUPPORTED


def test_gemm_act(L):
    def call(A=F, fa=0, sa=F, B=F, fb=0, sb=F, M=4, N=32, K=64, act=0, bias=None, res=None, rdt=0, z=None, D=F, ddt=0,
             q=None, qf=0, st=None, H=0, ws=None, n=0):
        return L.fp8_gemm_act(A, fa, sa, B, fb, sb, M, N, K, act, bias, res, rdt, z, D, ddt, q, qf, st, H, ws, n, None)

    for bad in (dict(A=None), dict(B=None), dict(sa=None), dict(sb=None), dict(fa=2), dict(fb=-1), dict(act=5),
                dict(act=-1), dict(M=-1), dict(D=None), dict(ddt=3), dict(rdt=2), dict(q=F), dict(q=F, st=F, H=0),
                dict(q=F, st=F, H=5000), dict(q=F, st=F, H=4, qf=2)):
        assert call(**bad) == sq.ERR_INVALID_ARG, bad
    for bad in (dict(K=0), dict(K=24), dict(N=20), dict(N=24, q=F, st=F, H=4), dict(M=1 << 31)):
        assert call(**bad) == sq.ERR_UNSUPPORTED, bad
    for bad in (dict(A=P(4104)), dict(B=P(4104)), dict(D=P(4104)), dict(z=P(4104)), dict(bias=P(4100)),
                dict(res=P(4104)), dict(sa=P(4098)), dict(q=P(4104), st=F, H=4), dict(ws=P(4096 + 16), n=1 << 30)):
        assert call(**bad) == sq.ERR_MISALIGNED, bad


def test_few_rows_workspace(L):
    """A workspace that is too small is refused, whatever the size says."""
    for M, N, K in ((1, 4096, 4096), (40, 1040, 2064), (10000, 256, 256)):
        need = sq.fp8_gemm_act_workspace_bytes(M, N, K)
        if need:
            r = L.fp8_gemm_act(F, 0, F, F, 0, F, M, N, K, 0, None, None, 0, None, F, 0, None, 0, None, 0, F, need - 1, None)
            assert r == sq.ERR_INVALID_ARG
        need = sq.fp8_glu_fwd_workspace_bytes(M, N, K)
        if need:
            r = L.fp8_glu_fwd(F, 0, F, F, 0, F, M, N, K, 0, None, F, None, 0, None, 0, F, need - 1, None)
            assert r == sq.ERR_INVALID_ARG
    assert sq.fp8_gemm_act_workspace_bytes(0, 16, 16) == 0
    assert sq.fp8_gemm_act_workspace_bytes(-1, 16, 16) == 0
    assert sq.fp8_gemm_act_workspace_bytes(100000, 4096, 4096) == 0


def test_glu(L):
    def fwd(A=F, fa=0, sa=F, W=F, fw=0, sw=F, M=4, N=32, K=64, act=4, gu=None, h=F, q=None, qf=0, st=None, H=0, ws=None,
            n=0):
        return L.fp8_glu_fwd(A, fa, sa, W, fw, sw, M, N, K, act, gu, h, q, qf, st, H, ws, n, None)

    for bad in (dict(A=None), dict(W=None), dict(sa=None), dict(fw=7), dict(act=9), dict(h=None), dict(h=None, gu=F),
                dict(q=F), dict(q=F, st=F)):
        assert fwd(**bad) == sq.ERR_INVALID_ARG, bad
    for bad in (dict(K=0), dict(K=8), dict(N=24), dict(N=1 << 30)):
        assert fwd(**bad) == sq.ERR_UNSUPPORTED, bad
    for bad in (dict(h=P(4104)), dict(gu=P(4104)), dict(W=P(4104)), dict(ws=P(4104), n=1 << 30)):
        assert fwd(**bad) == sq.ERR_MISALIGNED, bad

    def bwd(dY=F, fd=1, sd=F, Wd=F, fw=0, sw=F, M=4, N=32, K=64, gu=F, act=4, q=F, qf=1, st=F, H=4):
        return L.fp8_glu_bwd(dY, fd, sd, Wd, fw, sw, M, N, K, gu, act, q, qf, st, H, None)

    for bad in (dict(dY=None), dict(Wd=None), dict(gu=None), dict(q=None), dict(st=None), dict(H=0), dict(qf=3)):
        assert bwd(**bad) == sq.ERR_INVALID_ARG, bad
    for bad in (dict(N=8), dict(K=0), dict(K=40)):
        assert bwd(**bad) == sq.ERR_UNSUPPORTED, bad
    for bad in (dict(gu=P(4104)), dict(q=P(4104)), dict(st=P(4098))):
        assert bwd(**bad) == sq.ERR_MISALIGNED, bad


def test_act_bwd(L):
    need = sq.fp8_act_bwd_workspace_bytes(50, 33)

    def call(dy=F, z=F, M=50, N=33, act=1, db=F, dz=None, q=None, qf=1, st=None, H=0, ws=F, n=need):
        return L.fp8_act_bwd(dy, z, M, N, act, db, dz, q, qf, st, H, ws, n, None)

    for bad in (dict(dy=None), dict(z=None), dict(act=5), dict(M=-1), dict(db=None), dict(ws=None), dict(n=need - 1),
                dict(q=F), dict(q=F, st=F, H=0)):
        assert call(**bad) == sq.ERR_INVALID_ARG, bad
    for bad in (dict(dy=P(4104)), dict(dz=P(4104)), dict(db=P(4098)), dict(ws=P(4104))):
        assert call(**bad) == sq.ERR_MISALIGNED, bad


def test_no_gpu_is_an_error(L):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert L.fp8_layernorm_fwd(F, None, 0, F, F, c.c_float(1e-5), 4, 16, None, F, F, F, None, 0, None, 0, None) == sq.ERR_CUDA
    assert L.fp8_glu_bwd(F, 1, F, F, 0, F, 4, 32, 64, F, 4, F, 1, F, 4, None) == sq.ERR_CUDA


def test_binding_checks_shapes_and_types():
    z = lambda *s, dtype=f32: torch.zeros(s, dtype=dtype)                                        # noqa: E731
    x, g = z(4, 10, dtype=bf16), z(10)
    with pytest.raises(TypeError, match="y"):
        sq.fp8_layernorm_fwd(x, g, None, 1e-5, z(4, 10))
    with pytest.raises(ValueError, match="y"):
        sq.fp8_layernorm_fwd(x, g, None, 1e-5, z(4, 9, dtype=bf16))
    with pytest.raises(ValueError, match="gamma"):
        sq.fp8_layernorm_fwd(x, z(9), None, 1e-5, z(4, 10, dtype=bf16))
    with pytest.raises(ValueError, match="contiguous"):
        sq.fp8_layernorm_fwd(z(10, 4, dtype=bf16).t(), g, None, 1e-5, z(4, 10, dtype=bf16))
    with pytest.raises(ValueError, match="residual"):
        sq.fp8_layernorm_fwd(x, g, None, 1e-5, z(4, 10, dtype=bf16), residual=x)
    with pytest.raises(ValueError, match="y is required"):
        sq.fp8_layernorm_fwd(x, g, None, 1e-5, None)
    with pytest.raises(ValueError, match="q_state"):
        sq.fp8_layernorm_fwd(x, g, None, 1e-5, None, q_out=z(4, 10, dtype=u8), q_state=z(5), history_len=4)
    with pytest.raises(ValueError, match="rstd"):
        sq.fp8_layernorm_bwd(x, x, g, z(4), z(3), z(4, 10, dtype=bf16), g, g, z(1, dtype=u8))
    A, B, one = z(4, 32, dtype=u8), z(16, 32, dtype=u8), z(1)
    with pytest.raises(ValueError, match="D"):
        sq.fp8_gemm_act(A, 0, one, B, 0, one, 0, D=z(4, 15))
    with pytest.raises(TypeError, match="A"):
        sq.fp8_gemm_act(A.float(), 0, one, B, 0, one, 0, D=z(4, 16))
    with pytest.raises(ValueError, match="B"):
        sq.fp8_gemm_act(A, 0, one, z(16, 48, dtype=u8), 0, one, 0, D=z(4, 16))
    with pytest.raises(ValueError, match="q_state"):
        sq.fp8_gemm_act(A, 0, one, B, 0, one, 0, q_out=z(4, 16, dtype=u8), q_state=z(5), history_len=4)
    with pytest.raises(TypeError, match="z_out"):
        sq.fp8_gemm_act(A, 0, one, B, 0, one, 0, D=z(4, 16), z_out=z(4, 16))
    with pytest.raises(ValueError, match="W"):
        sq.fp8_glu_fwd(A, 0, one, z(33, 32, dtype=u8), 0, one, 4, h_out=z(4, 16, dtype=bf16))
    with pytest.raises(ValueError, match="gu"):
        sq.fp8_glu_bwd(A, 1, one, z(32, 16, dtype=u8), 0, one, z(4, 16, dtype=bf16), 4, z(4, 32, dtype=u8), 1, z(6), 4)
    with pytest.raises(ValueError, match="q_dgu"):
        sq.fp8_glu_bwd(A, 1, one, z(32, 16, dtype=u8), 0, one, z(4, 32, dtype=bf16), 4, z(4, 16, dtype=u8), 1, z(6), 4)
    with pytest.raises(ValueError, match="dy"):
        sq.fp8_act_bwd(z(4, 9, dtype=bf16), z(4, 10, dtype=bf16), 1, dz=z(4, 10, dtype=bf16))
