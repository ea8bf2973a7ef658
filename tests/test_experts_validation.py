"""Refusals of RMSNorm and of the experts' operators, on the host before anything
runs: the C entry points with pointers that are never read, and the binding."""
import ctypes

import pytest
import torch

import scaled_quantize_gemm_gb300 as sq
from scaled_quantize_gemm_gb300 import build as sqbuild

P, c = ctypes.c_void_p, ctypes
F = P(4096)              # aligned, never dereferenced
bf16, f32, u8, i32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


@pytest.fixture(scope="module")
def L():
    sqbuild.build()
    return sq.lib()


def _refuses(call, invalid=(), unsupported=(), misaligned=()):
    for code, cases in ((sq.ERR_INVALID_ARG, invalid), (sq.ERR_UNSUPPORTED, unsupported), (sq.ERR_MISALIGNED, misaligned)):
        for bad in cases:
            assert call(**bad) == code, bad


def test_rmsnorm_fwd(L):
    def call(x=F, res=None, dtype=0, gamma=F, eps=1e-5, M=4, K=10, total=None, y=F, rstd=F, q=None, qf=0, gran=0, st=None,
             H=0, sc=None):
        return L.fp8_rmsnorm_fwd(x, res, dtype, gamma, c.c_float(eps), M, K, total, y, rstd, q, qf, gran, st, H, sc, None)

    tile = dict(q=F, K=256, M=128, sc=F)
    _refuses(call,
             invalid=[dict(x=None), dict(gamma=None), dict(y=None), dict(dtype=2), dict(M=-1), dict(K=-1), dict(res=F), dict(total=F),
                      dict(eps=-1.0), dict(eps=float("nan")), dict(q=F), dict(q=F, st=F, H=0), dict(q=F, st=F, H=4, qf=5),
                      dict(tile, gran=1, sc=None), dict(tile, gran=3, qf=2)],
             unsupported=[dict(K=0), dict(M=1 << 31), dict(tile, gran=2), dict(tile, gran=5), dict(tile, gran=6), dict(tile, gran=8),
                          dict(tile, gran=10), dict(tile, gran=1, K=192), dict(tile, gran=3, K=48), dict(tile, gran=4, M=64),
                          dict(tile, gran=7, M=127), dict(tile, gran=9, K=160)],
             misaligned=[dict(x=P(4104)), dict(gamma=P(4100)), dict(y=P(4098)), dict(rstd=P(4098)), dict(res=P(4104), total=F),
                         dict(tile, gran=1, sc=P(4098)), dict(tile, gran=4, sc=P(4104)), dict(tile, gran=3, q=P(4104))])


def test_rmsnorm_bwd(L):
    need = sq.fp8_rmsnorm_bwd_workspace_bytes(100, 48)
    assert need >= 48 * 4 and sq.fp8_rmsnorm_bwd_workspace_bytes(0, 48) == 0

    def call(dy=F, x=F, dres=None, dtype=1, gamma=F, rstd=F, M=100, K=48, dx=F, dg=F, ws=F, n=need):
        return L.fp8_rmsnorm_bwd(dy, x, dres, dtype, gamma, rstd, M, K, dx, dg, ws, n, None)

    _refuses(call,
             invalid=[dict(dy=None), dict(x=None), dict(gamma=None), dict(rstd=None), dict(dx=None), dict(dg=None), dict(ws=None),
                      dict(n=need - 1), dict(dtype=-1), dict(M=-5)],
             unsupported=[dict(K=0), dict(K=1 << 31)],
             misaligned=[dict(dy=P(4104)), dict(dres=P(4104)), dict(dg=P(4097)), dict(ws=P(4104))])


ROUTING_BAD = dict(invalid=[dict(T=-1), dict(k=0), dict(E=0), dict(plan=None)],
                   unsupported=[dict(k=65), dict(E=1025), dict(T=1 << 31), dict(T=1 << 30)], misaligned=[dict(plan=P(4100))])


def _with(base, **more):
    return {kind: base.get(kind, []) + more.get(kind, []) for kind in ("invalid", "unsupported", "misaligned")}


def test_sizes(L):
    assert sq.fp8_expert_rows(1, 1, 1) == 32 and sq.fp8_expert_rows(0, 4, 4) == 0
    assert sq.fp8_expert_rows(64, 8, 64) == 512 + 31 * 64
    assert sq.fp8_expert_rows(1, 8, 64) == 8 + 31 * 8
    for bad in ((-1, 1, 1), (1, 0, 1), (1, 1, 0), (1, 65, 1), (1, 1, 1025)):
        assert sq.fp8_expert_rows(*bad) == 0 and sq.fp8_expert_plan_ints(*bad) == 0
    assert sq.fp8_expert_workspace_bytes(0, 1, 1, 64, 64) == 0 and sq.fp8_expert_workspace_bytes(1, 0, 1, 64, 64) == 0


def test_rows(L):
    def plan(ids=F, T=4, k=2, E=3, plan=F):
        return L.fp8_expert_plan(ids, T, k, E, plan, None)

    _refuses(plan, **_with(ROUTING_BAD, invalid=[dict(ids=None)], misaligned=[dict(ids=P(4098))]))

    def dispatch(x=F, size=1, K=16, plan=F, T=4, k=2, E=3, out=F):
        return L.fp8_expert_dispatch(x, size, K, plan, T, k, E, out, None)

    _refuses(dispatch, **_with(ROUTING_BAD, invalid=[dict(x=None), dict(out=None), dict(size=3), dict(K=-1)],
                               unsupported=[dict(K=1 << 30)], misaligned=[dict(x=P(4104)), dict(out=P(4104))]))

    def combine(rows=F, dtype=0, K=16, w=F, res=None, plan=F, T=4, k=2, E=3, y=F):
        return L.fp8_expert_combine(rows, dtype, K, w, res, plan, T, k, E, y, None)

    _refuses(combine, **_with(ROUTING_BAD, invalid=[dict(rows=None), dict(y=None), dict(dtype=2), dict(K=-1)],
                              unsupported=[dict(K=1 << 30)],
                              misaligned=[dict(rows=P(4104)), dict(y=P(4104)), dict(res=P(4104)), dict(w=P(4098))]))

    def bwd(dy=F, dtype=0, K=16, rows=F, w=F, plan=F, T=4, k=2, E=3, dw=F, drows=None, q=None, qf=1, st=None, H=0):
        return L.fp8_expert_combine_bwd(dy, dtype, K, rows, w, plan, T, k, E, dw, drows, q, qf, st, H, None)

    _refuses(bwd, **_with(ROUTING_BAD, invalid=[dict(dy=None), dict(w=None), dict(rows=None), dict(dw=None), dict(q=F), dict(dtype=7),
                                                dict(q=F, st=F, H=4, qf=2)],
                          misaligned=[dict(dy=P(4104)), dict(rows=P(4104)), dict(drows=P(4104)), dict(dw=P(4098)),
                                      dict(q=P(4104), st=F, H=4)]))


def test_products(L):
    def gemm(A=F, fa=0, sa=F, B=F, fb=0, sb=F, major=0, plan=F, T=4, k=2, E=3, N=32, K=64, D=F, dt=0, ws=None, n=0):
        return L.fp8_expert_gemm(A, fa, sa, B, fb, sb, major, plan, T, k, E, N, K, D, dt, ws, n, None)

    _refuses(gemm, **_with(ROUTING_BAD, invalid=[dict(A=None), dict(B=None), dict(sa=None), dict(sb=None), dict(fa=2), dict(major=2),
                                                 dict(D=None), dict(dt=2), dict(N=-16)],
                           unsupported=[dict(K=0), dict(K=24), dict(N=40), dict(major=1, K=48), dict(N=1 << 30), dict(E=1024, N=1 << 21)],
                           misaligned=[dict(A=P(4104)), dict(B=P(4104)), dict(D=P(4104)), dict(sb=P(4098)), dict(ws=P(4112), n=1 << 30)]))

    def glu(A=F, fa=0, sa=F, W=F, fw=0, sw=F, plan=F, T=4, k=2, E=3, N=32, K=64, act=4, gu=None, h=F, q=None, qf=0, st=None, H=0,
            ws=None, n=0):
        return L.fp8_expert_glu_fwd(A, fa, sa, W, fw, sw, plan, T, k, E, N, K, act, gu, h, q, qf, st, H, ws, n, None)

    _refuses(glu, **_with(ROUTING_BAD, invalid=[dict(A=None), dict(W=None), dict(h=None), dict(h=None, gu=F), dict(act=5), dict(q=F)],
                          unsupported=[dict(N=24), dict(K=8), dict(E=1024, N=1 << 20)],
                          misaligned=[dict(gu=P(4104)), dict(h=P(4104)), dict(q=P(4104), st=F, H=4)]))

    def bwd(dY=F, fd=1, sd=F, Wd=F, fw=0, sw=F, plan=F, T=4, k=2, E=3, N=32, K=64, gu=F, act=4, q=F, qf=1, st=F, H=4):
        return L.fp8_expert_glu_bwd(dY, fd, sd, Wd, fw, sw, plan, T, k, E, N, K, gu, act, q, qf, st, H, None)

    _refuses(bwd, **_with(ROUTING_BAD, invalid=[dict(dY=None), dict(Wd=None), dict(gu=None), dict(q=None), dict(st=None), dict(H=0)],
                          unsupported=[dict(N=8), dict(K=48)], misaligned=[dict(gu=P(4104)), dict(q=P(4104))]))

    def wgrad(A=F, fa=1, sa=F, B=F, fb=0, sb=F, plan=F, T=4, k=2, E=3, M=32, N=48, D=F, dt=1):
        return L.fp8_expert_wgrad(A, fa, sa, B, fb, sb, plan, T, k, E, M, N, D, dt, None)

    _refuses(wgrad, **_with(ROUTING_BAD, invalid=[dict(A=None), dict(B=None), dict(sa=None), dict(D=None), dict(fb=3), dict(M=-32)],
                            unsupported=[dict(M=48), dict(N=40), dict(E=1024, M=1 << 21)],
                            misaligned=[dict(A=P(4104)), dict(D=P(4104)), dict(sa=P(4098))]))


def test_workspaces_that_are_too_small_are_refused(L):
    for T, k, E, N, K in ((1, 8, 64, 4096, 1792), (1, 1, 1, 512, 4096), (64, 8, 64, 512, 512), (10000, 2, 4, 256, 256)):
        need = sq.fp8_expert_workspace_bytes(T, k, E, N, K)
        if need:
            assert L.fp8_expert_gemm(F, 0, F, F, 0, F, 0, F, T, k, E, N, K, F, 0, F, need - 1, None) == sq.ERR_INVALID_ARG
            assert L.fp8_expert_glu_fwd(F, 0, F, F, 0, F, F, T, k, E, N // 2, K, 0, None, F, None, 0, None, 0, F, need - 1,
                                        None) == sq.ERR_INVALID_ARG


def test_no_gpu_is_an_error(L):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert L.fp8_rmsnorm_fwd(F, None, 0, F, c.c_float(1e-5), 4, 16, None, F, F, None, 0, 0, None, 0, None, None) == sq.ERR_CUDA
    assert L.fp8_expert_plan(F, 4, 2, 3, F, None) == sq.ERR_CUDA
    assert L.fp8_expert_wgrad(F, 1, F, F, 0, F, F, 4, 2, 3, 32, 48, F, 1, None) == sq.ERR_CUDA


def test_binding_checks_shapes_and_types():
    z = lambda *s, dtype=f32: torch.zeros(s, dtype=dtype)                                        # noqa: E731
    x, g = z(4, 256, dtype=bf16), z(256)
    with pytest.raises(ValueError, match="y is required"):
        sq.fp8_rmsnorm_fwd(x, g, 1e-5, None)
    with pytest.raises(ValueError, match="residual and sum_out"):
        sq.fp8_rmsnorm_fwd(x, g, 1e-5, x, residual=x)
    with pytest.raises(TypeError, match="scales_out"):
        sq.fp8_rmsnorm_fwd(x, g, 1e-5, None, q_out=z(4, 256, dtype=u8), gran=sq.TILE_1x128, scales_out=z(8, dtype=u8))
    with pytest.raises(ValueError, match="scales_out"):
        sq.fp8_rmsnorm_fwd(x, g, 1e-5, None, q_out=z(4, 256, dtype=u8), gran=sq.TILE_1x128, scales_out=z(7))
    with pytest.raises(ValueError, match="q_state"):
        sq.fp8_rmsnorm_fwd(x, g, 1e-5, None, q_out=z(4, 256, dtype=u8), q_state=z(5), history_len=4)
    with pytest.raises(ValueError, match="rstd"):
        sq.fp8_rmsnorm_bwd(x, x, g, z(3), z(4, 256, dtype=bf16), g, z(1, dtype=u8))
    T, k, E = 4, 2, 3
    plan, R = z(sq.fp8_expert_plan_ints(T, k, E), dtype=i32), sq.fp8_expert_rows(T, k, E)
    one, codes, w = z(3), z(R, 32, dtype=u8), z(E, 16, 32, dtype=u8)
    with pytest.raises(TypeError, match="ids"):
        sq.fp8_expert_plan(z(T, k, dtype=torch.int64), E, plan)
    with pytest.raises(ValueError, match="plan"):
        sq.fp8_expert_plan(z(T, k, dtype=i32), E, plan[:-1])
    with pytest.raises(ValueError, match="rows"):
        sq.fp8_expert_dispatch(z(T, 32, dtype=u8), plan, k, E, codes[1:])
    with pytest.raises(TypeError, match="rows"):
        sq.fp8_expert_dispatch(z(T, 32), plan, k, E, codes)
    with pytest.raises(ValueError, match="weights"):
        sq.fp8_expert_combine(z(R, 32), plan, k, E, z(T, 32), weights=z(T, 3))
    with pytest.raises(ValueError, match="dweights"):
        sq.fp8_expert_combine_bwd(z(T, 32), plan, k, E, z(T, k), rows=z(R, 32), dweights=z(T, 1))
    with pytest.raises(ValueError, match="q_state"):
        sq.fp8_expert_combine_bwd(z(T, 32), plan, k, E, z(T, k), q_out=codes, q_state=z(5), history_len=4)
    with pytest.raises(ValueError, match="B"):
        sq.fp8_expert_gemm(codes, 0, one, w[0], 0, one, sq.K_MAJOR, plan, T, k, z(R, 16))
    with pytest.raises(ValueError, match="A"):
        sq.fp8_expert_gemm(codes, 0, one, w, 0, one, sq.MN_MAJOR, plan, T, k, z(R, 32))
    with pytest.raises(ValueError, match="b_scales"):
        sq.fp8_expert_gemm(codes, 0, one, w, 0, z(2), sq.K_MAJOR, plan, T, k, z(R, 16))
    with pytest.raises(ValueError, match="even"):
        sq.fp8_expert_glu_fwd(codes, 0, one, z(E, 15, 32, dtype=u8), 0, one, 4, plan, T, k, h_out=z(R, 7, dtype=bf16))
    with pytest.raises(ValueError, match="gu_out"):
        sq.fp8_expert_glu_fwd(codes, 0, one, w, 0, one, 4, plan, T, k, h_out=z(R, 8, dtype=bf16), gu_out=z(R, 8, dtype=bf16))
    with pytest.raises(ValueError, match="q_dgu"):
        sq.fp8_expert_glu_bwd(codes, 1, one, z(E, 32, 16, dtype=u8), 0, one, z(R, 32, dtype=bf16), 4, plan, T, k, None, 1, z(6), 4)
    with pytest.raises(ValueError, match="D"):
        sq.fp8_expert_wgrad(codes, 1, one, codes, 0, one, plan, T, k, z(32, 32))
