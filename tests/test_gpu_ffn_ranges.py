"""The feed-forward operators over random sizes, over more than 2^31 elements, and on two streams at once."""
import random

import pytest
import torch

import scaled_quantize_gemm_gb300 as sq
from _ffn_ref import ACTS, ELEM, GELU, NONE, SILU, U, act64, assert_within, gen, new_state, randn, to_codes, values
from test_gpu_ffn import BF, F32, H, _act_case, _empty, _glu_bwd_case, _glu_case, _workspace

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _log_size(rng, lo, hi, mult=1):
    return mult * int(round((lo / mult) * (hi / lo) ** rng.random())) or mult


@pytest.mark.parametrize("seed", range(12))
def test_random_sizes(seed):
    rng = random.Random(seed)
    M, K = _log_size(rng, 1, 1200), _log_size(rng, 16, 4096, 16)
    N, act = _log_size(rng, 16, 4096, 16), rng.choice(ACTS)
    _act_case(M, N, K, act, seed, bias=rng.random() < 0.5, res=rng.choice([None, BF, F32]), out=rng.choice([BF, F32]))
    _act_case(M, N, K, act, seed, out=None, z=True, q=rng.choice([sq.E4M3, sq.E5M2]))
    _glu_case(M, N, K, act, seed, h=rng.random() < 0.5, gu=rng.random() < 0.5)
    _glu_bwd_case(M, N, K, act, seed)


# ---------------------------------------------------------------- buffers on 16-byte boundaries only
def _shifted(t):
    """a copy of t that starts 16 bytes past a 256-byte boundary"""
    n = 16 // t.element_size()
    flat = torch.empty(t.numel() + n, dtype=t.dtype, device=t.device)
    out = flat[n:].view(t.shape)
    out.copy_(t)
    assert out.data_ptr() % 32 == 16
    return out


@pytest.mark.parametrize("M", [5, 64, 203])
def test_buffers_on_16_byte_boundaries_give_the_same(M):
    N, K = 272, 528
    g = gen(M)
    A, sa = to_codes(randn(g, M, K), 0)
    B, sb = to_codes(randn(g, 2 * N, K), 0)
    Wd, swd = to_codes(randn(g, K, N), 0)
    bias, gamma, beta = randn(g, N), randn(g, N), randn(g, N)
    x, dy, gu = randn(g, M, N).to(BF), randn(g, M, N).to(BF), randn(g, M, 2 * N).to(BF)
    res32 = randn(g, M, N)
    outs = []
    for f in (lambda t: t, _shifted):
        e = lambda *s, dtype=BF: f(torch.zeros(s, dtype=dtype, device=DEV))                      # noqa: E731
        st = [new_state(H, 3.0) for _ in range(4)]
        a, b, w = f(A), f(B), f(Wd)
        D, Z, Q, D32 = e(M, N), e(M, N), e(M, N, dtype=torch.uint8), e(M, N, dtype=F32)
        sq.fp8_gemm_act(a, 0, sa, b[:N].contiguous() if f is not _shifted else _shifted(B[:N]), 0, sb, SILU, D=D,
                        bias=f(bias), residual=f(x), z_out=Z, q_out=Q, q_state=st[0], history_len=H)
        sq.fp8_gemm_act(a, 0, sa, f(B[:N].contiguous()), 0, sb, GELU, D=D32, residual=f(res32))
        G, Hh, Qh = e(M, 2 * N), e(M, N), e(M, N, dtype=torch.uint8)
        sq.fp8_glu_fwd(a, 0, sa, b, 0, sb, SILU, gu_out=G, h_out=Hh, q_out=Qh, q_state=st[1], history_len=H)
        dq = e(M, 2 * N, dtype=torch.uint8)
        sq.fp8_glu_bwd(a, 0, sa, w, 0, swd, f(gu), SILU, dq, sq.E5M2, st[2], H)
        y, mu, rstd, s = e(M, N), torch.empty(M, device=DEV), torch.empty(M, device=DEV), e(M, N)
        sq.fp8_layernorm_fwd(f(x), f(gamma), f(beta), 1e-5, y, mu=mu, rstd=rstd, residual=f(dy), sum_out=s)
        dx, dg, db = e(M, N), torch.empty(N, device=DEV), torch.empty(N, device=DEV)
        ws = torch.empty(sq.fp8_layernorm_bwd_workspace_bytes(M, N), dtype=torch.uint8, device=DEV)
        sq.fp8_layernorm_bwd(f(dy), s, f(gamma), mu, rstd, dx, dg, db, ws, dres=f(x))
        dz, qz, dbias = e(M, N), e(M, N, dtype=torch.uint8), torch.empty(N, device=DEV)
        wb = torch.empty(sq.fp8_act_bwd_workspace_bytes(M, N), dtype=torch.uint8, device=DEV)
        sq.fp8_act_bwd(f(dy), f(x), GELU, dbias=dbias, dz=dz, q_out=qz, q_state=st[3], history_len=H, workspace=wb)
        torch.cuda.synchronize()
        outs.append([D, Z, Q, D32, G, Hh, Qh, dq, y, mu, rstd, s, dx, dg, db, dz, qz, dbias, *st])
    assert all(torch.equal(p, q) for p, q in zip(*outs))


# ---------------------------------------------------------------- more than 2^31 elements
ROWS = 160000                     # x 14336 columns: 2.29e9


def test_product_over_2_31_outputs():
    N, K, tail = 14336, 16, 300
    g = gen(1)
    A, sa = to_codes(randn(g, ROWS, K), 0)
    B, sb = to_codes(randn(g, N, K), 0)
    D, Q = torch.empty((ROWS, N), dtype=BF, device=DEV), torch.empty((ROWS, N), dtype=torch.uint8, device=DEV)
    st = new_state(H, 10.0)
    sq.fp8_gemm_act(A, 0, sa, B, 0, sb, SILU, D=D, q_out=Q, q_state=st, history_len=H)
    torch.cuda.synchronize()
    for rows in (slice(0, tail), slice(ROWS - tail, ROWS)):
        z = values(A[rows].contiguous(), 0) @ values(B, 0).T * (float(sa) * float(sb))
        y = act64(z, SILU)[0]
        assert_within(D[rows], y, ELEM * (1 + z.abs()) + 64 * U * z.abs(), "D")
        d = D[rows].float()
        near = (d * 10).clamp(-448, 448)
        got = Q[rows].contiguous().view(torch.float8_e4m3fn).float()
        # a code of the fp32 value whose bf16 rounding is d: half a step of each
        assert bool(((got - near).abs() <= 2.0 ** -4 * near.abs() + 2.0 ** -7 * near.abs() + 2.0 ** -9).all())


def test_gated_product_over_2_31_outputs():
    F, K, M, tail = 7168, 16, ROWS, 200
    g = gen(2)
    A, sa = to_codes(randn(g, M, K), 0)
    W, sw = to_codes(randn(g, 2 * F, K), 0)
    gu, h = torch.empty((M, 2 * F), dtype=BF, device=DEV), torch.empty((M, F), dtype=BF, device=DEV)
    sq.fp8_glu_fwd(A, 0, sa, W, 0, sw, SILU, h_out=h, gu_out=gu)
    dq, st = torch.empty((M, 2 * F), dtype=torch.uint8, device=DEV), new_state(H, 1.0)
    Wd, swd = to_codes(randn(g, K, F), 0)
    sq.fp8_glu_bwd(A, 0, sa, Wd, 0, swd, gu, NONE, dq, sq.E4M3, st, H)
    torch.cuda.synchronize()
    rows = slice(M - tail, M)
    z = values(A[rows].contiguous(), 0) @ values(W, 0).T * (float(sa) * float(sw))
    assert_within(gu[rows], z, 64 * U * z.abs() + 64 * U * (values(A[rows].contiguous(), 0).abs() @ values(W, 0).abs().T) * (float(sa) * float(sw)), "gu")
    want = act64(z[:, :F], SILU)[0] * z[:, F:]
    assert_within(h[rows], want, 2.0 ** -17 * (1 + z[:, :F].abs()) * (1 + z[:, F:].abs()), "h")
    dh = values(A[rows].contiguous(), 0) @ values(Wd, 0) * (float(sa) * float(swd))
    t = gu[rows].double()
    ref = torch.cat([dh * t[:, F:], dh * t[:, :F]], 1).clamp(-448, 448)
    got = dq[rows].contiguous().view(torch.float8_e4m3fn).double()
    assert bool(((got - ref).abs() <= 2.0 ** -4 * ref.abs() + 2.0 ** -9 + 2.0 ** -12).all())


def test_row_operators_over_2_31_elements():
    M, K, tail = 540000, 4096, 64
    g = gen(3)
    x = torch.empty((M, K), dtype=BF, device=DEV).normal_(generator=g)
    gamma, beta = randn(g, K) * 0.2 + 1, randn(g, K)
    y, mu, rstd = torch.empty_like(x), torch.empty(M, device=DEV), torch.empty(M, device=DEV)
    sq.fp8_layernorm_fwd(x, gamma, beta, 1e-5, y, mu=mu, rstd=rstd)
    dx, dg, db = torch.empty_like(x), torch.empty(K, device=DEV), torch.empty(K, device=DEV)
    ws = torch.empty(sq.fp8_layernorm_bwd_workspace_bytes(M, K), dtype=torch.uint8, device=DEV)
    sq.fp8_layernorm_bwd(y, x, gamma, mu, rstd, dx, dg, db, ws)
    torch.cuda.synchronize()
    rows = slice(M - tail, M)
    xs = x[rows].double()
    m = xs.mean(1, keepdim=True)
    r = ((xs - m).square().mean(1, keepdim=True) + 1e-5).rsqrt()
    xh = (xs - m) * r
    assert_within(y[rows], xh * gamma + beta, 2.0 ** -18 * (1 + xh.abs()) * (1 + beta.abs()), "y")
    w = y[rows].double() * gamma
    want = r * (w - w.mean(1, keepdim=True) - xh * (w * xh).mean(1, keepdim=True))
    assert_within(dx[rows], want, 2.0 ** -17 * r * (1 + w.abs() + xh.abs()), "dx")
    del dx, xs
    # dbeta: the column sums of y, in pieces
    s = sum(y[i:i + 60000].double().sum(0) for i in range(0, M, 60000))
    a = sum(y[i:i + 60000].double().abs().sum(0) for i in range(0, M, 60000))
    assert bool(((db.double() - s).abs() <= (M / 64 + 128) * U * a).all())
    q, st = torch.empty((M, K), dtype=torch.uint8, device=DEV), new_state(H, 50.0)
    dz = torch.empty_like(x)
    sq.fp8_act_bwd(y, x, GELU, dz=dz, q_out=q, q_format=sq.E4M3, q_state=st, history_len=H)
    torch.cuda.synchronize()
    d = y[rows].double() * act64(x[rows].double(), GELU)[1]
    assert_within(dz[rows], d, ELEM * y[rows].double().abs() * (1 + x[rows].double().abs()), "dz")


# ---------------------------------------------------------------- two streams
def test_two_streams_with_their_own_workspaces():
    M, N, K = 8, 2064, 4096
    g = gen(5)
    B, sb = to_codes(randn(g, N, K), 0)
    jobs = []
    for _ in range(2):
        A, sa = to_codes(randn(g, M, K), 0)
        jobs.append((A, sa, _workspace(sq.fp8_gemm_act_workspace_bytes(M, N, K)), _empty(M, N, dtype=F32), torch.cuda.Stream()))
    want = []
    for A, sa, ws, D, _ in jobs:
        sq.fp8_gemm_act(A, 0, sa, B, 0, sb, SILU, D=D, workspace=ws)
        torch.cuda.synchronize()
        want.append(D.clone())
    for _ in range(20):
        for A, sa, ws, D, s in jobs:
            sq.fp8_gemm_act(A, 0, sa, B, 0, sb, SILU, D=D, workspace=ws, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(j[3], w) for j, w in zip(jobs, want))
    assert sq.fp8_device_status(True) == sq.OK
