"""fp8_layernorm_fwd and fp8_layernorm_bwd against the definitions in 64 bits.

Bounds (u = 2^-24): a row sum of K fp32 terms is a tree over at least 32
strands, so its error is at most c = (K / 32 + 16) u of the sum of magnitudes.
mean: c mean|s|.  The variance then has a relative error of at most
2 c + 4 u |mean| / std and some units, rstd half of it, and y follows by the
product rule.  dgamma and dbeta add M terms over at least 64 strands:
(M / 64 + 128) u of the sum of magnitudes.
"""
import pytest
import torch

import scaled_quantize_gemm_gb300 as sq
from _ffn_ref import U, assert_amax, assert_codes, assert_within, gen, new_state, randn

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-5
DTYPES = [torch.bfloat16, torch.float32]
SIZES = [(1, 1), (1, 4096), (3, 7), (5, 16), (17, 1000), (33, 1535), (2, 8192), (64, 12288), (7, 16384), (3, 20000),
         (1500, 264), (700, 2048), (9, 12000), (4, 65552), (400, 1862), (130, 1004), (6, 9998), (20, 4094)]


def _fwd64(s, gamma, beta):
    mu = s.mean(1)
    var = (s - mu[:, None]).square().mean(1)
    rstd = (var + EPS).rsqrt()
    y = (s - mu[:, None]) * rstd[:, None] * gamma + (0 if beta is None else beta)
    return mu, rstd, y


def _check_fwd(s, gamma, beta, y, mu, rstd):
    s, gamma = s.double(), gamma.double()
    beta = None if beta is None else beta.double()
    K = s.shape[1]
    m64, r64, y64 = _fwd64(s, gamma, beta)
    c = (K / 32 + 16) * U
    e_mu = c * s.abs().mean(1) + U * m64.abs()
    # relative error of rstd: half the variance's, whose terms carry the
    # mean's error twice (2 |d| e + e^2) and their own rounding
    e_r = 0.5 * (2 * c + 8 * U + (2 * e_mu * r64 + (e_mu * r64) ** 2)) + 8 * U
    assert_within(mu, m64, e_mu, "mu")
    assert_within(rstd, r64, e_r * r64, "rstd")
    d = (s - m64[:, None]).abs()
    e_y = gamma.abs() * r64[:, None] * (e_mu[:, None] + 2 * U * d + d * e_r[:, None]) + 8 * U * (
        gamma.abs() * d * r64[:, None] + (0 if beta is None else beta.abs()))
    assert_within(y, y64, e_y, "y")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K", SIZES)
def test_forward(M, K, dtype):
    g = gen(M * 131 + K)
    x = (randn(g, M, K) * 2 + randn(g, M, 1)).to(dtype)
    gamma, beta = randn(g, K) * 0.2 + 1, randn(g, K) * 0.1
    for res, b in ((None, beta), (randn(g, M, K).to(dtype), None)):
        y = torch.full((M, K), 7.0, device=DEV, dtype=dtype)
        mu, rstd = torch.full((M,), 7.0, device=DEV), torch.full((M,), 7.0, device=DEV)
        total = torch.full((M, K), 7.0, device=DEV, dtype=dtype) if res is not None else None
        sq.fp8_layernorm_fwd(x, gamma, b, EPS, y, mu=mu, rstd=rstd, residual=res, sum_out=total)
        s = x
        if res is not None:
            s = (x.float() + res.float()).to(dtype)
            assert torch.equal(total, s)
        _check_fwd(s, gamma, b, y, mu, rstd)
        # without the statistics the outputs are the same
        y2 = torch.empty_like(y)
        sq.fp8_layernorm_fwd(x, gamma, b, EPS, y2, residual=res, sum_out=total)
        assert torch.equal(y, y2)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt,m", [(sq.E4M3, 60.0), (sq.E5M2, 5000.0)])
@pytest.mark.parametrize("M,K", [(1, 4096), (3, 7), (17, 1002), (33, 1535), (300, 264), (5, 12288), (2, 20000)])
def test_forward_codes(M, K, fmt, m, dtype):
    """The codes of y, with and without y itself, and the newest amax."""
    g = gen(M * 139 + K)
    x = (randn(g, M, K) * 2 + randn(g, M, 1)).to(dtype)
    gamma, beta = randn(g, K) * 0.2 + 1, randn(g, K) * 0.1
    m64, r64, y64 = _fwd64(x.double(), gamma.double(), beta.double())
    c = (K / 32 + 16) * U
    e_mu = c * x.double().abs().mean(1) + U * m64.abs()
    e_r = 0.5 * (2 * c + 8 * U + (2 * e_mu * r64 + (e_mu * r64) ** 2)) + 8 * U
    d = (x.double() - m64[:, None]).abs()
    e = gamma.double().abs() * r64[:, None] * (e_mu[:, None] + 2 * U * d + d * e_r[:, None]) + 8 * U * (
        gamma.double().abs() * d * r64[:, None] + beta.double().abs())
    y, mu, rstd = torch.empty_like(x), torch.empty(M, device=DEV), torch.empty(M, device=DEV)
    seen = []
    for out in (y, None):
        q, st = torch.full((M, K), 0x55, dtype=torch.uint8, device=DEV), new_state(16, m, 0.5)
        sq.fp8_layernorm_fwd(x, gamma, beta, EPS, out, mu=mu, rstd=rstd, q_out=q, q_format=fmt, q_state=st, history_len=16)
        assert_codes(q, y64, e, m, fmt, "codes")
        assert_amax(st, 0.5, y64, e, "amax")
        seen.append(q)
    assert torch.equal(*seen)
    _check_fwd(x, gamma, beta, y, mu, rstd)


def _bwd64(dy, x, gamma, mu, rstd, dres):
    dy, x, gamma, mu, rstd = (t.double() for t in (dy, x, gamma, mu, rstd))
    xh = (x - mu[:, None]) * rstd[:, None]
    w = dy * gamma
    c1, c2 = w.mean(1, keepdim=True), (w * xh).mean(1, keepdim=True)
    dx = rstd[:, None] * (w - c1 - xh * c2)
    if dres is not None:
        dx = dx + dres.double()
    return dx, (dy * xh).sum(0), dy.sum(0), xh, w


def _run_bwd(dy, x, gamma, mu, rstd, dres=None):
    M, K = x.shape
    dx = torch.full_like(x, 7.0)
    dg, db = torch.full((K,), 7.0, device=DEV), torch.full((K,), 7.0, device=DEV)
    ws = torch.full((max(1, sq.fp8_layernorm_bwd_workspace_bytes(M, K)),), 0xFF, dtype=torch.uint8, device=DEV)
    sq.fp8_layernorm_bwd(dy, x, gamma, mu, rstd, dx, dg, db, ws, dres=dres)
    return dx, dg, db


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K", SIZES)
def test_backward(M, K, dtype):
    g = gen(M * 137 + K)
    x = (randn(g, M, K) * 2 + randn(g, M, 1)).to(dtype)
    dy = (randn(g, M, K) * 1e-2).to(dtype)
    gamma = randn(g, K) * 0.2 + 1
    mu64, r64, _ = _fwd64(x.double(), gamma.double(), None)
    mu, rstd = mu64.float(), r64.float()
    for dres in (None, (randn(g, M, K) * 1e-2).to(dtype)):
        dx, dg, db = _run_bwd(dy, x, gamma, mu, rstd, dres)
        dx64, dg64, db64, xh, w = _bwd64(dy, x, gamma, mu, rstd, dres)
        c = (K / 32 + 16) * U
        r = rstd.double()[:, None]
        aw, ah = w.abs(), xh.abs()
        # xh is formed from x - mu and rstd, two roundings; its mean with w is c2
        e = r * ((c + 4 * U) * aw.mean(1, keepdim=True) + ah * (c + 8 * U) * (aw * ah).mean(1, keepdim=True) +
                 8 * U * aw) + (0 if dres is None else 2 * U * dres.double().abs())
        assert_within(dx, dx64, e, "dx")
        depth = (M / 64 + 128) * U
        ad = dy.double().abs()
        assert_within(dg, dg64, (depth + 4 * U) * (ad * ah).sum(0), "dgamma")
        assert_within(db, db64, depth * ad.sum(0), "dbeta")
        # a fixed order of sums: the same bits again
        again = _run_bwd(dy, x, gamma, mu, rstd, dres)
        assert all(torch.equal(a, b) for a, b in zip((dx, dg, db), again))


def test_backward_against_differences():
    """The gradients along random directions against central differences of the 64-bit forward."""
    M, K = 6, 264
    g = gen(3)
    x, dy = randn(g, M, K), randn(g, M, K)
    gamma, beta = randn(g, K) * 0.2 + 1, randn(g, K)
    y, mu, rstd = torch.empty_like(x), torch.empty(M, device=DEV), torch.empty(M, device=DEV)
    sq.fp8_layernorm_fwd(x, gamma, beta, EPS, y, mu=mu, rstd=rstd)
    dx, dg, db = _run_bwd(dy, x, gamma, mu, rstd)
    h = 1e-5
    loss = lambda a, b, c: float((_fwd64(a, b, c)[2] * dy.double()).sum())                       # noqa: E731
    base = [x.double(), gamma.double(), beta.double()]
    for i, grad in enumerate((dx, dg, db)):
        v = randn(g, *base[i].shape).double()
        up, down = list(base), list(base)
        up[i], down[i] = base[i] + h * v, base[i] - h * v
        want = (loss(*up) - loss(*down)) / (2 * h)
        # differences: h^2 of the third derivative and 2^-53 / h of the loss; the
        # gradient: fp32 sums over K or M terms of magnitude |grad v|
        tol = 1e-6 * float((grad.double() * v).abs().sum()) + 1e-6
        assert abs(float((grad.double() * v).sum()) - want) <= tol


def test_backward_takes_the_fused_casts_statistics():
    M, K, H = 48, 528, 16
    g = gen(9)
    x = (randn(g, M, K) + 0.5).to(torch.bfloat16)
    gamma, beta = randn(g, K) * 0.2 + 1, randn(g, K)
    st = torch.zeros(H + 2, device=DEV)
    st[H:] = 1.0
    q = torch.empty((M, K), dtype=torch.uint8, device=DEV)
    mu, rstd = torch.empty(M, device=DEV), torch.empty(M, device=DEV)
    sq.fp8_layernorm_quantize(x, gamma, beta, EPS, sq.E4M3, q, None, mu, rstd, st, H)
    dy = randn(g, M, K).to(torch.bfloat16)
    dx, dg, db = _run_bwd(dy, x, gamma, mu, rstd)
    y, mu2, rstd2 = torch.empty_like(x), torch.empty_like(mu), torch.empty_like(mu)
    sq.fp8_layernorm_fwd(x, gamma, beta, EPS, y, mu=mu2, rstd=rstd2)
    _check_fwd(x, gamma, beta, y, mu, rstd)
    dx64, dg64, db64, xh, w = _bwd64(dy, x, gamma, mu, rstd, None)
    c = (K / 32 + 32) * U
    e = rstd.double()[:, None] * (c * w.abs().mean(1, keepdim=True) + xh.abs() * c * (w * xh).abs().mean(1, keepdim=True) + 8 * U * w.abs())
    assert_within(dx, dx64, e, "dx")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("K", [7, 4096, 20000])
def test_constant_rows_and_non_finite_rows(K, dtype):
    """A constant row normalises to beta (its variance is 0); a row with a NaN or an infinity becomes NaN, alone."""
    M = 6
    g = gen(K)
    x = randn(g, M, K).to(dtype)
    x[1] = 3.0
    x[3, K // 2] = float("nan")
    x[4, 0] = float("inf")
    gamma, beta = randn(g, K), randn(g, K)
    y, mu, rstd = torch.empty_like(x), torch.empty(M, device=DEV), torch.empty(M, device=DEV)
    sq.fp8_layernorm_fwd(x, gamma, beta, EPS, y, mu=mu, rstd=rstd)
    assert torch.equal(y[1], beta.to(dtype))
    assert abs(float(rstd[1]) - EPS ** -0.5) <= 4 * U * EPS ** -0.5
    assert bool(torch.isnan(y[3]).all()) and bool(torch.isnan(y[4]).all())
    rows = [0, 2, 5]
    _check_fwd(x[rows], gamma, beta, y[rows], mu[rows], rstd[rows])


@pytest.mark.parametrize("dtype", DTYPES)
def test_no_rows(dtype):
    K = 40
    gamma = torch.ones(K, device=DEV)
    x = torch.empty((0, K), device=DEV, dtype=dtype)
    sq.fp8_layernorm_fwd(x, gamma, None, EPS, torch.empty_like(x))
    mu = torch.empty(0, device=DEV)
    dx, dg, db = _run_bwd(x, x, gamma, mu, mu)
    assert bool((dg == 0).all()) and bool((db == 0).all())


def test_other_stream_and_graph():
    """On a stream of its own, and captured into a graph and replayed on new inputs."""
    M, K = 300, 1000
    g = gen(5)
    x, dy = randn(g, M, K).to(torch.bfloat16), randn(g, M, K).to(torch.bfloat16)
    gamma, beta = randn(g, K), randn(g, K)
    y, mu, rstd = torch.empty_like(x), torch.empty(M, device=DEV), torch.empty(M, device=DEV)
    dx, dg, db = torch.empty_like(x), torch.empty(K, device=DEV), torch.empty(K, device=DEV)
    ws = torch.empty(sq.fp8_layernorm_bwd_workspace_bytes(M, K), dtype=torch.uint8, device=DEV)

    def step():
        sq.fp8_layernorm_fwd(x, gamma, beta, EPS, y, mu=mu, rstd=rstd)
        sq.fp8_layernorm_bwd(dy, x, gamma, mu, rstd, dx, dg, db, ws)

    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    first = [t.clone() for t in (y, dx, dg, db)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x.copy_(randn(g, M, K))
    dy.copy_(randn(g, M, K))
    graph.replay()
    torch.cuda.synchronize()
    replayed = [t.clone() for t in (y, dx, dg, db)]
    step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(replayed, (y, dx, dg, db)))
    assert not torch.equal(first[0], y)
