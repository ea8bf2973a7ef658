"""fp8_rmsnorm_fwd and fp8_rmsnorm_bwd against the definition in 64 bits.

u = 2^-24.  The sum of K squares: a thread adds at most n = max(16, K / 256) + 3
terms in turn and the rest is a tree of at most 10 levels, so its relative error
is at most (n + 10) u, that of rstd half of it and 3 u for the division, the root
and the reciprocal; y adds two products."""
import pytest
import torch

import scaled_quantize_gemm_gb300 as sq
from _ffn_ref import F8, FMAX, U, assert_amax, assert_codes, assert_within, gen, new_state, randn

pytestmark = pytest.mark.gpu
DEV, H, EPS = "cuda", 4, 1e-5
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
SHAPES = [(1, 1), (3, 7), (1, 128), (5, 100), (2, 4096), (700, 1535), (300, 2050), (1000, 512), (40, 12288), (33, 16384),
          (9, 16385), (5, 20032), (2100, 96), (64, 8200)]


def _seq(K):
    return max(16, K // 256) + 3 + 10


def _inputs(M, K, dtype, seed):
    g = gen(seed)
    x = randn(g, M, K) * (0.1 + 3 * torch.rand((M, 1), generator=g, device=DEV))
    return g, x.to(dtype), 0.5 + torch.rand(K, generator=g, device=DEV)


def _reference(x, gamma):
    x = x.double()
    rstd = (x.square().mean(1) + EPS) ** -0.5
    y = x * rstd[:, None] * gamma.double()
    er = (_seq(x.shape[1]) / 2 + 4) * U
    return y, rstd, (er + 3 * U) * y.abs(), er * rstd


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_forward(M, K, dtype, residual):
    g, x, gamma = _inputs(M, K, dtype, M + K)
    res = randn(g, M, K).to(dtype) if residual else None
    total = torch.full_like(x, 7.0) if residual else None
    y, rstd = torch.full_like(x, 7.0), torch.full((M,), 7.0, device=DEV)
    q, st = torch.full((M, K), 0x55, dtype=U8, device=DEV), new_state(H, 40.0, 0.25)
    sq.fp8_rmsnorm_fwd(x, gamma, EPS, y, rstd=rstd, residual=res, sum_out=total)
    sq.fp8_rmsnorm_fwd(x, gamma, EPS, None, residual=res, sum_out=total, q_out=q, q_state=st, history_len=H)
    s = x
    if residual:
        s = (x.float() + res.float()).to(dtype)
        assert torch.equal(total, s)
    want, wr, ey, er = _reference(s, gamma)
    assert_within(y, want, ey, "y")
    assert_within(rstd, wr, er, "rstd")
    assert_codes(q, want, ey, 40.0, sq.E4M3, "codes")
    assert_amax(st, 0.25, want, ey)


UNITS = [(sq.TILE_1x128, 128, 1), (sq.TILE_1x128_POW2, 128, 128), (sq.MX32, 32, 1), (sq.MX32_TILED, 128, 128),
         (sq.MX32_FLOOR_TILED, 128, 128)]


@pytest.mark.parametrize("fmt", [sq.E4M3, sq.E5M2])
@pytest.mark.parametrize("gran,kmul,mmul", UNITS)
@pytest.mark.parametrize("M,K", [(1, 128), (77, 384), (256, 4096), (128, 16384), (128, 16512), (384, 640)])
def test_codes_with_scales(M, K, gran, kmul, mmul, fmt):
    """In fp32 y is what the codes are cast from, so they and their scales are those of fp8_quantize, bit for bit;
    rows of zeros, infinities and NaN among them."""
    M = -(-M // mmul) * mmul
    _, x, gamma = _inputs(M, K, F32, M + K)
    x[M // 2] = 0.0
    if M > 4:
        x[1, 5], x[2, K - 1], x[3] = float("inf"), float("nan"), 1e-30
    y = torch.empty_like(x)
    f32 = gran == sq.TILE_1x128
    new = lambda: (torch.full((M, K), 0x55, dtype=U8, device=DEV),                                # noqa: E731
                   torch.full((M * K // 128,), 7.0, device=DEV) if f32 else torch.full((M * K // 32,), 0x33, dtype=U8, device=DEV))
    (q, s), (q2, s2), (q3, s3) = new(), new(), new()
    sq.fp8_rmsnorm_fwd(x, gamma, EPS, y, q_out=q, q_format=fmt, gran=gran, scales_out=s)
    sq.fp8_rmsnorm_fwd(x, gamma, EPS, None, q_out=q2, q_format=fmt, gran=gran, scales_out=s2)
    sq.fp8_quantize(y, fmt, gran, q3, scales_out=s3)
    torch.cuda.synchronize()
    assert torch.equal(q, q3) and torch.equal(s, s3)
    assert torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.parametrize("M,K", [(3, 32), (50, 96), (7, 16416)])
def test_mx_rows_of_odd_numbers_of_blocks(M, K):
    _, x, gamma = _inputs(M, K, F32, K)
    y, q, q2 = torch.empty_like(x), torch.empty((M, K), dtype=U8, device=DEV), torch.empty((M, K), dtype=U8, device=DEV)
    s, s2 = (torch.full((M * K // 32,), 0x33, dtype=U8, device=DEV) for _ in range(2))
    sq.fp8_rmsnorm_fwd(x, gamma, EPS, y, q_out=q, gran=sq.MX32, scales_out=s)
    sq.fp8_quantize(y, sq.E4M3, sq.MX32, q2, scales_out=s2)
    assert torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.parametrize("M,K", [(1, 256), (300, 4096), (17, 17024)])
def test_bf16_tiles(M, K):
    g, x, gamma = _inputs(M, K, BF, 3)
    res = randn(g, M, K).to(BF)
    total, q, s = torch.empty_like(x), torch.empty((M, K), dtype=U8, device=DEV), torch.empty((M, K // 128), device=DEV)
    sq.fp8_rmsnorm_fwd(x, gamma, EPS, None, residual=res, sum_out=total, q_out=q, gran=sq.TILE_1x128, scales_out=s)
    want, _, ey, _ = _reference(total, gamma)
    tiles, et = want.view(M, -1, 128), ey.view(M, -1, 128)
    a = tiles.abs().amax(2)
    assert_within(s, a / 448, et.amax(2) / 448 + U * a / 448, "scales")
    # the multiplier from the stored step: one more rounding each
    v = q.view(F8[0]).double().view(M, -1, 128) * s.double()[..., None]
    step = torch.maximum(tiles.abs() * 2.0 ** -4, s.double()[..., None] * 2.0 ** -10)          # half a step of e4m3
    assert bool(((v - tiles).abs() <= step * (1 + 2.0 ** -10) + et + 4 * U * a[..., None]).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,K", SHAPES + [(4000, 768), (1, 4096), (5001, 64)])
@pytest.mark.parametrize("dres", [False, True])
def test_backward(M, K, dtype, dres):
    g, x, gamma = _inputs(M, K, dtype, 2 * M + K)
    dy = randn(g, M, K).to(dtype)
    dr = randn(g, M, K).to(dtype) if dres else None
    rstd = (x.double().square().mean(1) + EPS).rsqrt().float()
    dx, dg = torch.full_like(x, 7.0), torch.full((K,), 7.0, device=DEV)
    ws = torch.full((sq.fp8_rmsnorm_bwd_workspace_bytes(M, K),), 0x7F, dtype=U8, device=DEV)
    sq.fp8_rmsnorm_bwd(dy, x, gamma, rstd, dx, dg, ws, dres=dr)
    again = torch.empty_like(dx), torch.empty_like(dg)
    sq.fp8_rmsnorm_bwd(dy, x, gamma, rstd, *again, ws, dres=dr)
    r = rstd.double()[:, None]
    xh, d = x.double() * r, dy.double()
    w = d * gamma.double()
    c = (w * xh).mean(1, keepdim=True)
    want = r * (w - xh * c)
    ec = (_seq(K) + 4) * U * (w * xh).abs().mean(1, keepdim=True)
    bound = r * (6 * U * (w.abs() + (xh * c).abs()) + xh.abs() * ec) + 2 * U * want.abs()
    if dres:
        want = want + dr.double()
        bound = bound + U * (want.abs() + dr.double().abs())
    assert_within(dx, want, bound, "dx")
    assert_within(dg, (d * xh).sum(0), (M + 4) * U * (d * xh).abs().sum(0), "dgamma")
    assert torch.equal(dx, again[0]) and torch.equal(dg, again[1])


def test_gradient_against_differences():
    """The formula's gradient is that of the formula's value: central differences of sum(c y) in 64 bits."""
    M, K = 3, 40
    g, x, gamma = _inputs(M, K, F32, 5)
    c = randn(g, M, K)
    dx, dg, rstd, y = torch.empty_like(x), torch.empty_like(gamma), torch.empty(M, device=DEV), torch.empty_like(x)
    sq.fp8_rmsnorm_fwd(x, gamma, EPS, y, rstd=rstd)
    ws = torch.empty(sq.fp8_rmsnorm_bwd_workspace_bytes(M, K), dtype=U8, device=DEV)
    sq.fp8_rmsnorm_bwd(c, x, gamma, rstd, dx, dg, ws)
    f = lambda x_, g_: float((c.double() * _reference(x_, g_)[0]).sum())                          # noqa: E731
    h = 1e-5                                    # the third derivative's share: h^2, below 1e-8 of the terms here
    for i in range(0, M * K, 7):
        e = torch.zeros(M * K, dtype=torch.float64, device=DEV)
        e[i] = h
        e = e.view(M, K)
        d = (f(x.double() + e, gamma) - f(x.double() - e, gamma)) / (2 * h)
        assert abs(d - float(dx.reshape(-1)[i])) <= 1e-5 * float(dx.abs().max())
    for i in range(0, K, 7):
        e = torch.zeros(K, dtype=torch.float64, device=DEV)
        e[i] = h
        d = (f(x, gamma.double() + e) - f(x, gamma.double() - e)) / (2 * h)
        assert abs(d - float(dg[i])) <= 1e-5 * float(dg.abs().max())


def test_no_rows():
    x, gamma = torch.empty((0, 64), device=DEV), torch.ones(64, device=DEV)
    sq.fp8_rmsnorm_fwd(x, gamma, EPS, torch.empty_like(x))
    dg = torch.full((64,), 7.0, device=DEV)
    sq.fp8_rmsnorm_bwd(x, x, gamma, torch.empty(0, device=DEV), torch.empty_like(x), dg, torch.empty(16, dtype=U8, device=DEV))
    torch.cuda.synchronize()
    assert not bool(dg.any())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,K", [(1000, 4096), (700, 1535), (40, 20001)])
@pytest.mark.parametrize("over", ["residual", "x"])
def test_sum_in_place(M, K, dtype, over):
    g, x, gamma = _inputs(M, K, dtype, 1)
    res, outs = randn(g, M, K).to(dtype), []
    for in_place in (False, True):
        a, b, y, rstd = x.clone(), res.clone(), torch.empty_like(x), torch.empty(M, device=DEV)
        s = (b if over == "residual" else a) if in_place else torch.empty_like(x)
        sq.fp8_rmsnorm_fwd(a, gamma, EPS, y, rstd=rstd, residual=b, sum_out=s)
        outs.append((y, rstd, s))
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(*outs))


def test_refusals():
    x, v = torch.zeros((128, 256), device=DEV), torch.ones(256, device=DEV)
    q, s = torch.zeros((128, 256), dtype=U8, device=DEV), torch.zeros(256, device=DEV)
    with pytest.raises(sq.Fp8Error, match="y overlaps x"):
        sq.fp8_rmsnorm_fwd(x, v, EPS, x)
    with pytest.raises(sq.Fp8Error, match="scales_out overlaps gamma"):
        sq.fp8_rmsnorm_fwd(x, v, EPS, None, q_out=q, gran=sq.TILE_1x128, scales_out=v)
    with pytest.raises(sq.Fp8Error, match="unit of a row"):
        sq.fp8_rmsnorm_fwd(x, v, EPS, None, q_out=q, gran=sq.BLOCK_128x128, scales_out=s.view(U8))
    with pytest.raises(sq.Fp8Error, match="dx overlaps dy"):
        sq.fp8_rmsnorm_bwd(x, torch.zeros_like(x), v, torch.zeros(128, device=DEV), x, s,
                           torch.zeros(sq.fp8_rmsnorm_bwd_workspace_bytes(128, 256), dtype=U8, device=DEV))
