"""LayerNorm backward over rows that 16 bytes do not divide, which a thread
copies whole with the blocks they begin and end in: every start within a block,
rows shorter than one, arrays that end inside one, one to three stages of rows,
and several groups a CTA (bounds: test_gpu_layernorm_grad.py)."""
import pytest
import torch

import scaled_quantize_gemm_gb300 as sq
from _ffn_ref import gen, randn
from test_gpu_layernorm_grad import DEV, DTYPES, EPS
from test_gpu_layernorm_grad import test_backward as _backward


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K", [(2, 1), (7, 2), (50, 3), (1000, 5), (1, 15), (4, 6), (3001, 9), (2500, 155), (700, 501),
                                 (2000, 2045), (160, 4095), (160, 4097), (153, 5001), (155, 8191), (310, 8193),
                                 (320, 9849), (153, 9850), (160, 12289), (155, 14001), (320, 16383)])
def test_backward_rows(M, K, dtype):
    _backward(M, K, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K", [(2500, 155), (600, 9849)])
def test_backward_reads_and_writes_its_rows_only(M, K, dtype):
    """Beside an array that ends inside a 16-byte block there may be anything: the
    results do not depend on it, it is not written, and a second call gives the same bits."""
    g = gen(M + K)
    pad = 64
    big = [torch.full((M * K + pad,), float("nan"), device=DEV, dtype=dtype) for _ in range(4)]
    x, dy, dres, dx = (b[:M * K].view(M, K) for b in big)
    for t in (x, dy, dres):
        t.copy_(randn(g, M, K).to(dtype))
    big[3].fill_(7.0)
    gamma = randn(g, K) * 0.2 + 1
    mu, rstd = x.float().mean(1), (x.float().var(1, unbiased=False) + EPS).rsqrt()
    ws = torch.empty(sq.fp8_layernorm_bwd_workspace_bytes(M, K), dtype=torch.uint8, device=DEV)
    outs = []
    for X, DY, DR in ((x, dy, dres), (x.clone(), dy.clone(), dres.clone())):
        dg, db = torch.empty(K, device=DEV), torch.empty(K, device=DEV)
        sq.fp8_layernorm_bwd(DY, X, gamma, mu, rstd, dx, dg, db, dres=DR, workspace=ws)
        outs.append((dx.clone(), dg, db))
    torch.cuda.synchronize()
    for a, b in zip(*outs):
        assert not bool(a.isnan().any()) and torch.equal(a, b)
    assert bool((big[3][M * K:] == 7.0).all())


@pytest.mark.gpu
def test_backward_beside_a_set_error_word():
    """LayerNorm does not wait on other kernels: a wait of theirs that ran out changes none of its results."""
    M, K = 400, 1535
    g = gen(3)
    x, dy = randn(g, M, K), randn(g, M, K)
    gamma = randn(g, K)
    mu, rstd = x.mean(1), (x.var(1, unbiased=False) + EPS).rsqrt()
    ws = torch.empty(sq.fp8_layernorm_bwd_workspace_bytes(M, K), dtype=torch.uint8, device=DEV)
    waited = torch.zeros(1, dtype=torch.int32, device=DEV)
    assert sq.fp8_device_status(True) == sq.OK
    outs = []
    for broken in (False, True):
        if broken:
            sq.fp8_selftest_wait_timeout(1000, waited)
        dx, dg, db = torch.empty_like(x), torch.empty(K, device=DEV), torch.empty(K, device=DEV)
        sq.fp8_layernorm_bwd(dy, x, gamma, mu, rstd, dx, dg, db, workspace=ws)
        outs.append((dx, dg, db))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    assert sq.fp8_device_status(True) == sq.ERR_TIMEOUT
