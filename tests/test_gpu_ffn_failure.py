"""A wait of some other kernel that runs out while products start: every one of
them ends, whichever of its warps sees the error word first, and the next ones
are right again once the word is cleared and the workspace zeroed."""
import pytest
import torch

import scaled_quantize_gemm_gb300 as sq
from _ffn_ref import NONE, gen, to_codes, randn
from test_gpu_ffn import DEV, F32, _empty, _workspace

pytestmark = pytest.mark.gpu


# the weights' tiles over all SMs: K split through the workspace, whole tiles, tiles of
# 256 x 256, and K over a cluster
@pytest.mark.parametrize("M,N,K", [(5, 10256, 8208), (16, 14336, 1040), (2300, 2064, 1040), (64, 4096, 4096)])
def test_a_word_set_while_products_start(M, N, K):
    g = gen(M)
    A, sa = to_codes(randn(g, M, K), 0)
    B, sb = to_codes(randn(g, N, K), 0)
    ws = _workspace(sq.fp8_gemm_act_workspace_bytes(M, N, K))
    D = _empty(M, N, dtype=F32)
    call = lambda s=None: sq.fp8_gemm_act(A, 0, sa, B, 0, sb, NONE, D=D, workspace=ws, stream=s)  # noqa: E731
    assert sq.fp8_device_status(True) == sq.OK
    call()
    torch.cuda.synchronize()
    want = D.clone()
    waited = torch.zeros(1, dtype=torch.int32, device=DEV)
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(24):
        # the wait runs out at a moment of its own among the products
        sq.fp8_selftest_wait_timeout(20 + 17 * i, waited, stream=two)
        for _ in range(30):
            call(one)
        torch.cuda.synchronize()
        assert sq.fp8_device_status(True) == sq.ERR_TIMEOUT
        if ws is not None:
            ws.zero_()
        call()
        torch.cuda.synchronize()
        assert torch.equal(D, want) and sq.fp8_device_status(True) == sq.OK


@pytest.mark.parametrize("gran,M,N,K", [(sq.TENSOR, 2300, 2064, 1040), (sq.TILE_1x128, 512, 1024, 1024),
                                          (sq.MX32_TILED, 512, 1024, 1024)])
def test_a_word_set_while_linear_products_start(gran, M, N, K):
    """The linear layer's products: per-tensor scales on CTA pairs, promoted tiles, block-scaled MX."""
    A = torch.full((M, K), 0x38, dtype=torch.uint8, device=DEV)          # 1.0
    B = torch.full((N, K), 0x38, dtype=torch.uint8, device=DEV)
    gb, na, nb = gran, 1, 1
    if gran == sq.TILE_1x128:
        gb, na, nb = sq.BLOCK_128x128, M * K // 128, N * K // (128 * 128)
    sa, sb = torch.ones(na, device=DEV), torch.ones(nb, device=DEV)
    if gran == sq.MX32_TILED:                                            # E8M0 code 127: 1.0
        sa, sb = (torch.full((n * K // 32,), 127, dtype=torch.uint8, device=DEV) for n in (M, N))
    D = _empty(M, N, dtype=F32)
    call = lambda s=None: sq.fp8_gemm(A, 0, sa, gran, B, 0, sb, gb, D, stream=s)                  # noqa: E731
    assert sq.fp8_device_status(True) == sq.OK
    waited = torch.zeros(1, dtype=torch.int32, device=DEV)
    p, q = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(24):
        sq.fp8_selftest_wait_timeout(20 + 17 * i, waited, stream=q)
        for _ in range(30):
            call(p)
        torch.cuda.synchronize()
        assert sq.fp8_device_status(True) == sq.ERR_TIMEOUT
        D.fill_(7.0)
        call()
        torch.cuda.synchronize()
        assert bool((D == float(K)).all()) and sq.fp8_device_status(True) == sq.OK
