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
