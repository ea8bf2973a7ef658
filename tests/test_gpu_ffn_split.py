"""Products of few rows whose K is split, over a cluster's shared memory or over
the whole grid, against the definitions in 64 bits (bounds: _ffn_ref.py)."""
import pytest
import torch

import scaled_quantize_gemm_gb300 as sq
from _ffn_ref import GELU, GELU_TANH, NONE, RELU, SILU, gen, randn, to_codes
from test_gpu_ffn import BF, DEV, F32, _act_case, _empty, _glu_case, _workspace

pytestmark = pytest.mark.gpu

# tiles of 16, 32, 64, 128 and 256 tokens; K of an odd number of blocks, ending
# inside one, of as few blocks as CTAs; a last tile of one token or one column
ACT = [(1, 4096, 4096), (1, 16, 256), (3, 1040, 6000), (13, 2064, 1040), (31, 1552, 1936), (33, 16, 1024), (64, 4096, 1040),
       (65, 4096, 2064), (129, 144, 4112), (200, 4096, 4096), (193, 1040, 6000), (250, 4096, 14336), (257, 2064, 1040),
       (500, 1040, 8208), (1, 4096, 14336), (5, 10256, 1040), (40, 10256, 656)]


@pytest.mark.parametrize("M,N,K", ACT)
def test_gemm_act_split(M, N, K):
    _act_case(M, N, K, NONE, 301, bias=False, res=BF)
    _act_case(M, N, K, SILU, 302, res=F32, out=F32)
    _act_case(M, N, K, GELU, 303, out=None, z=True, q=sq.E4M3)


@pytest.mark.parametrize("M,F,K", [(1, 4096, 4096), (1, 16, 256), (7, 2064, 1040), (30, 1040, 2064), (64, 1040, 4112),
                                   (65, 2064, 1040), (128, 4096, 4096), (250, 528, 6000), (5, 6160, 1040)])
def test_glu_fwd_split(M, F, K):
    _glu_case(M, F, K, SILU, 311)
    _glu_case(M, F, K, GELU_TANH, 312, gu=False, q=None)
    _glu_case(M, F, K, RELU, 313, h=False, q=sq.E5M2)


@pytest.mark.parametrize("fa,fb", [(0, 1), (1, 0), (1, 1)])
def test_split_formats(fa, fb):
    _act_case(20, 528, 1296, SILU, 321, fa=fa, fb=fb, res=BF, q=sq.E5M2)
    _glu_case(20, 528, 1296, SILU, 322, fa=fa, fw=fb)


@pytest.mark.parametrize("M,N,K", [(1, 4096, 14336), (64, 4096, 4096), (200, 4096, 4096), (5, 10256, 1040)])
def test_split_gives_the_same_bits(M, N, K):
    """Whatever the order in which the shares end, and with or beside another product on the same stream."""
    g = gen(M + N)
    A, sa = to_codes(randn(g, M, K), 0)
    B, sb = to_codes(randn(g, N, K), 0)
    ws = _workspace(sq.fp8_gemm_act_workspace_bytes(M, N, K))
    outs = [_empty(M, N, dtype=F32) for _ in range(24)]
    for i, D in enumerate(outs):
        sq.fp8_gemm_act(A, 0, sa, B, 0, sb, SILU, D=D, workspace=ws)
        if i % 3 == 0:
            sq.fp8_gemm_act(A[:1], 0, sa, B[:256], 0, sb, SILU, D=_empty(1, 256, dtype=F32))
    torch.cuda.synchronize()
    assert all(torch.equal(outs[0], D) for D in outs[1:])
    assert sq.fp8_device_status(True) == sq.OK


def test_split_in_a_graph_and_on_another_stream():
    M, N, K = 24, 2064, 2064
    g = gen(5)
    A, sa = to_codes(randn(g, M, K), 0)
    B, sb = to_codes(randn(g, N, K), 0)
    D, E = _empty(M, N, dtype=BF), _empty(M, N, dtype=BF)
    sq.fp8_gemm_act(A, 0, sa, B, 0, sb, SILU, D=D)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            sq.fp8_gemm_act(A, 0, sa, B, 0, sb, SILU, D=E)
        graph.replay()
    s.synchronize()
    assert torch.equal(D, E)


def test_split_skips_while_the_error_word_is_set():
    M, N, K = 2, 64, 1024
    A = torch.full((M, K), 0x38, dtype=torch.uint8, device=DEV)
    B = torch.full((N, K), 0x38, dtype=torch.uint8, device=DEV)
    one = torch.ones(1, device=DEV)
    D = _empty(M, N, dtype=F32)
    waited = torch.zeros(1, dtype=torch.int32, device=DEV)
    assert sq.fp8_device_status(True) == sq.OK
    sq.fp8_selftest_wait_timeout(1000, waited)
    sq.fp8_gemm_act(A, 0, one, B, 0, one, NONE, D=D)
    torch.cuda.synchronize()
    assert bool((D == 7.0).all())
    assert sq.fp8_device_status(True) == sq.ERR_TIMEOUT
    sq.fp8_gemm_act(A, 0, one, B, 0, one, NONE, D=D)
    torch.cuda.synchronize()
    assert bool((D == 1024.0).all())
