"""Each of the products' kernels by name: the 256 x 256 tiles over everything their epilogue does, and the split over
the workspace, which sizes alone do not show to be the one that ran (bounds: _ffn_ref.py)."""
import pytest
import torch

import scaled_quantize_gemm_gb300 as sq
from _ffn_kernels import COUNTERS, KSPLIT, PAIR, ROWS, expected, launched
from _ffn_ref import ACTS, GELU, GELU_TANH, NONE, RELU, SILU, gen, randn, to_codes
from test_gpu_ffn import BF, F32, _act_case, _empty, _glu_bwd_case, _glu_case, _workspace

pytestmark = pytest.mark.gpu

# more tiles than pairs, so that both accumulators and the ring go round; a last tile of few rows and of 8, 64 or
# 24 columns; K of whole blocks and ending inside one
TILES = [(2300, 2072, 2064), (2000, 5440, 1616), (2561, 5656, 1536)]


@pytest.mark.parametrize("M,N,K", TILES)
@pytest.mark.parametrize("act", ACTS)
def test_tiles_gemm_act(M, N, K, act):
    with expected(PAIR, "fp8_gemm_act"):
        _act_case(M, N, K, act, 401, bias=True, res=F32, out=F32, z=True)
        _act_case(M, N, K, act, 402, bias=False, res=BF, out=BF)
        if N % 16 == 0:
            _act_case(M, N, K, act, 403, bias=True, out=None, z=True, q=sq.E4M3)
            _act_case(M, N, K, act, 404, bias=False, res=F32, out=F32, z=True, q=sq.E5M2)


@pytest.mark.parametrize("M,N,K", TILES)
def test_tiles_every_combination_of_outputs(M, N, K):
    cases = [(bias, res, out, z, q) for bias in (False, True) for res in (None, BF, F32) for out in (None, BF, F32)
             for z in (False, True) for q in (None, sq.E4M3) if (out or z or q is not None) and not (q is not None and N % 16)]
    with expected(PAIR, "fp8_gemm_act") as seen:
        for i, (bias, res, out, z, q) in enumerate(cases):
            if i % 3 == M % 3 or (z and q is not None):
                _act_case(M, N, K, GELU, 410 + i, bias=bias, res=res, out=out, z=z, q=q)
    assert len(seen) >= 10


@pytest.mark.parametrize("fa,fb", [(0, 1), (1, 0), (1, 1)])
def test_tiles_formats(fa, fb):
    with expected(PAIR, "fp8_gemm_act"):
        _act_case(2000, 5440, 1616, SILU, 421, fa=fa, fb=fb, res=BF, q=sq.E5M2)
    with expected(PAIR, "fp8_glu_fwd"):
        _glu_case(1100, 5440, 1040, SILU, 422, fa=fa, fw=fb, q=sq.E5M2)


@pytest.mark.parametrize("M,F,K", [(2003, 2064, 1040), (1100, 5440, 2064), (700, 5200, 1536)])
@pytest.mark.parametrize("act", ACTS)
def test_tiles_glu_fwd(M, F, K, act):
    with expected(PAIR, "fp8_glu_fwd"):
        _glu_case(M, F, K, act, 431)
        _glu_case(M, F, K, act, 432, h=False, gu=False)
        _glu_case(M, F, K, act, 433, h=True, gu=True, q=None)


@pytest.mark.parametrize("M,F,K", [(2003, 2064, 1040), (1100, 5440, 2064)])
@pytest.mark.parametrize("act", ACTS)
def test_tiles_glu_bwd(M, F, K, act):
    with expected(PAIR, "fp8_glu_bwd"):
        _glu_bwd_case(M, F, K, act, 441)


def test_tiles_give_the_same_bits():
    M, N, K = 2300, 5440, 2064
    g = gen(9)
    A, sa = to_codes(randn(g, M, K), 0)
    B, sb = to_codes(randn(g, N, K), 0)
    R, bias = randn(g, M, N), randn(g, N)
    outs = [(_empty(M, N, dtype=F32), _empty(M, N, dtype=BF)) for _ in range(8)]
    with expected(PAIR, "fp8_gemm_act"):
        for D, Z in outs:
            sq.fp8_gemm_act(A, 0, sa, B, 0, sb, GELU_TANH, D=D, bias=bias, residual=R, z_out=Z)
    torch.cuda.synchronize()
    assert all(torch.equal(D, outs[0][0]) and torch.equal(Z, outs[0][1]) for D, Z in outs[1:])


def test_tiles_skip_while_the_error_word_is_set():
    M, N, K = 2300, 2064, 1040
    A = torch.full((M, K), 0x38, dtype=torch.uint8, device="cuda")
    B = torch.full((N, K), 0x38, dtype=torch.uint8, device="cuda")
    one = torch.ones(1, device="cuda")
    D = _empty(M, N, dtype=F32)
    waited = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = lambda: sq.fp8_gemm_act(A, 0, one, B, 0, one, NONE, D=D)                               # noqa: E731
    assert launched(call) == {PAIR} and sq.fp8_device_status(True) == sq.OK
    sq.fp8_selftest_wait_timeout(1000, waited)
    call()
    torch.cuda.synchronize()
    assert bool((D == 7.0).all()) and sq.fp8_device_status(True) == sq.ERR_TIMEOUT
    call()
    torch.cuda.synchronize()
    assert bool((D == float(K)).all())


# ---------------------------------------------------------------- K split through the workspace
# tiles of 16, 32 and 64 tokens, one to many partial blocks a tile, two and three token tiles
SPLIT_ACT = [(1, 10256, 8208), (5, 10256, 8208), (17, 10256, 8208), (40, 10256, 8208), (64, 10256, 8208), (1, 4096, 14336),
             (73, 16, 22560), (139, 16, 22960), (98, 128, 22640)]
SPLIT_GLU = [(1, 14336, 4096), (5, 5200, 4112), (17, 5200, 4112), (33, 10256, 4112), (64, 14336, 4096), (80, 16, 22768),
             (158, 32, 22608)]


@pytest.mark.parametrize("M,N,K", SPLIT_ACT)
def test_split_gemm_act(M, N, K):
    with expected(ROWS, "fp8_gemm_act", split=True):
        _act_case(M, N, K, SILU, 501, res=F32, out=F32)
        _act_case(M, N, K, NONE, 502, bias=False, res=BF)
        _act_case(M, N, K, GELU, 503, out=None, z=True, q=sq.E4M3)


@pytest.mark.parametrize("M,F,K", SPLIT_GLU)
def test_split_glu_fwd(M, F, K):
    with expected(ROWS, "fp8_glu_fwd", split=True):
        _glu_case(M, F, K, SILU, 511)
        _glu_case(M, F, K, GELU_TANH, 512, gu=False, q=None)
        _glu_case(M, F, K, RELU, 513, h=False, q=sq.E5M2)


def _jobs(shapes):
    out = []
    for M, N, K in shapes:
        g = gen(M + N)
        A, sa = to_codes(randn(g, M, K), 0)
        B, sb = to_codes(randn(g, N, K), 0)
        out.append((A, sa, B, sb, M, N, K))
    return out


def test_split_workspace_is_left_clean():
    """Calls of different sizes share one zeroed workspace and give, in any order, what a fresh one gives."""
    shapes = [(1, 10256, 8208), (64, 10256, 8208), (17, 10256, 8208), (139, 16, 22960), (1, 10256, 8208)]
    shared = _workspace(max(sq.fp8_gemm_act_workspace_bytes(*s) for s in shapes))
    for A, sa, B, sb, M, N, K in _jobs(shapes):
        outs = []
        for ws in (shared, torch.zeros_like(shared), shared):
            D = _empty(M, N, dtype=F32)
            with expected(ROWS, "fp8_gemm_act", split=True):
                sq.fp8_gemm_act(A, 0, sa, B, 0, sb, SILU, D=D, workspace=ws)
            outs.append(D)
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    # the gated block in the same workspace
    g = gen(3)
    A, sa = to_codes(randn(g, 17, 4112), 0)
    W, sw = to_codes(randn(g, 2 * 5200, 4112), 0)
    assert sq.fp8_glu_fwd_workspace_bytes(17, 5200, 4112) <= shared.numel()
    outs = []
    for ws in (shared, torch.zeros_like(shared)):
        h = _empty(17, 5200, dtype=BF)
        sq.fp8_glu_fwd(A, 0, sa, W, 0, sw, SILU, h_out=h, workspace=ws)
        outs.append(h)
    torch.cuda.synchronize()
    assert torch.equal(*outs) and not bool(shared[:COUNTERS].any())


@pytest.mark.parametrize("M,N,K", [(1, 10256, 8208), (40, 10256, 8208), (139, 16, 22960)])
def test_split_gives_the_same_bits_on_two_streams(M, N, K):
    """Whatever the order in which the shares end: each stream with a workspace of its own, beside the other's."""
    (A, sa, B, sb, *_), = _jobs([(M, N, K)])
    call = lambda D, ws, s=None: sq.fp8_gemm_act(A, 0, sa, B, 0, sb, SILU, D=D, workspace=ws, stream=s)  # noqa: E731
    jobs = [(torch.cuda.Stream(), _workspace(sq.fp8_gemm_act_workspace_bytes(M, N, K)),
             [_empty(M, N, dtype=F32) for _ in range(12)]) for _ in range(2)]
    assert launched(lambda: call(jobs[0][2][0], jobs[0][1])) == {ROWS}
    torch.cuda.synchronize()
    for i in range(12):
        for s, ws, outs in jobs:
            call(outs[i], ws, s)
    torch.cuda.synchronize()
    first = jobs[0][2][0]
    assert all(torch.equal(first, D) for _, _, outs in jobs for D in outs)
    for _, ws, _ in jobs:
        assert not bool(ws[:COUNTERS].any()) and bool(ws[COUNTERS:].any())
    assert sq.fp8_device_status(True) == sq.OK


# ---------------------------------------------------------------- K over a cluster, and whole tiles of few rows
@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (64, 4096, 4096), (200, 4096, 4096), (250, 4096, 14336)])
def test_clusters_are_taken(M, N, K):
    with expected(KSPLIT, "fp8_gemm_act"):
        _act_case(M, N, K, GELU, 521, res=F32, out=F32)


@pytest.mark.parametrize("M,N,K", [(16, 14336, 1040), (64, 20496, 2064), (777, 2064, 1040)])
def test_whole_tiles_of_few_rows_are_taken(M, N, K):
    with expected(ROWS, "fp8_gemm_act", split=False):
        _act_case(M, N, K, GELU, 531, res=F32, out=F32)
        _act_case(M, N, K, SILU, 532, bias=False, out=None, z=True, q=sq.E4M3)
