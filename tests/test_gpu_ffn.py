"""fp8_gemm_act, fp8_act_bwd, fp8_glu_fwd and fp8_glu_bwd against the
definitions in 64 bits (bounds: _ffn_ref.py)."""
import pytest
import torch

import scaled_quantize_gemm_gb300 as sq
from _ffn_ref import (ACTS, ELEM, FMAX, GELU, GELU_TANH, NONE, RELU, SILU, SLOPE, U, act64, assert_amax, assert_codes,
                      assert_within, gated, gen, new_state, product, randn, to_codes, values)

pytestmark = pytest.mark.gpu
DEV = "cuda"
H = 4
BF, F32 = torch.bfloat16, torch.float32
ACT_NAMES = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def _workspace(nbytes):
    return torch.zeros(nbytes, dtype=torch.uint8, device=DEV) if nbytes else None


def _empty(*shape, dtype):
    t = torch.empty(shape, dtype=dtype, device=DEV)
    return t.fill_(0x55 if dtype == torch.uint8 else 7.0)


# ---------------------------------------------------------------- gemm_act
def _act_case(M, N, K, act, seed, fa=sq.E4M3, fb=sq.E4M3, bias=True, res=None, out=BF, z=False, q=None, workspace=True,
              stream=None):
    g = gen(seed)
    A, sa = to_codes(randn(g, M, K), fa)
    B, sb = to_codes(randn(g, N, K) * K ** -0.5, fb)
    b = randn(g, N) * 0.5 if bias else None
    R = (randn(g, M, N) * 2).to(res) if res is not None else None
    D = _empty(M, N, dtype=out) if out is not None else None
    Z = _empty(M, N, dtype=BF) if z else None
    Q = _empty(M, N, dtype=torch.uint8) if q is not None else None
    m = 20.0 if q == sq.E4M3 else 3000.0
    st = new_state(H, m, 0.125) if q is not None else None
    ws = _workspace(sq.fp8_gemm_act_workspace_bytes(M, N, K)) if workspace else None
    sq.fp8_gemm_act(A, fa, sa, B, fb, sb, act, D=D, bias=b, residual=R, z_out=Z, q_out=Q,
                    q_format=q if q is not None else sq.E4M3, q_state=st, history_len=H if q is not None else 0,
                    workspace=ws, stream=stream)
    torch.cuda.synchronize()
    z64, ez = product(values(A, fa), values(B, fb), float(sa) * float(sb))
    if bias:
        z64 = z64 + b.double()
        ez = ez + 2 * U * (z64.abs() + b.double().abs())
    y64 = act64(z64, act)[0]
    ey = (0 if act == NONE else ELEM * z64.abs()) + SLOPE * ez
    if R is not None:
        y64 = y64 + R.double()
        ey = ey + 2 * U * y64.abs()
    what = f"{M}x{N}x{K} {ACT_NAMES[act]}"
    if Z is not None:
        assert_within(Z, z64, ez, what + " z")
    if D is not None:
        assert_within(D, y64, ey, what + " D")
    if Q is not None:
        assert_codes(Q, y64, ey, m, q, what + " codes")
        assert_amax(st, 0.125, y64, ey, what)
    if ws is not None:
        assert sq.fp8_device_status(True) == sq.OK
    return [t for t in (D, Z, Q, st) if t is not None]


SHAPES = [(1, 16, 16), (1, 264, 1040), (2, 4096, 2064), (5, 520, 144), (16, 2048, 512), (17, 2064, 4096),
          (33, 272, 8208), (64, 1024, 1024), (65, 528, 256), (100, 144, 272), (128, 640, 640), (129, 256, 128),
          (300, 784, 400), (513, 1040, 1296), (1000, 264, 32)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm_act_shapes(M, N, K):
    _act_case(M, N, K, SILU, 1)
    _act_case(M, N, K, NONE, 2, bias=False, res=BF)
    _act_case(M, N, K, GELU, 3, res=F32, out=F32)
    if N % 16 == 0:
        _act_case(M, N, K, GELU_TANH, 4, out=None, z=True, q=sq.E4M3)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [3, 150])
def test_gemm_act_activations(M, act):
    _act_case(M, 272, 528, act, 11 + act, out=F32)
    _act_case(M, 272, 528, act, 21 + act, bias=False, out=BF, z=True, q=sq.E4M3)


@pytest.mark.parametrize("fa,fb", [(0, 0), (0, 1), (1, 0), (1, 1)])
@pytest.mark.parametrize("M", [7, 200])
def test_gemm_act_formats(M, fa, fb):
    _act_case(M, 304, 432, RELU, 31, fa=fa, fb=fb, q=sq.E5M2, res=BF)
    _act_case(M, 304, 432, SILU, 32, fa=fa, fb=fb, out=F32, z=True)


@pytest.mark.parametrize("M", [1, 40, 260])
def test_gemm_act_without_workspace_agrees(M):
    """The split over K (few rows, with a workspace) and the unsplit product both hold their bounds."""
    _act_case(M, 528, 2064, SILU, 41, workspace=True)
    _act_case(M, 528, 2064, SILU, 41, workspace=False)


def test_gemm_act_workspace_is_left_clean():
    """Calls of different sizes share one zeroed workspace and give, in any order, what a fresh one gives."""
    sizes = [(1, 4096, 1024), (30, 1040, 4096), (2, 528, 16), (64, 2048, 2048), (1, 4096, 1024)]
    nbytes = max(sq.fp8_gemm_act_workspace_bytes(*s) for s in sizes)
    shared = torch.zeros(max(256, nbytes), dtype=torch.uint8, device=DEV)
    for M, N, K in sizes:
        g = gen(M + N)
        A, sa = to_codes(randn(g, M, K), 0)
        B, sb = to_codes(randn(g, N, K), 0)
        outs = []
        for ws in (shared, torch.zeros_like(shared), shared):
            D = _empty(M, N, dtype=F32)
            sq.fp8_gemm_act(A, 0, sa, B, 0, sb, SILU, D=D, workspace=ws)
            outs.append(D)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_gemm_act_empty():
    one = torch.ones(1, device=DEV)
    A, B = torch.empty((0, 32), dtype=torch.uint8, device=DEV), torch.zeros((16, 32), dtype=torch.uint8, device=DEV)
    sq.fp8_gemm_act(A, 0, one, B, 0, one, SILU, D=torch.empty((0, 16), device=DEV))
    sq.fp8_gemm_act(B, 0, one, A, 0, one, SILU, D=torch.empty((16, 0), device=DEV))
    torch.cuda.synchronize()


@pytest.mark.parametrize("M", [2, 140])
def test_gemm_act_nan_and_saturation(M):
    """A NaN code makes its row NaN and the amax NaN; large values clip at the format's largest."""
    K, N = 64, 48
    A = torch.full((M, K), 0x38, dtype=torch.uint8, device=DEV)          # 1.0
    B = torch.full((N, K), 0x38, dtype=torch.uint8, device=DEV)
    A[1, 5] = 0x7F
    one = torch.ones(1, device=DEV)
    st = new_state(H, 100.0)
    Q, D = _empty(M, N, dtype=torch.uint8), _empty(M, N, dtype=F32)
    sq.fp8_gemm_act(A, 0, one, B, 0, one, SILU, D=D, q_out=Q, q_state=st, history_len=H,
                    workspace=_workspace(sq.fp8_gemm_act_workspace_bytes(M, N, K)))
    torch.cuda.synchronize()
    v = Q.view(torch.float8_e4m3fn).float()
    assert bool(torch.isnan(D[1]).all()) and bool(torch.isnan(v[1]).all()) and bool(torch.isnan(st[0]))
    rows = [r for r in range(M) if r != 1]
    assert bool((D[rows] == 64.0).all()) and bool((v[rows] == 448.0).all())


# ---------------------------------------------------------------- act_bwd
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N", [(1, 1), (3, 7), (1, 4096), (17, 264), (700, 1000), (2000, 48), (65, 2056), (129, 8),
                                 (1, 17), (4000, 300)])
def test_act_bwd(M, N, act):
    g = gen(M + 3 * N)
    dy, z = randn(g, M, N).to(BF), (randn(g, M, N) * 3).to(BF)
    d64 = dy.double() * act64(z.double(), act)[1]
    # act' of a bf16 argument: the elementwise bound on its terms, |act''| u |z| among them
    e = dy.double().abs() * ELEM * (1 + z.double().abs())
    if act in (NONE, RELU):
        e = torch.zeros_like(e)
    for fmt, m in ((sq.E5M2, 4000.0), (sq.E4M3, 40.0)):
        dz, q, st = _empty(M, N, dtype=BF), _empty(M, N, dtype=torch.uint8), new_state(H, m, 0.25)
        db = _empty(N, dtype=F32)
        ws = torch.full((sq.fp8_act_bwd_workspace_bytes(M, N),), 0xFF, dtype=torch.uint8, device=DEV)
        sq.fp8_act_bwd(dy, z, act, dbias=db, dz=dz, q_out=q, q_format=fmt, q_state=st, history_len=H, workspace=ws)
        torch.cuda.synchronize()
        assert_within(dz, d64, e, "dz")
        assert_codes(q, d64, e, m, fmt, "codes")
        assert_amax(st, 0.25, d64, e, "amax")
        assert_within(db, d64.sum(0), ((M / 64 + 128) * U * d64.abs() + e).sum(0), "dbias")
    # each output alone gives the same
    dz2, q2, db2, st2 = _empty(M, N, dtype=BF), _empty(M, N, dtype=torch.uint8), _empty(N, dtype=F32), new_state(H, m)
    sq.fp8_act_bwd(dy, z, act, dz=dz2)
    sq.fp8_act_bwd(dy, z, act, q_out=q2, q_format=sq.E4M3, q_state=st2, history_len=H)
    sq.fp8_act_bwd(dy, z, act, dbias=db2, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(dz, dz2) and torch.equal(q, q2) and torch.equal(db, db2)


@pytest.mark.parametrize("act", ACTS)
def test_act_bwd_against_differences(act):
    g = gen(act)
    M, N, h = 8, 512, 1e-6
    z, dy = (randn(g, M, N) * 2).to(BF), randn(g, M, N).to(BF)
    dz = _empty(M, N, dtype=BF)
    sq.fp8_act_bwd(dy, z, act, dz=dz)
    v = randn(g, M, N).double()
    z64, dy64 = z.double(), dy.double()
    want = float(((act64(z64 + h * v, act)[0] - act64(z64 - h * v, act)[0]) * dy64).sum()) / (2 * h)
    got = dz.double() * v
    assert abs(float(got.sum()) - want) <= 2.0 ** -8 * float(got.abs().sum()) + 1e-6


@pytest.mark.parametrize("act", ACTS)
def test_act_bwd_extreme_arguments(act):
    """Large arguments give the limits of the derivative (0, or 1), never a NaN; a NaN stays one."""
    z = torch.tensor([-3e38, -1e20, -1e6, -1000.0, -200.0, -90.0, 90.0, 200.0, 1000.0, 1e6, 1e20, 3e38, float("nan"), 0.0, -0.0, 1.0],
                     device=DEV).to(BF).repeat(2, 1)
    dy = torch.ones_like(z)
    dz = _empty(2, 16, dtype=BF)
    sq.fp8_act_bwd(dy, z, act, dz=dz)
    torch.cuda.synchronize()
    lo = 1.0 if act == NONE else 0.0
    assert bool((dz[:, :6].float() - lo).abs().le(1e-30).all()) and bool((dz[:, 6:12] == 1).all())
    if act != NONE:
        assert bool(torch.isnan(dz[:, 12]).all())


def test_act_bwd_empty():
    z = torch.empty((0, 24), dtype=BF, device=DEV)
    db = _empty(24, dtype=F32)
    sq.fp8_act_bwd(z, z, SILU, dbias=db, workspace=torch.empty(1, dtype=torch.uint8, device=DEV))
    torch.cuda.synchronize()
    assert bool((db == 0).all())


# ---------------------------------------------------------------- glu
def _glu_case(M, F, K, act, seed, fa=sq.E4M3, fw=sq.E4M3, h=True, gu=True, q=sq.E4M3, workspace=True):
    g = gen(seed)
    A, sa = to_codes(randn(g, M, K), fa)
    W, sw = to_codes(randn(g, 2 * F, K) * K ** -0.5, fw)
    hb = _empty(M, F, dtype=BF) if h else None
    gub = _empty(M, 2 * F, dtype=BF) if gu else None
    Q = _empty(M, F, dtype=torch.uint8) if q is not None else None
    m = 30.0 if q == sq.E4M3 else 3000.0
    st = new_state(H, m, 0.0625) if q is not None else None
    ws = _workspace(sq.fp8_glu_fwd_workspace_bytes(M, F, K)) if workspace else None
    sq.fp8_glu_fwd(A, fa, sa, W, fw, sw, act, h_out=hb, gu_out=gub, q_out=Q, q_format=q if q is not None else 0,
                   q_state=st, history_len=H if q is not None else 0, workspace=ws)
    torch.cuda.synchronize()
    a, w, s = values(A, fa), values(W, fw), float(sa) * float(sw)
    z64, ez = product(a, w, s)
    h64, eh = gated(z64[:, :F], ez[:, :F], z64[:, F:], ez[:, F:], act)
    what = f"{M}x{F}x{K} {ACT_NAMES[act]}"
    if gub is not None:
        assert_within(gub, z64, ez, what + " gu")
    if hb is not None:
        assert_within(hb, h64, eh, what + " h")
    if Q is not None:
        assert_codes(Q, h64, eh, m, q, what + " codes")
        assert_amax(st, 0.0625, h64, eh, what)
    assert sq.fp8_device_status(True) == sq.OK


GLU_SHAPES = [(1, 16, 16), (1, 1040, 528), (3, 4096, 2048), (8, 144, 4112), (16, 2064, 256), (31, 272, 1040),
              (40, 6160, 304), (64, 1024, 2048), (65, 528, 272), (128, 400, 640), (130, 256, 128), (257, 48, 144),
              (600, 912, 528)]


@pytest.mark.parametrize("M,F,K", GLU_SHAPES)
def test_glu_fwd_shapes(M, F, K):
    _glu_case(M, F, K, SILU, 51)
    _glu_case(M, F, K, GELU_TANH, 52, h=True, gu=False, q=None)
    _glu_case(M, F, K, GELU, 53, h=False, gu=True, q=sq.E5M2)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [4, 180])
def test_glu_fwd_activations(M, act):
    _glu_case(M, 304, 528, act, 61 + act)


@pytest.mark.parametrize("fa,fw", [(0, 1), (1, 0), (1, 1)])
@pytest.mark.parametrize("M", [9, 200])
def test_glu_fwd_formats(M, fa, fw):
    _glu_case(M, 176, 400, SILU, 71, fa=fa, fw=fw)


@pytest.mark.parametrize("M", [1, 33])
def test_glu_fwd_without_workspace(M):
    _glu_case(M, 272, 1040, SILU, 81, workspace=False)


def _glu_bwd_case(M, F, K, act, seed, fdy=sq.E5M2, fw=sq.E4M3, q=sq.E5M2):
    g = gen(seed)
    dY, sd = to_codes(randn(g, M, K) * 1e-2, fdy)
    Wd, sw = to_codes(randn(g, K, F) * F ** -0.5, fw)
    gu = (randn(g, M, 2 * F) * 1.5).to(BF)
    Q = _empty(M, 2 * F, dtype=torch.uint8)
    m = 30000.0 if q == sq.E5M2 else 300.0
    st = new_state(H, m)
    sq.fp8_glu_bwd(dY, fdy, sd, Wd, fw, sw, gu, act, Q, q, st, H)
    torch.cuda.synchronize()
    dh, eh = product(values(dY, fdy), values(Wd, fw).T, float(sd) * float(sw))
    gg, uu = gu[:, :F].double(), gu[:, F:].double()
    f, d = act64(gg, act)
    ef = ELEM * (1 + gg.abs())
    want = torch.cat([dh * uu * d, dh * f], 1)
    e = torch.cat([uu.abs() * (eh * d.abs() + (dh.abs() + eh) * ef), eh * f.abs() + (dh.abs() + eh) * ef], 1) + ELEM * want.abs()
    what = f"{M}x{F}x{K} {ACT_NAMES[act]}"
    assert_codes(Q, want, e, m, q, what)
    assert_amax(st, 0.0, want, e, what)
    return dh, gg, uu, Q, m


@pytest.mark.parametrize("M,F,K", [(1, 16, 16), (1, 1040, 528), (16, 272, 144), (130, 528, 272), (257, 256, 128),
                                   (300, 400, 1040), (520, 784, 256)])
def test_glu_bwd_shapes(M, F, K):
    _glu_bwd_case(M, F, K, SILU, 91)
    _glu_bwd_case(M, F, K, GELU, 92, fdy=sq.E4M3, q=sq.E4M3)


@pytest.mark.parametrize("act", ACTS)
def test_glu_bwd_activations(act):
    _glu_bwd_case(140, 304, 272, act, 101 + act)


@pytest.mark.parametrize("act", [GELU, GELU_TANH, SILU])
def test_glu_bwd_against_differences(act):
    """Directional derivatives of sum(dh h(g, u)) from the codes, within their rounding (an eighth of a step's
    value each), against central differences."""
    M, F = 64, 272
    dh, g, u, Q, m = _glu_bwd_case(M, F, 144, act, 111)
    grad = values(Q, sq.E5M2) / m
    r = gen(7)
    vg, vu = randn(r, M, F).double(), randn(r, M, F).double()
    eps = 1e-6
    loss = lambda t: float((act64(g + t * vg, act)[0] * (u + t * vu) * dh).sum())                # noqa: E731
    want = (loss(eps) - loss(-eps)) / (2 * eps)
    terms = grad * torch.cat([vg, vu], 1)
    # rounding errors are half a step each; the smallest subnormal's half step below the normal range
    tol = 2.0 ** -3 * float(terms.abs().sum()) + 2.0 ** -17 / m * float(vg.abs().sum() + vu.abs().sum()) + 1e-7
    assert abs(float(terms.sum()) - want) <= tol


def test_glu_whole_step_matches_64_bits():
    """Forward codes -> down projection, then the gradient codes through the framework's products, as a user chains
    them: each product against 64 bits on the codes that went in."""
    M, K, F = 272, 144, 400
    g = gen(17)
    x, sx = to_codes(randn(g, M, K), 0)
    w, sw = to_codes(randn(g, 2 * F, K) * K ** -0.5, 0)
    wd, swd = to_codes(randn(g, K, F) * F ** -0.5, 0)
    dy, sdy = to_codes(randn(g, M, K) * 1e-3, 1)
    sth, stg = new_state(H, 60.0), new_state(H, 1e6)
    q, gu, dq = _empty(M, F, dtype=torch.uint8), _empty(M, 2 * F, dtype=BF), _empty(M, 2 * F, dtype=torch.uint8)
    y, dx, dw, dwd = _empty(M, K, dtype=BF), _empty(M, K, dtype=BF), _empty(2 * F, K, dtype=F32), _empty(K, F, dtype=F32)
    sq.fp8_glu_fwd(x, 0, sx, w, 0, sw, SILU, gu_out=gu, q_out=q, q_state=sth, history_len=H)
    sq.fp8_gemm_act(q, 0, sth[H + 1:], wd, 0, swd, NONE, D=y)
    sq.fp8_glu_bwd(dy, 1, sdy, wd, 0, swd, gu, SILU, dq, 1, stg, H)
    sq.fp8_gemm_layout(dq, 1, stg[H + 1:], sq.K_MAJOR, w, 0, sw, sq.MN_MAJOR, dx, M, K, 2 * F)
    sq.fp8_gemm_layout(dq, 1, stg[H + 1:], sq.MN_MAJOR, x, 0, sx, sq.MN_MAJOR, dw, 2 * F, K, M)
    sq.fp8_gemm_layout(dy, 1, sdy, sq.MN_MAJOR, q, 0, sth[H + 1:], sq.MN_MAJOR, dwd, K, F, M)
    torch.cuda.synchronize()
    X, W, WD, DY, Qv, DQ = values(x, 0), values(w, 0), values(wd, 0), values(dy, 1), values(q, 0), values(dq, 1)
    sh, sg = float(sth[H + 1]), float(stg[H + 1])
    for got, a, b, s in ((y, Qv, WD, sh * float(swd)), (dx, DQ, W.T, sg * float(sw)), (dw, DQ.T, X.T, sg * float(sx)),
                         (dwd, DY.T, Qv.T, float(sdy) * sh)):
        assert_within(got, *product(a, b, s), "product")


# ---------------------------------------------------------------- streams, graphs, failure
@pytest.mark.parametrize("M", [2, 200])
def test_other_stream_and_graph(M):
    K, F = 528, 400
    g = gen(23)
    x, sx = to_codes(randn(g, M, K), 0)
    w, sw = to_codes(randn(g, 2 * F, K), 0)
    wd, swd = to_codes(randn(g, K, F), 0)
    st = new_state(H, 1.0)
    q, y = _empty(M, F, dtype=torch.uint8), _empty(M, K, dtype=F32)
    wa, wb = _workspace(sq.fp8_glu_fwd_workspace_bytes(M, F, K)), _workspace(sq.fp8_gemm_act_workspace_bytes(M, K, F))

    def step():
        sq.fp8_glu_fwd(x, 0, sx, w, 0, sw, SILU, q_out=q, q_state=st, history_len=H, workspace=wa)
        sq.fp8_gemm_act(q, 0, st[H + 1:], wd, 0, swd, NONE, D=y, workspace=wb)

    step()
    torch.cuda.synchronize()
    want = y.clone()
    y.zero_()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x.copy_(to_codes(randn(g, M, K), 0)[0])
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    replayed = y.clone()
    step()
    torch.cuda.synchronize()
    assert torch.equal(replayed, y) and not torch.equal(y, want)


@pytest.mark.parametrize("M", [2, 200])
def test_products_skip_while_the_error_word_is_set(M):
    K, N = 128, 64
    A = torch.full((M, K), 0x38, dtype=torch.uint8, device=DEV)
    B = torch.full((N, K), 0x38, dtype=torch.uint8, device=DEV)
    one = torch.ones(1, device=DEV)
    ws = _workspace(sq.fp8_gemm_act_workspace_bytes(M, N, K))
    D = _empty(M, N, dtype=F32)
    waited = torch.zeros(1, dtype=torch.int32, device=DEV)
    assert sq.fp8_device_status(True) == sq.OK
    sq.fp8_selftest_wait_timeout(1000, waited)
    sq.fp8_gemm_act(A, 0, one, B, 0, one, NONE, D=D, workspace=ws)
    torch.cuda.synchronize()
    assert bool((D == 7.0).all())
    assert sq.fp8_device_status(True) == sq.ERR_TIMEOUT
    if ws is not None:
        ws.zero_()
    sq.fp8_gemm_act(A, 0, one, B, 0, one, NONE, D=D, workspace=ws)
    torch.cuda.synchronize()
    assert bool((D == 128.0).all())
