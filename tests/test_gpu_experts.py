"""The experts' products against the definitions in 64 bits, expert by expert (bounds: _ffn_ref.py)."""
import pytest
import torch

import scaled_quantize_gemm_gb300 as sq
from _experts_ref import make_plan, place, routing, walk
from _ffn_ref import (ELEM, GELU, GELU_TANH, SILU, U, act64, assert_amax, assert_codes, assert_within,
                      gated, gen, new_state, product, randn, to_codes, values)

pytestmark = pytest.mark.gpu
DEV, H = "cuda", 4
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


class Case:
    """A routing, its sorted codes and the experts' weights."""

    def __init__(self, T, k, E, how, seed=1):
        self.T, self.k, self.E, self.g = T, k, E, gen(seed)
        self.ids = routing(self.g, T, k, E, how)
        self.plan = make_plan(self.ids, E)
        row, self.offsets, self.counts = walk(self.ids, E)
        self.row, self.R = row.to(DEV), sq.fp8_expert_rows(T, k, E)
        self.end = self.offsets[-1]

    def rows(self, K, fmt, scale=1.0):
        q, s = to_codes(randn(self.g, self.T, K) * scale, fmt)
        return place(self.row, q, self.R), s

    def weights(self, n, k, fmt=0):
        q, s = zip(*(to_codes(randn(self.g, n, k) * k ** -0.5 * (1 + e % 3), fmt) for e in range(self.E)))
        return torch.stack(q), torch.cat(s)

    def experts(self):
        return [(e, slice(self.offsets[e], self.offsets[e + 1])) for e in range(self.E) if self.counts[e]]

    def empty(self, *shape, dtype):
        return torch.full(shape, 0x55 if dtype == U8 else 7.0, dtype=dtype, device=DEV)

    def untouched(self, *outs):
        for t in outs:
            assert bool((t[self.end:] == (0x55 if t.dtype == U8 else 7.0)).all()), "rows behind the last segment"

    def workspace(self, N, K):
        n = sq.fp8_expert_workspace_bytes(self.T, self.k, self.E, N, K)
        return torch.zeros(n, dtype=U8, device=DEV) if n else None


# T, k, E, routing, hidden, inner
CASES = [(1, 1, 1, "spread", 32, 16), (1, 8, 64, "spread", 1024, 272), (7, 2, 3, "masked", 160, 144), (37, 3, 5, "skewed", 544, 80),
         (300, 1, 2, "one", 96, 528), (333, 4, 7, "masked", 256, 320), (1000, 2, 16, "last", 64, 256),
         (5000, 1, 2, "skewed", 32, 48), (5, 2, 4, "none", 64, 32), (64, 8, 24, "spread", 4096, 512), (40, 4, 40, "skewed", 2304, 144),
         (200, 4, 40, "skewed", 160, 96), (3, 2, 6, "spread", 2720, 4112), (1200, 2, 3, "spread", 2080, 1040)]


@pytest.mark.parametrize("T,k,E,how,d,F", CASES)
@pytest.mark.parametrize("split", [True, False])
def test_products(T, k, E, how, d, F, split):
    """K-major and MN-major weights, bf16 and fp32, mixed formats."""
    c = Case(T, k, E, how)
    A, sa = c.rows(d, sq.E4M3)
    B, sb = c.weights(F, d)
    D, D32 = c.empty(c.R, F, dtype=BF), c.empty(c.R, F, dtype=F32)
    ws = c.workspace(F, d) if split else None
    sq.fp8_expert_gemm(A, 0, sa, B, 0, sb, sq.K_MAJOR, c.plan, T, k, D, workspace=ws)
    sq.fp8_expert_gemm(A, 0, sa, B, 0, sb, sq.K_MAJOR, c.plan, T, k, D32, workspace=ws)
    A5, sa5 = c.rows(d, sq.E5M2)
    Bt, sbt = c.weights(d, F)
    Dt = c.empty(c.R, F, dtype=BF)
    sq.fp8_expert_gemm(A5, 1, sa5, Bt, 0, sbt, sq.MN_MAJOR, c.plan, T, k, Dt)
    for e, r in c.experts():
        z, ez = product(values(A[r], 0), values(B[e], 0), float(sa) * float(sb[e]))
        assert_within(D[r], z, ez, f"expert {e}")
        assert_within(D32[r], z, ez, f"expert {e} fp32")
        z, ez = product(values(A5[r], 1), values(Bt[e], 0).T, float(sa5) * float(sbt[e]))
        assert_within(Dt[r], z, ez, f"expert {e} MN-major")
    c.untouched(D, D32, Dt)
    assert sq.fp8_device_status(True) == sq.OK


@pytest.mark.parametrize("T,k,E,how,d,F", CASES)
@pytest.mark.parametrize("act", [SILU, GELU])
def test_gated(T, k, E, how, d, F, act):
    c = Case(T, k, E, how, seed=2)
    A, sa = c.rows(d, sq.E4M3)
    W, sw = c.weights(2 * F, d)
    gu, h, q, st = c.empty(c.R, 2 * F, dtype=BF), c.empty(c.R, F, dtype=BF), c.empty(c.R, F, dtype=U8), new_state(H, 20.0, 0.125)
    sq.fp8_expert_glu_fwd(A, 0, sa, W, 0, sw, act, c.plan, T, k, h_out=h, gu_out=gu, q_out=q, q_state=st, history_len=H,
                          workspace=c.workspace(2 * F, d))
    q2, st2 = c.empty(c.R, F, dtype=U8), new_state(H, 20.0, 0.125)
    sq.fp8_expert_glu_fwd(A, 0, sa, W, 0, sw, act, c.plan, T, k, q_out=q2, q_state=st2, history_len=H)
    want, err = torch.zeros((0, F), dtype=torch.float64, device=DEV), torch.zeros((0, F), dtype=torch.float64, device=DEV)
    for e, r in c.experts():
        z, ez = product(values(A[r], 0), values(W[e], 0), float(sa) * float(sw[e]))
        assert_within(gu[r], z, ez, f"expert {e} g, u")
        y, ey = gated(z[:, :F], ez[:, :F], z[:, F:], ez[:, F:], act)
        assert_within(h[r], y, ey, f"expert {e} h")
        assert_codes(q[r], y, ey, 20.0, 0, f"expert {e}")
        assert_codes(q2[r], y, ey, 20.0, 0, f"expert {e}")
        want, err = torch.cat([want, y]), torch.cat([err, ey])
    assert_amax(st, 0.125, want, err)
    assert_amax(st2, 0.125, want, err)
    c.untouched(gu, h, q, q2)
    assert sq.fp8_device_status(True) == sq.OK


@pytest.mark.parametrize("T,k,E,how,d,F", CASES)
@pytest.mark.parametrize("act", [SILU, GELU_TANH])
def test_gated_backward(T, k, E, how, d, F, act):
    c = Case(T, k, E, how, seed=3)
    dY, sd = c.rows(d, sq.E5M2)
    Wd, sw = c.weights(d, F)
    gu = place(c.row, randn(c.g, T, k, 2 * F).to(BF), c.R)
    q, st = c.empty(c.R, 2 * F, dtype=U8), new_state(H, 300.0, 0.125)
    sq.fp8_expert_glu_bwd(dY, 1, sd, Wd, 0, sw, gu, act, c.plan, T, k, q, sq.E5M2, st, H)
    want, err = [torch.zeros((0, 2 * F), dtype=torch.float64, device=DEV)], [torch.zeros((0, 2 * F), dtype=torch.float64, device=DEV)]
    for e, r in c.experts():
        dh, eh = product(values(dY[r], 1), values(Wd[e], 0).T, float(sd) * float(sw[e]))
        g, u = gu[r, :F].double(), gu[r, F:].double()
        f, df = act64(g, act)
        y = torch.cat([dh * u * df, dh * f], 1)
        # derivative and value of the activation: ELEM of what enters them
        ed = ELEM * (1 + g.abs())
        ey = torch.cat([eh * (u * df).abs() + dh.abs() * u.abs() * ed, eh * f.abs() + dh.abs() * ELEM * g.abs()], 1)
        ey = ey + 4 * U * y.abs() + torch.cat([eh * u.abs() * ed, eh * ELEM * g.abs()], 1)
        assert_codes(q[r], y, ey, 300.0, 1, f"expert {e}")
        want.append(y)
        err.append(ey)
    assert_amax(st, 0.125, torch.cat(want), torch.cat(err))
    c.untouched(q)
    assert sq.fp8_device_status(True) == sq.OK


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("T,k,E,how,d,F", CASES)
def test_weight_gradients(T, k, E, how, d, F, out):
    c = Case(T, k, E, how, seed=4)
    A, sa = c.rows(d, sq.E5M2)
    B, sb = c.rows(F, sq.E4M3)
    # rows behind the last segment are not summed, whatever they hold
    A[c.end:], B[c.end:] = 0x7F, 0x7F
    D = c.empty(E, d, F, dtype=out)
    sq.fp8_expert_wgrad(A, 1, sa, B, 0, sb, c.plan, T, k, D)
    seen = dict(c.experts())
    for e in range(E):
        if e not in seen:
            assert not bool(D[e].any()), "an expert without rows"
            continue
        z, ez = product(values(A[seen[e]], 1).T.contiguous(), values(B[seen[e]], 0).T.contiguous(), float(sa) * float(sb))
        assert_within(D[e], z, ez, f"expert {e}")
    assert sq.fp8_device_status(True) == sq.OK


def test_neighbours_do_not_mix():
    """NaN codes in one expert's rows and weights stay with that expert."""
    c = Case(90, 2, 6, "spread", seed=5)
    A, sa = c.rows(256, 0)
    B, sb = c.weights(160, 256)
    Bt, sbt = c.weights(256, 160)
    r = slice(c.offsets[2], c.offsets[3])
    A[r], B[2], Bt[2] = 0x7F, 0x7F, 0x7F
    for b, s, major in ((B, sb, sq.K_MAJOR), (Bt, sbt, sq.MN_MAJOR)):
        D = c.empty(c.R, 160, dtype=F32)
        sq.fp8_expert_gemm(A, 0, sa, b, 0, s, major, c.plan, 90, 2, D)
        bad = torch.isnan(D[:c.end]).all(1)
        assert bool(bad[r].all()) and int(bad.sum()) == r.stop - r.start and int(torch.isnan(D[:c.end]).any(1).sum()) == int(bad.sum())
    D = c.empty(6, 256, 160, dtype=F32)
    X, sx = c.rows(160, 0)
    sq.fp8_expert_wgrad(A, 0, sa, X, 0, sx, c.plan, 90, 2, D)
    bad = torch.isnan(D).any(2).any(1).tolist()
    assert bad == [e == 2 for e in range(6)]


def test_repeats_streams_and_graphs():
    """The same bits every time, on another stream, in a graph whose routing changes, two calls at once."""
    T, k, E, d, F = 700, 3, 10, 512, 416
    c = Case(T, k, E, "skewed", seed=6)
    A, sa = c.rows(d, 0)
    W, sw = c.weights(2 * F, d)
    Wd, sd = c.weights(d, F)
    st = new_state(H, 20.0)

    def call(plan, q, D, dW, stream=None):
        sq.fp8_expert_glu_fwd(A, 0, sa, W, 0, sw, SILU, plan, T, k, q_out=q, q_state=st, history_len=H, stream=stream)
        sq.fp8_expert_gemm(q, 0, st[H + 1:], Wd, 0, sd, sq.K_MAJOR, plan, T, k, D, stream=stream)
        sq.fp8_expert_wgrad(q, 0, st[H + 1:], A, 0, sa, plan, T, k, dW, stream=stream)
    z = lambda *s, dtype=F32: torch.zeros(s, dtype=dtype, device=DEV)                             # noqa: E731
    outs = lambda: (z(c.R, F, dtype=U8), z(c.R, d), z(E, F, d))                                   # noqa: E731
    first = outs()
    call(c.plan, *first)
    torch.cuda.synchronize()
    sets = [outs() for _ in range(4)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i, o in enumerate(sets):
        call(c.plan, *o, stream=streams[i & 1])
    torch.cuda.synchronize()
    for o in sets:
        assert all(torch.equal(p, q) for p, q in zip(first, o))
    ids, plan, o = c.ids.clone(), c.plan.clone(), outs()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sq.fp8_expert_plan(ids, E, plan)
        call(plan, *o)
    ids.copy_(routing(c.g, T, k, E, "none"))
    graph.replay()
    assert not bool(o[2].any()) and not bool(o[0].any())
    ids.copy_(c.ids)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, o))
    assert sq.fp8_device_status(True) == sq.OK


def test_products_skip_while_the_error_word_is_set():
    T, k, E, d, F = 300, 2, 4, 256, 256
    c = Case(T, k, E, "spread", seed=7)
    A, sa = c.rows(d, 0)
    B, sb = c.weights(F, d)
    D, want = c.empty(c.R, F, dtype=F32), c.empty(c.R, F, dtype=F32)
    call = lambda o: sq.fp8_expert_gemm(A, 0, sa, B, 0, sb, sq.K_MAJOR, c.plan, T, k, o, workspace=c.workspace(F, d))  # noqa: E731
    call(want)
    sq.fp8_selftest_wait_timeout(1000, torch.zeros(1, dtype=torch.int32, device=DEV))
    call(D)
    torch.cuda.synchronize()
    assert bool((D == 7).all())
    assert sq.fp8_device_status(True) == sq.ERR_TIMEOUT
    call(D)
    torch.cuda.synchronize()
    assert torch.equal(D, want) and sq.fp8_device_status(True) == sq.OK


def test_no_tokens():
    E, d, F = 3, 64, 32
    plan = make_plan(torch.empty((0, 2), dtype=torch.int32, device=DEV), E)
    D, u8 = torch.full((E, d, F), 7.0, device=DEV), lambda *s: torch.empty(s, dtype=U8, device=DEV)       # noqa: E731
    one = torch.ones(3, device=DEV)
    sq.fp8_expert_wgrad(u8(0, d), 0, one, u8(0, F), 0, one, plan, 0, 2, D)
    sq.fp8_expert_gemm(u8(0, d), 0, one, u8(E, F, d), 0, one, sq.K_MAJOR, plan, 0, 2, torch.empty((0, F), device=DEV))
    sq.fp8_expert_glu_fwd(u8(0, d), 0, one, u8(E, 2 * F, d), 0, one, SILU, plan, 0, 2, h_out=torch.empty((0, F), dtype=BF, device=DEV))
    torch.cuda.synchronize()
    assert not bool(D.any())
