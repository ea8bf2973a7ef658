"""RMSNorm and the experts' operators over random sizes, more than 2^31 elements, and while other waits run out."""
import random

import pytest
import torch

import scaled_quantize_gemm_gb300 as sq
from _experts_ref import make_plan, routing, walk
from _ffn_ref import SILU, U, assert_amax, assert_codes, assert_within, gated, gen, new_state, product, randn, to_codes, values
from test_gpu_experts import BF, DEV, F32, H, U8, Case

pytestmark = pytest.mark.gpu


def _log(rng, lo, hi, mult=1):
    return max(1, round((lo / mult) * (hi / lo) ** rng.random())) * mult


@pytest.mark.parametrize("seed", range(24))
def test_random_sublayers(seed):
    """Dispatch, gated product, down projection, combination; and the weight gradients of what comes of them."""
    rng = random.Random(seed)
    E = _log(rng, 1, 100)
    k = rng.randint(1, min(8, E))
    T, d, F = _log(rng, 1, 3000 // k), _log(rng, 32, 1500, 32), _log(rng, 16, 900, 16)
    c = Case(T, k, E, rng.choice(["spread", "masked", "skewed", "one", "last"]), seed=seed)
    q, sx = to_codes(randn(c.g, T, d), 0)
    x = c.empty(c.R, d, dtype=U8)
    sq.fp8_expert_dispatch(q, c.plan, k, E, x)
    W, sw = c.weights(2 * F, d)
    Wd, sd = c.weights(d, F)
    h, y, st = c.empty(c.R, F, dtype=U8), c.empty(c.R, d, dtype=BF), new_state(H, 20.0, 0.125)
    sq.fp8_expert_glu_fwd(x, 0, sx, W, 0, sw, SILU, c.plan, T, k, q_out=h, q_state=st, history_len=H, workspace=c.workspace(2 * F, d))
    sq.fp8_expert_gemm(h, 0, st[H + 1:], Wd, 0, sd, sq.K_MAJOR, c.plan, T, k, y, workspace=c.workspace(d, F))
    res, w = randn(c.g, T, d).to(BF), torch.rand((T, k), generator=c.g, device=DEV)
    out = torch.empty_like(res)
    sq.fp8_expert_combine(y, c.plan, k, E, out, weights=w, residual=res)
    D = c.empty(E, d, F, dtype=F32)
    sq.fp8_expert_wgrad(x, 0, sx, h, 0, st[H + 1:], c.plan, T, k, D)
    what = f"T {T} k {k} E {E} d {d} F {F}"
    step = float(st[H + 1])
    for e, r in c.experts():
        z, ez = product(values(x[r], 0), values(W[e], 0), float(sx) * float(sw[e]))
        v, ev = gated(z[:, :F], ez[:, :F], z[:, F:], ez[:, F:], SILU)
        assert_codes(h[r], v, ev, 20.0, 0, what)
        z, ez = product(values(h[r], 0), values(Wd[e], 0), step * float(sd[e]))
        assert_within(y[r], z, ez, what)
        z, ez = product(values(x[r], 0).T.contiguous(), values(h[r], 0).T.contiguous(), float(sx) * step)
        assert_within(D[e], z, ez, what)
    want, mag = res.double(), res.double().abs()
    for j in range(k):
        on = c.row[:, j] >= 0
        v = y[c.row[on, j].long()].double() * w[on, j:j + 1].double()
        want[on] += v
        mag[on] += v.abs()
    assert_within(out, want, (k + 2) * U * mag, what)
    c.untouched(x, h, y)
    assert sq.fp8_device_status(True) == sq.OK


def test_rows_beyond_31_bits():
    """The last rows of sorted buffers with more than 2^31 elements."""
    T, k, E, K = 300001, 2, 3, 4096
    g = gen(1)
    ids = routing(g, T, k, E, "spread")
    plan = make_plan(ids, E)
    offsets, counts, row = sq.expert_plan_views(plan, T, k, E)
    R = sq.fp8_expert_rows(T, k, E)
    assert R * K > 1 << 31
    x = torch.randint(0, 120, (T, K), generator=g, device=DEV, dtype=U8)
    rows = torch.empty((R, K), dtype=U8, device=DEV)
    sq.fp8_expert_dispatch(x, plan, k, E, rows)
    for j in range(k):
        for lo in range(0, T, 65536):
            at = row[lo:lo + 65536, j].long()
            assert torch.equal(rows[at], x[lo:lo + 65536])
    # and a product of them: the last expert's rows
    B, sb = to_codes(randn(g, E * 4096, 32).view(E * 4096, 32), 0)
    B, sb = B.view(E, 4096, 32), sb.repeat(E)
    A = rows.view(-1)[:R * 32].view(R, 32)
    D = torch.empty((R, 4096), dtype=BF, device=DEV)
    sq.fp8_expert_gemm(A, 0, sb, B, 0, sb, sq.K_MAJOR, plan, T, k, D)
    s = slice(int(offsets[E]) - 500, int(offsets[E]))
    z, ez = product(values(A[s], 0), values(B[E - 1], 0), float(sb[0]) ** 2)
    assert_within(D[s], z, ez, "the last rows")
    del x, rows, A
    # back: bf16 rows of more than 2^32 bytes
    w, y, dw = torch.rand((T, k), generator=g, device=DEV), torch.empty((T, 4096), dtype=BF, device=DEV), torch.empty((T, k), device=DEV)
    sq.fp8_expert_combine(D, plan, k, E, y, weights=w)
    dy = randn(g, T, 4096).to(BF)
    q, st = torch.empty((R, 4096), dtype=U8, device=DEV), new_state(H, 500.0)
    sq.fp8_expert_combine_bwd(dy, plan, k, E, w, rows=D, dweights=dw, q_out=q, q_format=sq.E5M2, q_state=st, history_len=H)
    t = torch.cat([torch.arange(200, device=DEV), torch.arange(T - 200, T, device=DEV)])
    v = D[row[t].long()].double()
    p = v * w[t][:, :, None].double()
    assert_within(y[t], p.sum(1), (k + 2) * U * p.abs().sum(1), "combine")
    p = v * dy[t][:, None].double()
    assert_within(dw[t], p.sum(2), 4100 * U * p.abs().sum(2), "dweights")
    d = dy[t][:, None].double() * w[t][:, :, None].double()
    assert_codes(q[row[t].long()], d, 2 * U * d.abs(), 500.0, sq.E5M2, "drows")
    assert sq.fp8_device_status(True) == sq.OK


def test_weight_gradients_beyond_31_bits():
    E, M, N = 70, 4128, 8192
    c = Case(400, 1, E, "spread")
    assert E * M * N > 1 << 31
    A, sa = c.rows(M, 1)
    B, sb = c.rows(N, 0)
    D = torch.empty((E, M, N), dtype=BF, device=DEV)
    sq.fp8_expert_wgrad(A, 1, sa, B, 0, sb, c.plan, 400, 1, D)
    for e, r in [c.experts()[0], c.experts()[-1]]:
        z, ez = product(values(A[r], 1).T[-300:].contiguous(), values(B[r], 0).T.contiguous(), float(sa) * float(sb))
        assert_within(D[e][-300:], z, ez, f"expert {e}")


# the few-rows kernel with K split, one CTA a tile, tiles of 256 rows, the weights MN-major, weight gradients
@pytest.mark.parametrize("how,T,k,E,N,K", [("few", 4, 1, 4, 2064, 4096), ("single", 30, 4, 24, 2064, 4096), ("tiles", 2000, 2, 5, 1040, 1056), ("mn", 2000, 2, 5, 1040, 1056),
                                          ("wgrad", 2000, 2, 5, 1040, 1056)])
def test_a_word_set_while_products_start(how, T, k, E, N, K):
    c = Case(T, k, E, "spread", seed=T)
    A, sa = c.rows(K, 0)
    B, sb = c.weights(K, N) if how == "mn" else c.weights(N, K) if how != "wgrad" else c.rows(N, 0)
    D = torch.zeros((E, K, N) if how == "wgrad" else (c.R, N), device=DEV)
    ws = c.workspace(N, K)
    assert (ws is not None) == (how == "few")

    def call(s=None):
        if how == "wgrad":
            sq.fp8_expert_wgrad(A, 0, sa, B, 0, sb, c.plan, T, k, D, stream=s)
        else:
            sq.fp8_expert_gemm(A, 0, sa, B, 0, sb, sq.MN_MAJOR if how == "mn" else sq.K_MAJOR, c.plan, T, k, D, workspace=ws, stream=s)
    assert sq.fp8_device_status(True) == sq.OK
    call()
    torch.cuda.synchronize()
    want = D.clone()
    waited = torch.zeros(1, dtype=torch.int32, device=DEV)
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(24):
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


# one plan buffer for one routing after another, the product right behind the sort: what its CTAs fetch before their
# wait follows the routing before
@pytest.mark.parametrize("how,T,k,E,N,K", [("few", 4, 1, 4, 2064, 4096), ("single", 30, 4, 24, 2064, 4096), ("tiles", 2000, 2, 5, 1040, 1056), ("mn", 2000, 2, 5, 1040, 1056)])
def test_products_right_behind_their_plan(how, T, k, E, N, K):
    c = Case(T, k, E, "spread", seed=T + 1)
    A, sa = to_codes(randn(c.g, c.R, K), 0)
    B, sb = c.weights(K, N) if how == "mn" else c.weights(N, K)
    ws = c.workspace(N, K)
    ways = [routing(c.g, T, k, E, h) for h in ("spread", "last", "none", "masked", "one", "skewed", "spread", "masked")]
    plan = torch.zeros_like(c.plan)

    def call(p, out):
        sq.fp8_expert_gemm(A, 0, sa, B, 0, sb, sq.MN_MAJOR if how == "mn" else sq.K_MAJOR, p, T, k, out, workspace=ws)
    want = []
    for ids in ways:
        want.append(torch.zeros((c.R, N), device=DEV))
        p = make_plan(ids, E)
        torch.cuda.synchronize()
        call(p, want[-1])
        torch.cuda.synchronize()
    got = [torch.zeros((c.R, N), device=DEV) for _ in ways]

    def chain():
        for ids, out in zip(ways, got):
            sq.fp8_expert_plan(ids, E, plan)
            call(plan, out)
    chain()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for _ in range(5):
        for out in got:
            out.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_products_refuse_outputs_over_other_buffers():
    T, k, E, d, F = 40, 2, 3, 64, 96
    c = Case(T, k, E, "spread")
    buf = torch.zeros(1 << 20, dtype=U8, device=DEV)
    v = lambda *s: buf[:s[0] * s[1] * (s[2] if len(s) > 2 else 1)].view(*s)                       # noqa: E731
    A, W, one, st = torch.zeros((c.R, d), dtype=U8, device=DEV), torch.zeros((E, 2 * F, d), dtype=U8, device=DEV), torch.ones(E, device=DEV), new_state(H, 1.0)
    q = torch.zeros((c.R, F), dtype=U8, device=DEV)
    for names, call in ((("q_out", "A"), lambda: sq.fp8_expert_glu_fwd(v(c.R, d), 0, one, W, 0, one, SILU, c.plan, T, k, q_out=v(c.R, F), q_state=st, history_len=H)),
                        (("D", "B"), lambda: sq.fp8_expert_gemm(q, 0, one, v(E, d, F), 0, one, sq.K_MAJOR, c.plan, T, k, buf[:4 * c.R * d].view(F32).view(c.R, d))),
                        (("q_dgu", "Wd"), lambda: sq.fp8_expert_glu_bwd(A, 1, one, v(E, d, F), 0, one, torch.zeros((c.R, 2 * F), dtype=BF, device=DEV), SILU,
                                                                        c.plan, T, k, v(c.R, 2 * F), 1, st, H)),
                        (("D", "A"), lambda: sq.fp8_expert_wgrad(v(c.R, d), 1, one, q, 0, one, c.plan, T, k, buf[:4 * E * d * F].view(F32).view(E, d, F)))):
        with pytest.raises(sq.Fp8Error, match="overlaps") as err:
            call()
        assert err.value.code == sq.ERR_INVALID_ARG and all(n in str(err.value) for n in names), str(err.value)
    torch.cuda.synchronize()
    assert not bool(buf.any())
