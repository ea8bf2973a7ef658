"""Each form of the experts' products by the kernel that runs it: beside a wait that runs out, right behind the plan of
another routing, with every activation and both formats of the weights (bounds: _ffn_ref.py)."""
import os
import re
import tempfile
import warnings

import pytest
import torch

import scaled_quantize_gemm_gb300 as sq
from _experts_ref import make_plan, place, routing
from _ffn_ref import (ELEM, GELU, GELU_TANH, NONE, RELU, SILU, U, act64, assert_amax, assert_codes, assert_within, gated, new_state, product, randn, to_codes,
                      values)
from test_gpu_experts import BF, DEV, F32, H, U8, Case

pytestmark = pytest.mark.gpu

ROWS, SINGLE, PAIRS = "rows", "one CTA a tile", "pairs"
# form: (tokens, top_k, experts, hidden, inner): K split over all SMs, with the weights sent for ahead of the wait and
# (short K) without; one CTA a tile; CTA pairs
GATED = {"few": (4, 1, 4, 4096, 1024), "few, short": (4, 1, 4, 1056, 1040), "single": (30, 4, 24, 1056, 1040), "pairs": (2000, 2, 5, 1056, 528)}
KERNEL = {"few": ROWS, "few, short": ROWS, "single": SINGLE, "pairs": PAIRS, "backward": PAIRS, "weights": PAIRS}


def kernels(call):
    """The products' kernels that a call launches, by the names in a captured graph (nothing runs)."""
    sq.fp8_device_status(False)                  # (loads the library's device code, which a capture must not)
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    graph.enable_debug_mode()
    with torch.cuda.graph(graph):
        call()
    with tempfile.TemporaryDirectory() as d:
        path = os.path.join(d, "graph.dot")
        with warnings.catch_warnings():          # (it warns that it dumps)
            warnings.simplefilter("ignore")
            graph.debug_dump(path)
        text = open(path).read()
    found = set()
    for name, mangled, plain in re.findall(r"k_ffn_(pair|rows)(?:I((?:L[ib]\d+E)+)E|<([^>]*)>)", text):
        last = re.findall(r"\d+|true|false", mangled or plain)[-1]
        found.add(ROWS if name == "rows" else PAIRS if last in ("1", "true") else SINGLE)
    return found


class Forms:
    """The operands of one form and its call: call(plan, outputs)."""

    def __init__(self, how, seed):
        self.how = how
        T, k, E, d, F = GATED[how] if how in GATED else GATED["pairs"]
        c = self.c = Case(T, k, E, "spread", seed=seed)
        A, sa = to_codes(randn(c.g, c.R, d), 0)
        if how in GATED:
            W, sw = c.weights(2 * F, d)
            self.ws = c.workspace(2 * F, d)
            self.st = new_state(H, 20.0)
            self.shapes = ((c.R, 2 * F, BF), (c.R, F, BF), (c.R, F, U8))
            self.run = lambda p, o, s: sq.fp8_expert_glu_fwd(A, 0, sa, W, 0, sw, SILU, p, T, k, gu_out=o[0], h_out=o[1], q_out=o[2], q_state=self.st,
                                                             history_len=H, workspace=self.ws, stream=s)
        elif how == "backward":
            Wd, sw = c.weights(d, F)
            gu = randn(c.g, c.R, 2 * F).to(BF)
            self.ws, self.st = None, new_state(H, 300.0)
            self.shapes = ((c.R, 2 * F, U8),)
            self.run = lambda p, o, s: sq.fp8_expert_glu_bwd(A, 0, sa, Wd, 0, sw, gu, SILU, p, T, k, o[0], sq.E5M2, self.st, H, stream=s)
        else:
            B, sb = to_codes(randn(c.g, c.R, F), 0)
            self.ws = None
            self.shapes = ((E, d, F, F32),)
            self.run = lambda p, o, s: sq.fp8_expert_wgrad(A, 0, sa, B, 0, sb, p, T, k, o[0], stream=s)

    def outs(self):
        return [torch.zeros(s[:-1], dtype=s[-1], device=DEV) for s in self.shapes]

    def __call__(self, plan, outs, stream=None):
        self.run(plan, outs, stream)


def _same(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("how", KERNEL)
def test_the_kernel_of_each_form(how):
    f = Forms(how, 1)
    assert kernels(lambda: f(f.c.plan, f.outs())) == {KERNEL[how]}
    assert (f.ws is not None) == (KERNEL[how] == ROWS)


@pytest.mark.parametrize("how", [*GATED, "backward"])
def test_a_word_set_while_gated_products_start(how):
    f = Forms(how, 2)
    plan, want, got = f.c.plan, f.outs(), f.outs()
    assert sq.fp8_device_status(True) == sq.OK
    f(plan, want)
    f(plan, got)
    waited = torch.zeros(1, dtype=torch.int32, device=DEV)
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(24):
        # the wait runs out at a moment of its own among the products
        sq.fp8_selftest_wait_timeout(20 + 17 * i, waited, stream=two)
        for _ in range(30):
            f(plan, got, one)
        torch.cuda.synchronize()
        assert sq.fp8_device_status(True) == sq.ERR_TIMEOUT
        if f.ws is not None:
            f.ws.zero_()
        f(plan, got)
        torch.cuda.synchronize()
        assert _same(got, want) and sq.fp8_device_status(True) == sq.OK


# one plan buffer for one routing after another, the product right behind the sort: what its CTAs fetch before their
# wait (the gated forms the gate's and the up projection's rows) follows the routing before
@pytest.mark.parametrize("how", KERNEL)
def test_products_right_behind_the_plan_of_another_routing(how):
    f = Forms(how, 3)
    c = f.c
    ways = [routing(c.g, c.T, c.k, c.E, h) for h in ("spread", "last", "none", "masked", "one", "skewed", "spread", "masked")]
    want = []
    for ids in ways:
        want.append(f.outs())
        p = make_plan(ids, c.E)
        torch.cuda.synchronize()
        f(p, want[-1])
        torch.cuda.synchronize()
    got, plan = [f.outs() for _ in ways], torch.zeros_like(c.plan)

    def chain():
        for ids, o in zip(ways, got):
            sq.fp8_expert_plan(ids, c.E, plan)
            f(plan, o)
    chain()
    assert all(_same(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for _ in range(5):
        for o in got:
            for t in o:
                t.zero_()
        graph.replay()
        assert all(_same(a, b) for a, b in zip(got, want))
    assert sq.fp8_device_status(True) == sq.OK


@pytest.mark.parametrize("T", [3, 40, 700])
def test_rows_moved_right_behind_what_writes_them(T):
    """The same buffers one call after another: norm, dispatch and combination each start under the kernel before."""
    k, E, K = 2, 6, 512
    c = Case(T, k, E, "masked", seed=T)
    xs = [randn(c.g, T, K).to(BF) for _ in range(6)]
    ways = [routing(c.g, T, k, E, h) for h in ("spread", "masked", "one", "last", "skewed", "spread")]
    gamma, w = torch.ones(K, device=DEV), torch.rand((T, k), generator=c.g, device=DEV)
    bufs = lambda: (torch.empty((T, K), dtype=BF, device=DEV), torch.zeros((c.R, K), dtype=BF, device=DEV), torch.zeros_like(c.plan))     # noqa: E731

    def call(x, ids, n, rows, plan, y):
        sq.fp8_rmsnorm_fwd(x, gamma, 1e-5, n)
        sq.fp8_expert_plan(ids, E, plan)
        sq.fp8_expert_dispatch(n, plan, k, E, rows)
        sq.fp8_rmsnorm_fwd(y, gamma, 1e-5, n)             # (what the dispatch reads, written again)
        sq.fp8_expert_combine(rows, plan, k, E, y, weights=w, residual=n)
        sq.fp8_expert_dispatch(y, plan, k, E, rows)
        sq.fp8_expert_combine(rows, plan, k, E, n, weights=w)
        return n

    def run(shared):
        outs, held = [], bufs()
        for x, ids in zip(xs, ways):
            n, rows, plan = held if shared else bufs()
            y = x.clone()
            if not shared:
                torch.cuda.synchronize()
            outs.append((call(x, ids, n, rows, plan, y).clone(), y))
        torch.cuda.synchronize()
        return outs
    want = run(False)
    assert all(bool(torch.isfinite(v).all()) for o in want for v in o)
    for _ in range(5):
        assert all(_same(a, b) for a, b in zip(run(True), want))


SMALL = [(7, 2, 3, "masked", 160, 144), (64, 8, 24, "spread", 1056, 272), (333, 4, 7, "masked", 256, 320), (1200, 2, 3, "spread", 544, 400)]


@pytest.mark.parametrize("fa,fw", [(0, 0), (0, 1), (1, 1)])
@pytest.mark.parametrize("act", [NONE, RELU, GELU, GELU_TANH, SILU])
@pytest.mark.parametrize("T,k,E,how,d,F", SMALL)
def test_gated_forms_of_every_activation_and_format(T, k, E, how, d, F, act, fa, fw):
    c = Case(T, k, E, how, seed=4)
    A, sa = c.rows(d, fa)
    W, sw = c.weights(2 * F, d, fw)
    gu, h, q, st = c.empty(c.R, 2 * F, dtype=BF), c.empty(c.R, F, dtype=BF), c.empty(c.R, F, dtype=U8), new_state(H, 20.0, 0.125)
    sq.fp8_expert_glu_fwd(A, fa, sa, W, fw, sw, act, c.plan, T, k, gu_out=gu, h_out=h, q_out=q, q_state=st, history_len=H, workspace=c.workspace(2 * F, d))
    dY, sd = c.rows(d, fa)
    Wd, swd = c.weights(d, F, fw)
    kept = place(c.row, randn(c.g, T, k, 2 * F).to(BF), c.R)
    dq, dst = c.empty(c.R, 2 * F, dtype=U8), new_state(H, 300.0, 0.125)
    sq.fp8_expert_glu_bwd(dY, fa, sd, Wd, fw, swd, kept, act, c.plan, T, k, dq, sq.E5M2, dst, H)
    none = torch.zeros((0, F), dtype=torch.float64, device=DEV)
    want, err, dwant, derr = [none], [none], [none.repeat(1, 2)], [none.repeat(1, 2)]
    for e, r in c.experts():
        z, ez = product(values(A[r], fa), values(W[e], fw), float(sa) * float(sw[e]))
        assert_within(gu[r], z, ez, f"expert {e} g, u")
        y, ey = gated(z[:, :F], ez[:, :F], z[:, F:], ez[:, F:], act)
        assert_within(h[r], y, ey, f"expert {e} h")
        assert_codes(q[r], y, ey, 20.0, 0, f"expert {e}")
        want.append(y)
        err.append(ey)
        dh, eh = product(values(dY[r], fa), values(Wd[e], fw).T, float(sd) * float(swd[e]))
        g, u = kept[r, :F].double(), kept[r, F:].double()
        f, df = act64(g, act)
        v = torch.cat([dh * u * df, dh * f], 1)
        # derivative and value of the activation: ELEM of what enters them
        ed = ELEM * (1 + g.abs())
        ev = torch.cat([eh * (u * df).abs() + dh.abs() * u.abs() * ed, eh * f.abs() + dh.abs() * ELEM * g.abs()], 1)
        ev = ev + 4 * U * v.abs() + torch.cat([eh * u.abs() * ed, eh * ELEM * g.abs()], 1)
        assert_codes(dq[r], v, ev, 300.0, 1, f"expert {e} backward")
        dwant.append(v)
        derr.append(ev)
    assert_amax(st, 0.125, torch.cat(want), torch.cat(err))
    assert_amax(dst, 0.125, torch.cat(dwant), torch.cat(derr))
    c.untouched(gu, h, q, dq)
    assert sq.fp8_device_status(True) == sq.OK


@pytest.mark.parametrize("fa,fb", [(0, 1), (1, 1)])
@pytest.mark.parametrize("T,k,E,how,d,F", SMALL)
def test_products_of_e5m2_weights(T, k, E, how, d, F, fa, fb):
    c = Case(T, k, E, how, seed=5)
    A, sa = c.rows(d, fa)
    B, sb = c.weights(F, d, fb)
    Bt, sbt = c.weights(d, F, fb)
    X, sx = c.rows(F, fb)
    D, Dt, dW = c.empty(c.R, F, dtype=F32), c.empty(c.R, F, dtype=F32), c.empty(E, d, F, dtype=F32)
    sq.fp8_expert_gemm(A, fa, sa, B, fb, sb, sq.K_MAJOR, c.plan, T, k, D, workspace=c.workspace(F, d))
    sq.fp8_expert_gemm(A, fa, sa, Bt, fb, sbt, sq.MN_MAJOR, c.plan, T, k, Dt)
    sq.fp8_expert_wgrad(A, fa, sa, X, fb, sx, c.plan, T, k, dW)
    for e, r in c.experts():
        z, ez = product(values(A[r], fa), values(B[e], fb), float(sa) * float(sb[e]))
        assert_within(D[r], z, ez, f"expert {e}")
        z, ez = product(values(A[r], fa), values(Bt[e], fb).T, float(sa) * float(sbt[e]))
        assert_within(Dt[r], z, ez, f"expert {e} MN-major")
        z, ez = product(values(A[r], fa).T.contiguous(), values(X[r], fb).T.contiguous(), float(sa) * float(sx))
        assert_within(dW[e], z, ez, f"expert {e} weights' gradient")
    c.untouched(D, Dt)
    assert sq.fp8_device_status(True) == sq.OK
