"""The plan of a routing, dispatch, combine and its backward pass (bounds: _experts_ref.py)."""
import pytest
import torch

import scaled_quantize_gemm_gb300 as sq
from _experts_ref import ROUTINGS, TILE, make_plan, place, routing, walk
from _ffn_ref import U, assert_amax, assert_codes, assert_within, gen, new_state, randn

pytestmark = pytest.mark.gpu
DEV, H = "cuda", 4
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
COLS = [16, 256, 4096, 1, 7, 100, 202, 1032, 5000]


def _case(T, k, E, how, seed=1):
    g = gen(seed)
    ids = routing(g, T, k, E, how)
    row, offsets, counts = walk(ids, E)
    return g, ids, make_plan(ids, E), row.to(DEV), offsets, counts


@pytest.mark.parametrize("T,k,E,how", ROUTINGS + [(0, 3, 5, "spread"), (131072, 1, 8, "skewed"), (4097, 8, 1000, "masked")])
def test_plan(T, k, E, how):
    g, ids, plan, row, offsets, counts = _case(T, k, E, how)
    o, c, r = sq.expert_plan_views(plan, T, k, E)
    assert o.tolist() == offsets and c.tolist() == counts and torch.equal(r, row)
    R = sq.fp8_expert_rows(T, k, E)
    assert offsets[-1] <= R <= T * k + 31 * E and R % 32 == 0
    # the products' tiles: every expert's rows once, in groups of one expert
    n, at = int(plan[2 * E + 1]), (2 * E + 2 + 3) // 4 * 4
    tiles = plan[at:at + 4 * n].view(n, 4).tolist()
    seen = []
    for i, (first, ge, row0, end) in enumerate(tiles):
        e, size = ge >> 8, ge & 0xFF
        assert first <= i < first + size and tiles[first] == tiles[i] and end == offsets[e + 1]
        seen.append((e, row0 + (i - first) * TILE))
    assert seen == [(e, x) for e in range(E) for x in range(offsets[e], offsets[e + 1], TILE)]


@pytest.mark.parametrize("dtype", [U8, BF, F32])
@pytest.mark.parametrize("T,k,E,how", ROUTINGS)
def test_dispatch(T, k, E, how, dtype):
    K = COLS[(T + k) % len(COLS)]
    g, ids, plan, row, offsets, _ = _case(T, k, E, how)
    x = torch.randint(1, 255, (T, K), generator=g, device=DEV, dtype=U8) if dtype == U8 else (randn(g, T, K) + 10).to(dtype)
    R = sq.fp8_expert_rows(T, k, E)
    rows = torch.full((R, K), 0x55, dtype=dtype, device=DEV)
    sq.fp8_expert_dispatch(x, plan, k, E, rows)
    want = place(row, x, R)
    want[offsets[-1]:] = 0x55                    # behind the last segment nothing is written
    assert torch.equal(rows, want)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,k,E,how", ROUTINGS)
def test_combine(T, k, E, how, dtype):
    K = COLS[(T + E) % len(COLS)]
    g, ids, plan, row, offsets, _ = _case(T, k, E, how)
    R = sq.fp8_expert_rows(T, k, E)
    rows = randn(g, R, K).to(dtype)
    live = torch.zeros(R, dtype=torch.bool, device=DEV)
    live[row[row >= 0].long()] = True
    rows[~live] = float("nan")                   # what no slot names is never read
    w = torch.rand((T, k), generator=g, device=DEV)
    w[row < 0] = float("nan")
    res = randn(g, T, K).to(dtype)
    for weights, residual in ((w, res), (None, None), (w, None)):
        y = torch.full((T, K), 7.0, dtype=dtype, device=DEV)
        sq.fp8_expert_combine(rows, plan, k, E, y, weights=weights, residual=residual)
        want = torch.zeros((T, K), dtype=torch.float64, device=DEV)
        mag = want.clone()
        for j in range(k):
            on = row[:, j] >= 0
            v = rows[row[on, j].long()].double() * (1 if weights is None else w[on, j:j + 1].double())
            want[on] += v
            mag[on] += v.abs()
        if residual is not None:
            want, mag = want + res.double(), mag + res.double().abs()
        assert_within(y, want, (k + 2) * U * mag, "y")
    over = res.clone()
    y = torch.empty_like(res)
    sq.fp8_expert_combine(rows, plan, k, E, y, weights=w, residual=res)
    sq.fp8_expert_combine(rows, plan, k, E, over, weights=w, residual=over)
    assert torch.equal(over, y)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,k,E,how", ROUTINGS)
def test_combine_backward(T, k, E, how, dtype):
    K = COLS[(T + 2 * k) % len(COLS)]
    g, ids, plan, row, offsets, _ = _case(T, k, E, how)
    R, end = sq.fp8_expert_rows(T, k, E), offsets[-1]
    rows, dy, w = randn(g, R, K).to(dtype), randn(g, T, K).to(dtype), torch.rand((T, k), generator=g, device=DEV)
    live = torch.zeros(R, dtype=torch.bool, device=DEV)
    live[row[row >= 0].long()] = True
    rows[~live] = float("nan")
    w[row < 0] = float("nan")
    dw = torch.full((T, k), 7.0, device=DEV)
    drows, q = torch.full((R, K), 7.0, dtype=dtype, device=DEV), torch.full((R, K), 0x55, dtype=U8, device=DEV)
    st = new_state(H, 3000.0, 0.125)
    sq.fp8_expert_combine_bwd(dy, plan, k, E, w, rows=rows, dweights=dw, drows=drows, q_out=q, q_format=sq.E5M2, q_state=st,
                              history_len=H)
    v = dy.double()[:, None, :] * torch.where(row >= 0, w, 0.0).double()[:, :, None]
    want = place(row, v, R)
    assert_within(drows[:end], want[:end], 2 * U * want[:end].abs(), "drows")
    assert_codes(q[:end], want[:end], 2 * U * want[:end].abs(), 3000.0, sq.E5M2, "codes")
    assert_amax(st, 0.125, want, 2 * U * want.abs())
    assert bool((drows[end:] == 7).all()) and bool((q[end:] == 0x55).all())
    on = row >= 0
    t = torch.arange(T, device=DEV)[:, None].expand(T, k)[on]
    p = dy[t].double() * rows[row[on].long()].double()
    assert_within(dw[on], p.sum(1), (K + 4) * U * p.abs().sum(1), "dweights")
    assert not bool(dw[~on].any())
    # each output alone, the same bits
    dw2, drows2, q2, st2 = torch.empty_like(dw), torch.empty_like(drows), torch.empty_like(q), new_state(H, 3000.0, 0.125)
    sq.fp8_expert_combine_bwd(dy, plan, k, E, w, rows=rows, dweights=dw2)
    sq.fp8_expert_combine_bwd(dy, plan, k, E, w, drows=drows2)
    sq.fp8_expert_combine_bwd(dy, plan, k, E, w, q_out=q2, q_format=sq.E5M2, q_state=st2, history_len=H)
    assert torch.equal(dw, dw2) and torch.equal(drows[:end], drows2[:end]) and torch.equal(q[:end], q2[:end])
    assert torch.equal(st, st2)


def test_no_columns():
    g, ids, plan, row, _, _ = _case(5, 2, 3, "spread")
    dw, e = torch.full((5, 2), 7.0, device=DEV), lambda n: torch.empty((n, 0), device=DEV)        # noqa: E731
    sq.fp8_expert_combine_bwd(e(5), plan, 2, 3, torch.ones((5, 2), device=DEV), rows=e(sq.fp8_expert_rows(5, 2, 3)), dweights=dw)
    sq.fp8_expert_combine(e(sq.fp8_expert_rows(5, 2, 3)), plan, 2, 3, e(5))
    sq.fp8_expert_dispatch(e(5), plan, 2, 3, e(sq.fp8_expert_rows(5, 2, 3)))
    torch.cuda.synchronize()
    assert not bool(dw.any())


def test_gradients_against_differences():
    """combine is linear in its rows and in its weights, so differences give its gradients exactly in 64 bits: of
    sum(c y) with respect to a row's element and to a weight; and dispatch's gradient is combine without weights."""
    T, k, E, K = 6, 2, 3, 20
    g, ids, plan, row, offsets, _ = _case(T, k, E, "masked", seed=4)
    R = sq.fp8_expert_rows(T, k, E)
    c, w, x = randn(g, T, K), torch.rand((T, k), generator=g, device=DEV), randn(g, T, K)
    rows = torch.zeros((R, K), device=DEV)
    sq.fp8_expert_dispatch(x, plan, k, E, rows)
    drows, dw, dx, y = torch.zeros_like(rows), torch.empty_like(w), torch.empty_like(x), torch.empty_like(x)
    sq.fp8_expert_combine_bwd(c, plan, k, E, w, rows=rows, dweights=dw, drows=drows)
    sq.fp8_expert_combine(drows, plan, k, E, dx)

    def f(x_, w_):
        out = torch.zeros((T, K), dtype=torch.float64, device=DEV)
        for j in range(k):
            on = row[:, j] >= 0
            out[on] += x_.double()[on] * w_.double()[on, j:j + 1]
        return float((c.double() * out).sum())
    for i in range(T * K):
        e = torch.zeros(T * K, dtype=torch.float64, device=DEV)
        e[i] = 0.5
        assert abs(f(x.double() + e.view(T, K), w) - f(x.double() - e.view(T, K), w) - float(dx.reshape(-1)[i])) <= 1e-5
    for i in range(T * k):
        e = torch.zeros(T * k, dtype=torch.float64, device=DEV)
        e[i] = 0.5
        assert abs(f(x, w.double() + e.view(T, k)) - f(x, w.double() - e.view(T, k)) - float(dw.reshape(-1)[i])) <= 1e-4


def test_a_captured_plan_follows_its_routing():
    T, k, E, K = 200, 4, 9, 320
    g = gen(3)
    ids = routing(g, T, k, E, "spread")
    x, rows, y = randn(g, T, K), torch.zeros((sq.fp8_expert_rows(T, k, E), K), device=DEV), torch.empty((T, K), device=DEV)
    plan = make_plan(ids, E)

    def call():
        sq.fp8_expert_plan(ids, E, plan)
        sq.fp8_expert_dispatch(x, plan, k, E, rows)
        sq.fp8_expert_combine(rows, plan, k, E, y)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for how in ("masked", "one", "none", "skewed"):
        ids.copy_(routing(g, T, k, E, how))
        graph.replay()
        torch.cuda.synchronize()
        n = ((ids >= 0) & (ids < E)).sum(1, keepdim=True)
        assert_within(y, x.double() * n, k * U * x.double().abs() * n, how)


def test_refusals():
    T, k, E, K = 4, 2, 3, 16
    plan = make_plan(torch.zeros((T, k), dtype=torch.int32, device=DEV), E)
    R = sq.fp8_expert_rows(T, k, E)
    x, rows, w = torch.zeros((T, K), device=DEV), torch.zeros((R, K), device=DEV), torch.zeros((T, k), device=DEV)
    with pytest.raises(sq.Fp8Error, match="y overlaps rows"):
        sq.fp8_expert_combine(rows, plan, k, E, rows[:T])
    with pytest.raises(sq.Fp8Error, match="out overlaps x"):
        sq.fp8_expert_dispatch(rows[:T], plan, k, E, rows)
    with pytest.raises(sq.Fp8Error, match="dweights overlaps weights"):
        sq.fp8_expert_combine_bwd(x, plan, k, E, w, rows=rows, dweights=w)
    with pytest.raises(sq.Fp8Error, match="plan overlaps ids"):
        sq.fp8_expert_plan(plan[:T * k].view(T, k), E, plan)
