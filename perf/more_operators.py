"""The operators of a mixture-of-experts feed-forward sublayer on the FP8 path: RMSNorm with the residual's addition and
an output in FP8, tokens sorted by expert and back with their gradients, and the experts' products.  `own` selects the
framework's calls; otherwise `run` computes the same in elementary torch operations."""
import math

import torch

own = False

H = 16                      # amax history of the delayed-scaling states
EPS = 1e-5
PAD = 32                    # an expert's rows start and end on multiples of it
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one token's residual stream in front of a block, cast with the scale of the last steps: latency
        {"name": "rms_token", "op": "rms_fwd", "rows": 1, "cols": 4096, "dtype": "bf16", "residual": True,
         "out": "codes"},
        # a training step's tokens, in tiles of 128 values for a fine-grained linear
        {"name": "rms_train", "op": "rms_fwd", "rows": 16384, "cols": 4096, "dtype": "bf16", "residual": True,
         "out": "tiles"},
        # its backward pass, the residual branch's gradient added to dx
        {"name": "rms_bwd_train", "op": "rms_bwd", "rows": 16384, "cols": 4096, "dtype": "bf16", "dres": True},
        # fp32 master activations, odd sizes: rows that start on no vector boundary
        {"name": "rms_bwd_odd", "op": "rms_bwd", "rows": 2051, "cols": 1535, "dtype": "f32", "dres": False},
        # serving: a batch of tokens' codes to their experts
        {"name": "dispatch_batch", "op": "dispatch", "tokens": 64, "top_k": 8, "experts": 64, "hidden": 4096,
         "dtype": "codes", "masked": False},
        # a training step's codes to their experts; padded tokens go to none
        {"name": "dispatch_train", "op": "dispatch", "tokens": 16384, "top_k": 4, "experts": 16, "hidden": 4096,
         "dtype": "codes", "masked": True},
        # serving: the experts' outputs back into the residual stream
        {"name": "combine_batch", "op": "combine", "tokens": 40, "top_k": 6, "experts": 48, "hidden": 2304,
         "dtype": "bf16", "residual": True, "masked": False},
        # training: the outputs' gradient cast for the experts' products, and that of the routing weights
        {"name": "combine_bwd_train", "op": "combine_bwd", "tokens": 8192, "top_k": 4, "experts": 16, "hidden": 4096,
         "masked": True},
        # serving: one token through the weights of its eight experts
        {"name": "experts_token", "op": "experts_fwd", "tokens": 1, "top_k": 8, "experts": 64, "hidden": 4096,
         "inner": 1792, "act": "silu", "save": False, "masked": False},
        # a small batch, a few rows to an expert, over a ragged inner size
        {"name": "experts_batch", "op": "experts_fwd", "tokens": 192, "top_k": 4, "experts": 32, "hidden": 2304,
         "inner": 1040, "act": "gelu_tanh", "save": False, "masked": False},
        # a training step's forward pass, gate and up values kept
        {"name": "experts_train", "op": "experts_fwd", "tokens": 8192, "top_k": 4, "experts": 16, "hidden": 4096,
         "inner": 3584, "act": "silu", "save": True, "masked": True},
        # and its backward pass: the rows' gradient and both weight gradients
        {"name": "experts_bwd_train", "op": "experts_bwd", "tokens": 4096, "top_k": 4, "experts": 16, "hidden": 4096,
         "inner": 3584, "act": "silu", "masked": True},
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(rng, m, lo, hi):
    return m * _logint(rng, lo // m, hi // m)


def draw(rng):
    op = rng.choice(["rms_fwd", "rms_fwd", "rms_bwd", "dispatch", "combine", "combine_bwd", "experts_fwd",
                     "experts_fwd", "experts_bwd"])
    yes = lambda: rng.random() < 0.5                                                                # noqa: E731
    if op in ("rms_fwd", "rms_bwd"):
        out = rng.choice(["y", "codes", "tiles"]) if op == "rms_fwd" else None
        cols = (_mult(rng, 128, 128, 12288) if out == "tiles" else
                _logint(rng, 100, 12000) if yes() else _mult(rng, 16, 128, 12288))
        c = {"op": op, "rows": _logint(rng, 1, min(16384, (1 << 26) // cols)), "cols": cols,
             "dtype": rng.choice(["bf16", "f32"])}
        return {**c, "residual": yes(), "out": out} if out else {**c, "dres": yes()}
    experts = _logint(rng, 2, 96)
    top_k = rng.randint(1, min(8, experts))
    c = {"op": op, "tokens": _logint(rng, 1, 32768 // top_k), "top_k": top_k, "experts": experts}
    if op in ("dispatch", "combine", "combine_bwd"):
        c["hidden"] = _mult(rng, 16, 128, 4096) if op == "combine_bwd" or yes() else _logint(rng, 100, 4096)
        if op == "dispatch":
            c["dtype"] = rng.choice(["codes", "bf16", "f32"])
        if op == "combine":
            c["dtype"], c["residual"] = rng.choice(["bf16", "f32"]), yes()
        return {**c, "masked": yes()}
    c["hidden"] = _mult(rng, 32, 256, 4096)
    c["inner"] = _mult(rng, 16, 256, 3584)
    while c["experts"] * c["hidden"] * c["inner"] > 235e6 and c["inner"] > 256:      # the largest listed one's weights
        c["inner"] = c["inner"] // 32 * 16
    if op == "experts_bwd":
        c["tokens"] = max(1, c["tokens"] // 2)
        return {**c, "act": rng.choice(["silu", "gelu", "gelu_tanh"]), "masked": yes()}
    return {**c, "act": rng.choice(["relu", "gelu", "gelu_tanh", "silu"]), "save": yes(), "masked": yes()}


# ---------------------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _codes(x, fmt):
    """An operand as a user holds it: FP8 codes and the scale that turns them back, from the tensor's maximum."""
    s = max(float(x.abs().max()), 1e-30) / FMAX[fmt]
    q = (x * (1.0 / s)).clamp_(-FMAX[fmt], FMAX[fmt]).to(F8[fmt])
    return q.view(torch.uint8), torch.full((1,), s, device="cuda")


def _state(fmt, amax):
    """A delayed-scaling state whose history says `amax`: [history, m, s]."""
    st = torch.zeros(H + 2, device="cuda")
    st[1] = amax
    st[H], st[H + 1] = FMAX[fmt] / amax, amax / FMAX[fmt]
    return st


def _acts(g, rows, cols):
    """What leaves a normalisation: unit rows, a few channels much larger than the others."""
    x = _randn(g, rows, cols)
    x[:, :: max(1, cols // 7)] *= 6.0
    return x


def _stream(g, rows, cols, dtype):
    """A residual stream: rows of their own spread, a few large channels."""
    x = _acts(g, rows, cols)
    x *= 0.5 + 1.5 * torch.rand((rows, 1), generator=g, device="cuda")
    return x.to(dtype)


def _weights(g, experts, n, k):
    """Codes [E][n][k] of the experts' weights, each with its own scale."""
    q, s = torch.empty((experts, n, k), device="cuda", dtype=torch.uint8), torch.empty(experts, device="cuda")
    for e in range(experts):
        q[e], s[e:e + 1] = _codes(_randn(g, n, k) * k ** -0.5, "e4m3")
    return q, s


def _route(g, c):
    """A router's choice: the experts of every token (some more wanted than others) and their weights.  Masked: a few
    tokens are padding and go to no expert."""
    T, E, k = c["tokens"], c["experts"], c["top_k"]
    v, ids = (_randn(g, T, E) + 0.6 * _randn(g, 1, E)).topk(k, 1)
    ids = ids.int()
    if c["masked"]:
        ids[torch.rand(T, generator=g, device="cuda") < 0.03] = -1
    return ids.contiguous(), torch.softmax(v, 1).contiguous()


def rows_of(c):
    """Rows that the sorted buffers are made for: every assignment, and what fills the last PAD rows of each expert."""
    n = c["tokens"] * c["top_k"]
    return (n + (PAD - 1) * min(c["experts"], n)) // PAD * PAD


def _sort(ids, E, R):
    """(offsets [E + 1], counts [E], row of each assignment or -1): the assignments of an expert in the order of tokens,
    its rows padded to a multiple of PAD."""
    flat = ids.reshape(-1).long()
    e = torch.where((flat >= 0) & (flat < E), flat, E)
    counts = torch.zeros(E + 1, dtype=torch.long, device=e.device).scatter_add_(0, e, torch.ones_like(e))
    offsets = torch.zeros(E + 1, dtype=torch.long, device=e.device)
    offsets[1:] = ((counts[:E] + PAD - 1) // PAD * PAD).cumsum(0)
    order = torch.argsort(e, stable=True)
    start = counts.cumsum(0) - counts
    es = e[order]
    rank = torch.arange(e.numel(), device=e.device) - start[es]
    row = torch.empty_like(e)
    row[order] = torch.where(es < E, offsets[es] + rank, -1)
    return offsets.int(), counts[:E].int(), row.reshape(ids.shape).int()


def _place(rows, row_of, values):
    """rows[row_of[t, j]] = values[t] (or values[t, j]); rows has one more, which takes what goes nowhere."""
    for j in range(row_of.shape[1]):
        at = row_of[:, j].long()
        rows[torch.where(at >= 0, at, rows.shape[0] - 1)] = values[:, j] if values.dim() == 3 else values
    return rows[:-1]


def prepare(case, seed):
    g, c, op = _gen(seed), case, case["op"]
    e = torch.empty
    z = torch.zeros
    st = {"case": c, "ws": {}}
    if op in ("rms_fwd", "rms_bwd"):
        R, K, dt = c["rows"], c["cols"], DT[c["dtype"]]
        st["x"] = _stream(g, R, K, dt)
        st["gamma"] = 0.5 + torch.rand(K, generator=g, device="cuda")
        if op == "rms_fwd":
            st["res"] = _randn(g, R, K).to(dt) if c["residual"] else None
            st["sum"] = e((R, K), device="cuda", dtype=dt) if c["residual"] else None
            st["y"] = e((R, K), device="cuda", dtype=dt) if c["out"] == "y" else None
            st["rstd"] = e(R, device="cuda")
            st["q"] = e((R, K), device="cuda", dtype=torch.uint8) if c["out"] != "y" else None
            st["state"] = _state("e4m3", 30.0) if c["out"] == "codes" else None
            st["scales"] = e((R, K // 128), device="cuda") if c["out"] == "tiles" else None
        else:
            st["dy"] = (1e-3 * _acts(g, R, K)).to(dt)
            st["dres"] = (1e-3 * _randn(g, R, K)).to(dt) if c["dres"] else None
            st["rstd"] = (st["x"].float().square().mean(1) + EPS).rsqrt()
            st["dx"], st["dgamma"] = e((R, K), device="cuda", dtype=dt), e(K, device="cuda")
        return st
    T, E, k, d, R = c["tokens"], c["experts"], c["top_k"], c["hidden"], rows_of(c)
    st["ids"], st["w"] = _route(g, c)
    st["offsets"], st["counts"], st["row_of"] = _sort(st["ids"], E, R)
    if op == "dispatch":
        st["x"] = _codes(_acts(g, T, d), "e4m3")[0] if c["dtype"] == "codes" else _acts(g, T, d).to(DT[c["dtype"]])
        st["rows"] = z((R, d), device="cuda", dtype=st["x"].dtype)
    elif op == "combine":
        dt = DT[c["dtype"]]
        st["rows"] = (0.5 * _acts(g, R, d)).to(dt)
        st["res"] = _stream(g, T, d, dt) if c["residual"] else None
        st["y"] = e((T, d), device="cuda", dtype=dt)
    elif op == "combine_bwd":
        st["rows"] = (0.5 * _acts(g, R, d)).to(torch.bfloat16)
        st["dy"] = (1e-3 * _acts(g, T, d)).to(torch.bfloat16)
        st["q"], st["state"] = z((R, d), device="cuda", dtype=torch.uint8), _state("e5m2", 0.03)
        st["dw"] = e((T, k), device="cuda")
    else:
        F = c["inner"]
        st["segments"] = st["offsets"].tolist()
        x, st["sx"] = _codes(_acts(g, T, d), "e4m3")
        st["x"] = _place(z((R + 1, d), device="cuda", dtype=torch.uint8), st["row_of"], x)
        st["wd"], st["swd"] = _weights(g, E, d, F)
        st["wgu"], st["swgu"] = _weights(g, E, 2 * F, d)
        if op == "experts_fwd":
            st["h"], st["state"] = z((R, F), device="cuda", dtype=torch.uint8), _state("e4m3", 24.0)
            st["gu"] = z((R, 2 * F), device="cuda", dtype=torch.bfloat16) if c["save"] else None
            st["y"] = z((R, d), device="cuda", dtype=torch.bfloat16)
        else:
            # rows that fill up an expert's segment are zero in every buffer, as the forward pass left them
            dy, st["sdy"] = _codes(1e-3 * _acts(g, T, d), "e5m2")
            gu = (1.3 * _randn(g, T, k, 2 * F)).to(torch.bfloat16)
            h, st["sh"] = _codes(_act(gu[..., :F].float(), c["act"]) * gu[..., F:].float(), "e4m3")
            st["dy"] = _place(z((R + 1, d), device="cuda", dtype=torch.uint8), st["row_of"], dy)
            st["gu"] = _place(z((R + 1, 2 * F), device="cuda", dtype=torch.bfloat16), st["row_of"], gu)
            st["h"] = _place(z((R + 1, F), device="cuda", dtype=torch.uint8), st["row_of"], h)
            del gu, h
            st["q"], st["state"] = z((R, 2 * F), device="cuda", dtype=torch.uint8), _state("e5m2", 0.05)
            st["dx"] = z((R, d), device="cuda", dtype=torch.bfloat16)
            st["dw"] = e((E, 2 * F, d), device="cuda", dtype=torch.bfloat16)
            st["dwd"] = e((E, d, F), device="cuda", dtype=torch.bfloat16)
    return st


def _workspace(state, name, nbytes):
    """The scratch a user's program keeps for these sizes: zeroed once, then left to the library."""
    ws = state["ws"].get(name)
    if ws is None:
        ws = state["ws"][name] = torch.zeros(max(1, nbytes), dtype=torch.uint8, device="cuda")
    return ws


def _plan(state):
    """The plan of the routing, which a program makes once and gives to all of a sublayer's calls."""
    import scaled_quantize_gemm_gb300 as sq

    c = state["case"]
    p = state.get("plan")
    if p is None:
        p = state["plan"] = torch.empty(sq.fp8_expert_plan_ints(c["tokens"], c["top_k"], c["experts"]),
                                        dtype=torch.int32, device="cuda")
        sq.fp8_expert_plan(state["ids"], c["experts"], p)
    return p


# ---------------------------------------------------------------------------------------------------- one pass
def _act(x, act):
    if act == "relu":
        return torch.where(x > 0, x, torch.zeros_like(x))
    if act == "silu":
        return x / (1 + torch.exp(-x))
    if act == "gelu":
        return 0.5 * x * (1 + torch.erf(x * 0.5 ** 0.5))
    return 0.5 * x * (1 + torch.tanh((2 / math.pi) ** 0.5 * (x + 0.044715 * x * x * x)))


def _dact(x, act):
    if act == "relu":
        return (x > 0).to(x.dtype)
    if act == "silu":
        s = 1 / (1 + torch.exp(-x))
        return s * (1 + x * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(x * 0.5 ** 0.5)) + x * torch.exp(-0.5 * x * x) * (2 * math.pi) ** -0.5
    a = (2 / math.pi) ** 0.5
    t = torch.tanh(a * (x + 0.044715 * x * x * x))
    return 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * a * (1 + 3 * 0.044715 * x * x)


def _values(q, fmt):
    return q.view(F8[fmt]).float()


def _cast(x, fmt, state):
    """Codes (as FP8 values) under a delayed state, and the newest amax."""
    q = (x * state[H]).clamp(-FMAX[fmt], FMAX[fmt]).to(F8[fmt])
    return q, torch.maximum(state[:1], x.abs().amax().reshape(1))


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import scaled_quantize_gemm_gb300 as sq

    c = s["case"]
    op = c["op"]
    acts = {"relu": sq.ACT_RELU, "gelu": sq.ACT_GELU, "gelu_tanh": sq.ACT_GELU_TANH, "silu": sq.ACT_SILU}
    if op == "rms_fwd":
        sq.fp8_rmsnorm_fwd(s["x"], s["gamma"], EPS, s["y"], rstd=s["rstd"], residual=s["res"], sum_out=s["sum"],
                           q_out=s["q"], q_format=sq.E4M3, gran=sq.TILE_1x128 if c["out"] == "tiles" else sq.TENSOR,
                           q_state=s["state"], history_len=H if s["state"] is not None else 0, scales_out=s["scales"])
        out = {k: s[k] for k in ("y", "sum", "rstd", "scales") if s[k] is not None}
        if s["q"] is not None:
            out["q"] = s["q"].view(F8["e4m3"])
        if s["state"] is not None:
            out["amax"] = s["state"][:1]
        return out
    if op == "rms_bwd":
        ws = _workspace(s, "rms", sq.fp8_rmsnorm_bwd_workspace_bytes(c["rows"], c["cols"]))
        sq.fp8_rmsnorm_bwd(s["dy"], s["x"], s["gamma"], s["rstd"], s["dx"], s["dgamma"], ws, dres=s["dres"])
        return {k: s[k] for k in ("dx", "dgamma")}
    T, k, E = c["tokens"], c["top_k"], c["experts"]
    if op == "dispatch":
        p = s.get("plan")
        if p is None:
            p = s["plan"] = torch.empty(sq.fp8_expert_plan_ints(T, k, E), dtype=torch.int32, device="cuda")
        sq.fp8_expert_plan(s["ids"], E, p)
        sq.fp8_expert_dispatch(s["x"], p, k, E, s["rows"])
        offsets, counts, row_of = sq.expert_plan_views(p, T, k, E)
        rows = s["rows"].view(F8["e4m3"]) if c["dtype"] == "codes" else s["rows"]
        return {"rows": rows, "offsets": offsets, "counts": counts, "row_of": row_of}
    p = _plan(s)
    if op == "combine":
        sq.fp8_expert_combine(s["rows"], p, k, E, s["y"], weights=s["w"], residual=s["res"])
        return {"y": s["y"]}
    if op == "combine_bwd":
        sq.fp8_expert_combine_bwd(s["dy"], p, k, E, s["w"], rows=s["rows"], dweights=s["dw"], q_out=s["q"],
                                  q_format=sq.E5M2, q_state=s["state"], history_len=H)
        return {"drows": s["q"].view(F8["e5m2"]), "amax": s["state"][:1], "dw": s["dw"]}
    d, F = c["hidden"], c["inner"]
    if op == "experts_fwd":
        ws = _workspace(s, "gu", sq.fp8_expert_workspace_bytes(T, k, E, 2 * F, d))
        wd = _workspace(s, "down", sq.fp8_expert_workspace_bytes(T, k, E, d, F))
        sq.fp8_expert_glu_fwd(s["x"], sq.E4M3, s["sx"], s["wgu"], sq.E4M3, s["swgu"], acts[c["act"]], p, T, k,
                              gu_out=s["gu"], q_out=s["h"], q_format=sq.E4M3, q_state=s["state"], history_len=H,
                              workspace=ws)
        sq.fp8_expert_gemm(s["h"], sq.E4M3, s["state"][H + 1:], s["wd"], sq.E4M3, s["swd"], sq.K_MAJOR, p, T, k, s["y"],
                           workspace=wd)
        return {"h": s["h"].view(F8["e4m3"]), "amax": s["state"][:1], "y": s["y"],
                **({"gu": s["gu"]} if c["save"] else {})}
    sq.fp8_expert_glu_bwd(s["dy"], sq.E5M2, s["sdy"], s["wd"], sq.E4M3, s["swd"], s["gu"], acts[c["act"]], p, T, k,
                          s["q"], sq.E5M2, s["state"], H)
    sdz = s["state"][H + 1:]
    sq.fp8_expert_gemm(s["q"], sq.E5M2, sdz, s["wgu"], sq.E4M3, s["swgu"], sq.MN_MAJOR, p, T, k, s["dx"])
    sq.fp8_expert_wgrad(s["q"], sq.E5M2, sdz, s["x"], sq.E4M3, s["sx"], p, T, k, s["dw"])
    sq.fp8_expert_wgrad(s["dy"], sq.E5M2, s["sdy"], s["h"], sq.E4M3, s["sh"], p, T, k, s["dwd"])
    return {"dgu": s["q"].view(F8["e5m2"]), "amax": s["state"][:1], "dx": s["dx"], "dw": s["dw"], "dwd": s["dwd"]}


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "rms_fwd":
        dt = DT[c["dtype"]]
        x = s["x"].float()
        out = {}
        if c["residual"]:
            out["sum"] = (x + s["res"].float()).to(dt)
            x = out["sum"].float()
        rstd = 1 / torch.sqrt(x.square().mean(1, keepdim=True) + EPS)
        y = x * rstd * s["gamma"]
        out["rstd"] = rstd[:, 0]
        if c["out"] == "y":
            out["y"] = y.to(dt)
        elif c["out"] == "codes":
            out["q"], out["amax"] = _cast(y, "e4m3", s["state"])
        else:
            t = y.reshape(c["rows"], -1, 128)
            a = t.abs().amax(2, keepdim=True)
            fm = torch.full_like(a, FMAX["e4m3"])
            m, sc = torch.where(a > 0, fm / a, 1.0), torch.where(a > 0, a / fm, 1.0)
            out["q"] = (t * m).clamp(-FMAX["e4m3"], FMAX["e4m3"]).to(F8["e4m3"]).reshape(y.shape)
            out["scales"] = sc[..., 0]
        return out
    if op == "rms_bwd":
        x, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
        xh = x * rstd
        w = dy * s["gamma"]
        dx = rstd * (w - xh * (w * xh).mean(1, keepdim=True))
        if c["dres"]:
            dx = dx + s["dres"].float()
        # a sum over all rows, whose terms cancel: in 64 bits
        return {"dx": dx.to(DT[c["dtype"]]), "dgamma": (dy * xh).sum(0, dtype=torch.float64).float()}
    R = rows_of(c)
    if op == "dispatch":
        offsets, counts, row_of = _sort(s["ids"], c["experts"], R)
        x = s["x"]
        rows = _place(torch.zeros((R + 1, x.shape[1]), device=x.device, dtype=x.dtype), row_of, x)
        return {"rows": rows.view(F8["e4m3"]) if c["dtype"] == "codes" else rows, "offsets": offsets,
                "counts": counts, "row_of": row_of}
    if op in ("combine", "combine_bwd"):
        at = s["row_of"].long()
        live = (at >= 0)
        at = at.clamp_min(0)
        k = c["top_k"]
    if op == "combine":
        dt = DT[c["dtype"]]
        y = torch.zeros(s["y"].shape, device=at.device)
        for j in range(k):
            v = s["rows"][at[:, j]].float() * s["w"][:, j:j + 1]
            y = y + torch.where(live[:, j:j + 1], v, torch.zeros_like(v))
        if c["residual"]:
            y = y + s["res"].float()
        return {"y": y.to(dt)}
    if op == "combine_bwd":
        dy = s["dy"].float()
        q, amax = torch.zeros((R + 1, dy.shape[1]), device=dy.device, dtype=torch.uint8), s["state"][:1]
        dw = torch.zeros(s["w"].shape, device=dy.device)
        for j in range(k):
            lj = live[:, j]
            v = torch.where(lj[:, None], dy * s["w"][:, j:j + 1], torch.zeros_like(dy))
            qj, amax = _cast(v, "e5m2", torch.cat([amax, s["state"][1:]]))
            q[torch.where(lj, at[:, j], R)] = qj.view(torch.uint8)
            p = (dy * s["rows"][at[:, j]].float()).sum(1, dtype=torch.float64).float()
            dw[:, j] = torch.where(lj, p, torch.zeros_like(p))
        return {"drows": q[:-1].view(F8["e5m2"]), "amax": amax, "dw": dw}
    F, E = c["inner"], c["experts"]
    seg = [(e, slice(s["segments"][e], s["segments"][e + 1])) for e in range(E)]
    zeros = lambda *shape, dtype=torch.float32: torch.zeros(shape, device=s["x"].device, dtype=dtype)    # noqa: E731
    b = torch.bfloat16
    if op == "experts_fwd":
        hq, y, amax = zeros(R, F, dtype=torch.uint8), zeros(R, c["hidden"], dtype=b), s["state"][:1]
        gu = zeros(R, 2 * F, dtype=b) if c["save"] else None
        for e, r in seg:
            if r.start == r.stop:
                continue
            zz = (_values(s["x"][r], "e4m3") @ _values(s["wgu"][e], "e4m3").t()) * (s["sx"] * s["swgu"][e])
            q, amax = _cast(_act(zz[:, :F], c["act"]) * zz[:, F:], "e4m3", torch.cat([amax, s["state"][1:]]))
            hq[r] = q.view(torch.uint8)
            y[r] = ((q.float() @ _values(s["wd"][e], "e4m3").t()) * (s["state"][H + 1] * s["swd"][e])).to(b)
            if c["save"]:
                gu[r] = zz.to(b)
        return {"h": hq.view(F8["e4m3"]), "amax": amax, "y": y, **({"gu": gu} if c["save"] else {})}
    q, dx, amax = zeros(R, 2 * F, dtype=torch.uint8), zeros(R, c["hidden"], dtype=b), s["state"][:1]
    dw, dwd = torch.zeros_like(s["dw"]), torch.zeros_like(s["dwd"])
    sdz = s["state"][H + 1]
    for e, r in seg:
        if r.start == r.stop:
            continue
        dyv = _values(s["dy"][r], "e5m2")
        dh = (dyv @ _values(s["wd"][e], "e4m3")) * (s["sdy"] * s["swd"][e])
        gate, up = s["gu"][r, :F].float(), s["gu"][r, F:].float()
        dgu = torch.cat([dh * up * _dact(gate, c["act"]), dh * _act(gate, c["act"])], 1)
        qe, amax = _cast(dgu, "e5m2", torch.cat([amax, s["state"][1:]]))
        q[r] = qe.view(torch.uint8)
        qv = qe.float()
        dx[r] = ((qv @ _values(s["wgu"][e], "e4m3")) * (sdz * s["swgu"][e])).to(b)
        dw[e] = ((qv.t() @ _values(s["x"][r], "e4m3")) * (sdz * s["sx"])).to(b)
        dwd[e] = ((dyv.t() @ _values(s["h"][r], "e4m3")) * (s["sdy"] * s["sh"])).to(b)
    return {"dgu": q.view(F8["e5m2"]), "amax": amax, "dx": dx, "dw": dw, "dwd": dwd}


# ---------------------------------------------------------------------------------------------------- work, definition
def work(case):
    c, op = case, case["op"]
    if op in ("rms_fwd", "rms_bwd"):
        R, K = c["rows"], c["cols"]
        e = 2 if c["dtype"] == "bf16" else 4
        if op == "rms_fwd":
            o = e if c["out"] == "y" else 1 + (1 / 32 if c["out"] == "tiles" else 0)
            return {"bytes": int((3 if c["residual"] else 1) * e * R * K + o * R * K) + 4 * K + 4 * R,
                    "flops": 5 * R * K}
        return {"bytes": (4 if c["dres"] else 3) * e * R * K + 8 * K + 4 * R, "flops": 10 * R * K}
    T, k, E, d = c["tokens"], c["top_k"], c["experts"], c["hidden"]
    n = T * k
    if op == "dispatch":
        e = {"codes": 1, "bf16": 2, "f32": 4}[c["dtype"]]
        return {"bytes": e * d * (T + n) + 8 * n, "flops": 4 * n}
    if op == "combine":
        e = 2 if c["dtype"] == "bf16" else 4
        return {"bytes": e * d * (n + T * (2 if c["residual"] else 1)) + 8 * n, "flops": 2 * n * d}
    if op == "combine_bwd":
        return {"bytes": d * (2 * T + 2 * n + n) + 12 * n, "flops": 4 * n * d}
    F = c["inner"]
    used = E * (1 - (1 - k / E) ** T)               # experts that some token has chosen
    if op == "experts_fwd":
        return {"bytes": int(used * 3 * d * F) + n * (d + 2 * F + 2 * d + (4 * F if c["save"] else 0)),
                "flops": 6 * n * d * F}
    # read dy, x, h, [g | u] and both weights; write the codes of [dg | du], dx and both weight gradients
    return {"bytes": int(used * 3 * d * F) + n * (2 * d + F + 4 * F + 2 * F + 2 * d) + 6 * E * d * F,
            "flops": 12 * n * d * F}


def _act64(z, act):
    """(act(z), act'(z)) from the definitions with the normal distribution function and the logistic function."""
    if act == "relu":
        return z.clamp_min(0), torch.heaviside(z, torch.zeros_like(z))
    if act == "gelu":
        phi = torch.special.ndtr(z)
        return z * phi, phi + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    # silu: z sigma(z); the tanh form of gelu: z sigma(2 a (z + b z^3))
    a, b = ((1.0, 0.0) if act == "silu" else (2 * math.sqrt(2 / math.pi), 0.044715))
    s = torch.sigmoid(a * (z + b * z ** 3))
    return z * s, s + z * s * torch.sigmoid(-a * (z + b * z ** 3)) * a * (1 + 3 * b * z ** 2)


def _cast64(v, fmt, st):
    """Codes of 64-bit values, the FP8 numbers nearest to the scaled and clipped values, and the values' maximum."""
    q = (v * st[H].double()).clamp(-FMAX[fmt], FMAX[fmt]).float().to(F8[fmt])
    return q, v.abs().max().reshape(1)


def _where_rows(c, ids):
    """For every expert the assignments t top_k + j that chose it, in order, and the first of its rows: a walk."""
    lists = [[] for _ in range(c["experts"])]
    for i, e in enumerate(ids.reshape(-1).tolist()):
        if 0 <= e < c["experts"]:
            lists[e].append(i)
    first = [0]
    for a in lists:
        first.append(first[-1] + -(-len(a) // PAD) * PAD)
    return lists, first


def exact(case, seed):
    c, op = case, case["op"]
    s = prepare(case, seed)
    val = lambda t, fmt: t.view(F8[fmt]).double()                                                   # noqa: E731
    if op == "rms_fwd":
        x = s["x"].double()
        out = {}
        if c["residual"]:
            out["sum"] = (x + s["res"].double()).to(DT[c["dtype"]])
            x = out["sum"].double()
        rstd = (torch.einsum("rc,rc->r", x, x) / c["cols"] + EPS) ** -0.5
        out["rstd"] = rstd
        y = torch.einsum("rc,r,c->rc", x, rstd, s["gamma"].double())
        if c["out"] == "y":
            out["y"] = y
        elif c["out"] == "codes":
            out["q"], a = _cast64(y, "e4m3", s["state"])
            out["amax"] = torch.maximum(a, s["state"][:1].double())
        else:
            t = y.view(-1, 128)
            a = t.abs().max(1).values
            sc = torch.where(a > 0, a / FMAX["e4m3"], torch.ones_like(a))
            out["q"] = (t / sc[:, None]).clamp(-FMAX["e4m3"], FMAX["e4m3"]).float().to(F8["e4m3"]).view(y.shape)
            out["scales"] = sc.view(c["rows"], -1)
        return out
    if op == "rms_bwd":
        x, dy = s["x"].double(), s["dy"].double()
        rstd = s["rstd"].double()
        xh = torch.einsum("rc,r->rc", x, rstd)
        w = torch.einsum("rc,c->rc", dy, s["gamma"].double())
        dx = torch.einsum("rc,r->rc", w - xh * (torch.einsum("rc,rc->r", w, xh) / c["cols"])[:, None], rstd)
        if c["dres"]:
            dx += s["dres"].double()
        return {"dx": dx, "dgamma": torch.einsum("rc,rc->c", dy, xh)}
    T, k, E, R = c["tokens"], c["top_k"], c["experts"], rows_of(c)
    lists, first = _where_rows(c, s["ids"])
    dev = s["ids"].device
    if op in ("dispatch", "combine", "combine_bwd"):
        at = [-1] * (T * k)
        for e, a in enumerate(lists):
            for r, i in enumerate(a):
                at[i] = first[e] + r
        src = torch.tensor([i for a in lists for i in a], dtype=torch.long, device=dev)
        dst = torch.tensor(at, dtype=torch.long, device=dev)
        to = dst[src]
        tok, w = src // k, s["w"].reshape(-1)[src].double()
    if op == "dispatch":
        rows = torch.zeros_like(s["rows"])
        rows[to] = s["x"][tok]
        return {"rows": rows.view(F8["e4m3"]) if c["dtype"] == "codes" else rows,
                "offsets": torch.tensor(first, dtype=torch.int32, device=dev),
                "counts": torch.tensor([len(a) for a in lists], dtype=torch.int32, device=dev),
                "row_of": dst.int().view(T, k)}
    if op == "combine":
        y = s["res"].double() if c["residual"] else torch.zeros(s["y"].shape, dtype=torch.float64, device=dev)
        return {"y": y.index_add(0, tok, s["rows"][to].double() * w[:, None])}
    if op == "combine_bwd":
        v = s["dy"][tok].double()
        dw = torch.zeros(T * k, dtype=torch.float64, device=dev)
        dw[src] = torch.einsum("rc,rc->r", v, s["rows"][to].double())
        q = torch.zeros((R, c["hidden"]), dtype=torch.uint8, device=dev)
        amax = s["state"][:1].double()
        if len(src):
            qv, a = _cast64(v * w[:, None], "e5m2", s["state"])
            q[to] = qv.view(torch.uint8)
            amax = torch.maximum(amax, a)
        return {"drows": q.view(F8["e5m2"]), "amax": amax, "dw": dw.view(T, k)}
    F = c["inner"]
    f64 = lambda *shape: torch.zeros(shape, dtype=torch.float64, device=dev)                        # noqa: E731
    amax = s["state"][:1].double()
    step = s["state"][H + 1].double()
    if op == "experts_fwd":
        h, y = torch.zeros((R, F), dtype=torch.uint8, device=dev), f64(R, c["hidden"])
        gu = f64(R, 2 * F) if c["save"] else None
        for e, a in enumerate(lists):
            if not a:
                continue
            r = slice(first[e], first[e] + len(a))
            zz = torch.mm(val(s["x"][r], "e4m3"), val(s["wgu"][e], "e4m3").T) * (s["sx"].double() * s["swgu"][e].double())
            q, m = _cast64(_act64(zz[:, :F], c["act"])[0] * zz[:, F:], "e4m3", s["state"])
            amax = torch.maximum(amax, m)
            h[r] = q.view(torch.uint8)
            y[r] = torch.mm(q.double(), val(s["wd"][e], "e4m3").T) * (step * s["swd"][e].double())
            if c["save"]:
                gu[r] = zz
        return {"h": h.view(F8["e4m3"]), "amax": amax, "y": y, **({"gu": gu} if c["save"] else {})}
    dgu, dx = torch.zeros((R, 2 * F), dtype=torch.uint8, device=dev), f64(R, c["hidden"])
    dw, dwd = f64(*s["dw"].shape), f64(*s["dwd"].shape)
    for e, a in enumerate(lists):
        if not a:
            continue
        r = slice(first[e], first[e] + len(a))
        dy = val(s["dy"][r], "e5m2")
        dh = torch.mm(dy, val(s["wd"][e], "e4m3")) * (s["sdy"].double() * s["swd"][e].double())
        gate, up = s["gu"][r].double().split(F, 1)
        f, df = _act64(gate, c["act"])
        q, m = _cast64(torch.cat([dh * up * df, dh * f], 1), "e5m2", s["state"])
        amax = torch.maximum(amax, m)
        dgu[r] = q.view(torch.uint8)
        qd = q.double()
        dx[r] = torch.mm(qd, val(s["wgu"][e], "e4m3")) * (step * s["swgu"][e].double())
        dw[e] = torch.mm(qd.T, val(s["x"][r], "e4m3")) * (step * s["sx"].double())
        dwd[e] = torch.mm(dy.T, val(s["h"][r], "e4m3")) * (s["sdy"].double() * s["sh"].double())
    return {"dgu": dgu.view(F8["e5m2"]), "amax": amax, "dx": dx, "dw": dw, "dwd": dwd}
