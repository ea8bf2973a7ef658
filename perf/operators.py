"""The operators of a feed-forward sublayer around the FP8 linear: LayerNorm forward and backward, the gated block
(both projections, activation and product in one product) with its backward pass, and the matrix product with bias,
activation and residual in its epilogue with its backward pass.  `own` selects the framework's calls; otherwise `run`
computes the same in elementary torch operations."""
import math

import torch

own = False

H = 16                      # amax history of the delayed-scaling states
EPS = 1e-5
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one token's residual stream in front of the block: latency
        {"name": "ln_fwd_token", "op": "ln_fwd", "rows": 1, "cols": 4096, "dtype": "bf16", "residual": True},
        # a training step's tokens: the residual add and the normalisation in one pass
        {"name": "ln_fwd_train", "op": "ln_fwd", "rows": 16384, "cols": 4096, "dtype": "bf16", "residual": True},
        # its backward pass, the residual branch's gradient added to dx
        {"name": "ln_bwd_train", "op": "ln_bwd", "rows": 16384, "cols": 4096, "dtype": "bf16", "dres": True},
        # fp32 master activations, odd sizes: rows that start on no vector boundary
        {"name": "ln_bwd_odd", "op": "ln_bwd", "rows": 2051, "cols": 1535, "dtype": "f32", "dres": False},
        # serving: one token through both projections, then a small batch over a ragged inner size
        {"name": "glu_token", "op": "glu_fwd", "tokens": 1, "hidden": 4096, "inner": 14336, "act": "silu",
         "save": False},
        {"name": "glu_batch", "op": "glu_fwd", "tokens": 40, "hidden": 2304, "inner": 6160, "act": "gelu_tanh",
         "save": False},
        # the training step: codes of the product, gate and up values kept for the backward pass
        {"name": "glu_train", "op": "glu_fwd", "tokens": 16384, "hidden": 4096, "inner": 14336, "act": "silu",
         "save": True},
        {"name": "glu_bwd_train", "op": "glu_bwd", "tokens": 8192, "hidden": 4096, "inner": 14336, "act": "silu"},
        # serving: one token's projection back to the residual stream
        {"name": "act_token", "op": "act_fwd", "tokens": 1, "k": 14336, "n": 4096, "act": "none", "bias": False,
         "residual": True, "save": False, "out": "bf16"},
        # ragged fp32 outputs
        {"name": "act_ragged", "op": "act_fwd", "tokens": 777, "k": 1040, "n": 2064, "act": "gelu", "bias": True,
         "residual": True, "save": False, "out": "f32"},
        # the training step of a block with bias and GELU: z kept, the next linear's codes written
        {"name": "act_train", "op": "act_fwd", "tokens": 16384, "k": 4096, "n": 14336, "act": "gelu_tanh",
         "bias": True, "residual": False, "save": True, "out": "codes"},
        {"name": "act_bwd_train", "op": "act_bwd", "tokens": 16384, "n": 14336, "act": "gelu_tanh"},
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult16(rng, lo, hi):
    return 16 * _logint(rng, lo // 16, hi // 16)


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "glu_fwd", "glu_fwd", "glu_bwd", "act_fwd", "act_fwd", "act_bwd"])
    act = rng.choice(["relu", "gelu", "gelu_tanh", "silu"])
    yes = lambda: rng.random() < 0.5                                                                # noqa: E731
    if op in ("ln_fwd", "ln_bwd"):
        cols = _logint(rng, 100, 12000) if yes() else _mult16(rng, 128, 12288)
        c = {"op": op, "rows": _logint(rng, 1, min(16384, (1 << 26) // cols)), "cols": cols,
             "dtype": rng.choice(["bf16", "f32"])}
        return {**c, "residual": yes()} if op == "ln_fwd" else {**c, "dres": yes()}
    if op == "glu_fwd":
        return {"op": op, "tokens": _logint(rng, 1, 8192), "hidden": _mult16(rng, 256, 4096),
                "inner": _mult16(rng, 512, 14336), "act": act, "save": yes()}
    if op == "glu_bwd":
        return {"op": op, "tokens": 16 * _logint(rng, 1, 512), "hidden": _mult16(rng, 256, 4096),
                "inner": _mult16(rng, 512, 14336), "act": act}
    if op == "act_fwd":
        out = rng.choice(["bf16", "f32", "codes"])
        # the contraction over the inner size ends in the bf16 residual stream
        return {"op": op, "tokens": _logint(rng, 1, 8192), "k": _mult16(rng, 256, 14336 if out == "bf16" else 4096),
                "n": _mult16(rng, 256, 14336), "act": act if out == "codes" or yes() else "none", "bias": yes(),
                "residual": out != "codes" and yes(), "save": out == "codes", "out": out}
    return {"op": op, "tokens": _logint(rng, 1, 8192), "n": _mult16(rng, 256, 14336), "act": act}


# ---------------------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _codes(x, fmt):
    """An operand as a user holds it: FP8 codes and the scale that turns them back, from the tensor's maximum."""
    s = float(x.abs().max()) / FMAX[fmt]
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
    """A residual stream: rows of their own mean and spread, a few large channels."""
    x = _acts(g, rows, cols)
    x *= 0.5 + 1.5 * torch.rand((rows, 1), generator=g, device="cuda")
    x += 0.5 + 0.5 * _randn(g, rows, 1)
    return x.to(dtype)


def prepare(case, seed):
    g, c, op = _gen(seed), case, case["op"]
    e = torch.empty
    st = {"case": c}
    if op in ("ln_fwd", "ln_bwd"):
        R, K, dt = c["rows"], c["cols"], DT[c["dtype"]]
        st["x"] = _stream(g, R, K, dt)
        st["gamma"] = 0.5 + torch.rand(K, generator=g, device="cuda")
        if op == "ln_fwd":
            st["beta"] = 0.1 * _randn(g, K)
            st["res"] = _randn(g, R, K).to(dt) if c["residual"] else None
            st["y"], st["sum"] = e((R, K), device="cuda", dtype=dt), e((R, K), device="cuda", dtype=dt) if c["residual"] else None
            st["mu"], st["rstd"] = e(R, device="cuda"), e(R, device="cuda")
        else:
            st["dy"] = (1e-3 * _acts(g, R, K)).to(dt)
            st["dres"] = (1e-3 * _randn(g, R, K)).to(dt) if c["dres"] else None
            x = st["x"].double() if R * K < 1 << 24 else st["x"].float()
            mu = x.mean(1, keepdim=True)
            st["mu"], st["rstd"] = mu[:, 0].float(), ((x - mu).square().mean(1) + EPS).rsqrt().float()
            del x
            st["dx"] = e((R, K), device="cuda", dtype=dt)
            st["dgamma"], st["dbeta"] = e(K, device="cuda"), e(K, device="cuda")
    elif op == "glu_fwd":
        T, d, F = c["tokens"], c["hidden"], c["inner"]
        st["x"], st["sx"] = _codes(_acts(g, T, d), "e4m3")
        st["w"], st["sw"] = _codes(_randn(g, 2 * F, d) * d ** -0.5, "e4m3")
        st["q"], st["state"] = e((T, F), device="cuda", dtype=torch.uint8), _state("e4m3", 24.0)
        st["gu"] = e((T, 2 * F), device="cuda", dtype=torch.bfloat16) if c["save"] else None
    elif op == "glu_bwd":
        T, d, F = c["tokens"], c["hidden"], c["inner"]
        st["x"], st["sx"] = _codes(_acts(g, T, d), "e4m3")
        st["w"], st["sw"] = _codes(_randn(g, 2 * F, d) * d ** -0.5, "e4m3")
        st["wd"], st["swd"] = _codes(_randn(g, d, F) * F ** -0.5, "e4m3")
        st["dy"], st["sdy"] = _codes(1e-3 * _randn(g, T, d), "e5m2")
        st["gu"] = (1.3 * _randn(g, T, 2 * F)).to(torch.bfloat16)
        gf, uf = st["gu"][:, :F].float(), st["gu"][:, F:].float()
        st["h"], st["sh"] = _codes(_act(gf, c["act"]) * uf, "e4m3")
        del gf, uf
        st["q"], st["state"] = e((T, 2 * F), device="cuda", dtype=torch.uint8), _state("e5m2", 0.05)
        st["dx"] = e((T, d), device="cuda", dtype=torch.bfloat16)
        st["dw"] = e((2 * F, d), device="cuda", dtype=torch.bfloat16)
        st["dwd"] = e((d, F), device="cuda", dtype=torch.bfloat16)
    elif op == "act_fwd":
        T, K, N = c["tokens"], c["k"], c["n"]
        st["x"], st["sx"] = _codes(_acts(g, T, K), "e4m3")
        st["w"], st["sw"] = _codes(_randn(g, N, K) * K ** -0.5, "e4m3")
        st["bias"] = 0.1 * _randn(g, N) if c["bias"] else None
        dt = DT.get(c["out"])
        st["res"] = _stream(g, T, N, dt) if c["residual"] else None
        st["d"] = e((T, N), device="cuda", dtype=dt) if dt else None
        st["z"] = e((T, N), device="cuda", dtype=torch.bfloat16) if c["save"] else None
        st["q"] = e((T, N), device="cuda", dtype=torch.uint8) if c["out"] == "codes" else None
        st["state"] = _state("e4m3", 12.0) if c["out"] == "codes" else None
    else:
        T, N = c["tokens"], c["n"]
        st["dy"] = (1e-3 * _randn(g, T, N)).to(torch.bfloat16)
        st["z"] = (1.5 * _randn(g, T, N)).to(torch.bfloat16)
        st["q"], st["state"] = e((T, N), device="cuda", dtype=torch.uint8), _state("e5m2", 0.01)
        st["dbias"] = e(N, device="cuda")
    st["ws"] = {}
    return st


def _workspace(state, nbytes):
    """The scratch a user's program keeps for these sizes: zeroed once, then left to the library."""
    ws = state["ws"].get(nbytes)
    if ws is None:
        ws = state["ws"][nbytes] = torch.zeros(max(1, nbytes), dtype=torch.uint8, device="cuda")
    return ws


# ---------------------------------------------------------------------------------------------------- one pass
def _act(x, act):
    if act == "none":
        return x
    if act == "relu":
        return torch.where(x > 0, x, torch.zeros_like(x))
    if act == "silu":
        return x / (1 + torch.exp(-x))
    if act == "gelu":
        return 0.5 * x * (1 + torch.erf(x * 0.5 ** 0.5))
    return 0.5 * x * (1 + torch.tanh((2 / math.pi) ** 0.5 * (x + 0.044715 * x * x * x)))


def _dact(x, act):
    if act == "none":
        return torch.ones_like(x)
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
    acts = {"none": sq.ACT_NONE, "relu": sq.ACT_RELU, "gelu": sq.ACT_GELU, "gelu_tanh": sq.ACT_GELU_TANH, "silu": sq.ACT_SILU}
    if op == "ln_fwd":
        sq.fp8_layernorm_fwd(s["x"], s["gamma"], s["beta"], EPS, s["y"], mu=s["mu"], rstd=s["rstd"],
                             residual=s["res"], sum_out=s["sum"])
        return {k: s[k] for k in ("y", "sum", "mu", "rstd") if s[k] is not None}
    if op == "ln_bwd":
        ws = _workspace(s, sq.fp8_layernorm_bwd_workspace_bytes(c["rows"], c["cols"]))
        sq.fp8_layernorm_bwd(s["dy"], s["x"], s["gamma"], s["mu"], s["rstd"], s["dx"], s["dgamma"], s["dbeta"], ws,
                             dres=s["dres"])
        return {k: s[k] for k in ("dx", "dgamma", "dbeta")}
    if op == "glu_fwd":
        ws = _workspace(s, sq.fp8_glu_fwd_workspace_bytes(c["tokens"], c["inner"], c["hidden"]))
        sq.fp8_glu_fwd(s["x"], sq.E4M3, s["sx"], s["w"], sq.E4M3, s["sw"], acts[c["act"]], gu_out=s["gu"],
                       q_out=s["q"], q_format=sq.E4M3, q_state=s["state"], history_len=H, workspace=ws)
        return {"h": s["q"].view(F8["e4m3"]), "amax": s["state"][:1], **({"gu": s["gu"]} if c["save"] else {})}
    if op == "glu_bwd":
        T, d, F = c["tokens"], c["hidden"], c["inner"]
        sq.fp8_glu_bwd(s["dy"], sq.E5M2, s["sdy"], s["wd"], sq.E4M3, s["swd"], s["gu"], acts[c["act"]], s["q"],
                       sq.E5M2, s["state"], H)
        sdz = s["state"][H + 1:]
        sq.fp8_gemm_layout(s["q"], sq.E5M2, sdz, sq.K_MAJOR, s["w"], sq.E4M3, s["sw"], sq.MN_MAJOR, s["dx"], T, d,
                           2 * F)
        sq.fp8_gemm_layout(s["q"], sq.E5M2, sdz, sq.MN_MAJOR, s["x"], sq.E4M3, s["sx"], sq.MN_MAJOR, s["dw"], 2 * F,
                           d, T)
        sq.fp8_gemm_layout(s["dy"], sq.E5M2, s["sdy"], sq.MN_MAJOR, s["h"], sq.E4M3, s["sh"], sq.MN_MAJOR, s["dwd"],
                           d, F, T)
        return {"dgu": s["q"].view(F8["e5m2"]), "amax": s["state"][:1], "dx": s["dx"], "dw": s["dw"], "dwd": s["dwd"]}
    if op == "act_fwd":
        ws = _workspace(s, sq.fp8_gemm_act_workspace_bytes(c["tokens"], c["n"], c["k"]))
        sq.fp8_gemm_act(s["x"], sq.E4M3, s["sx"], s["w"], sq.E4M3, s["sw"], acts[c["act"]], D=s["d"], bias=s["bias"],
                        residual=s["res"], z_out=s["z"], q_out=s["q"], q_format=sq.E4M3, q_state=s["state"],
                        history_len=H if s["state"] is not None else 0, workspace=ws)
        if s["q"] is None:
            return {"d": s["d"]}
        return {"q": s["q"].view(F8["e4m3"]), "amax": s["state"][:1], "z": s["z"]}
    ws = _workspace(s, sq.fp8_act_bwd_workspace_bytes(c["tokens"], c["n"]))
    sq.fp8_act_bwd(s["dy"], s["z"], acts[c["act"]], dbias=s["dbias"], q_out=s["q"], q_format=sq.E5M2,
                   q_state=s["state"], history_len=H, workspace=ws)
    return {"dz": s["q"].view(F8["e5m2"]), "amax": s["state"][:1], "dbias": s["dbias"]}


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "ln_fwd":
        dt = DT[c["dtype"]]
        x = s["x"].float()
        out = {}
        if c["residual"]:
            out["sum"] = (x + s["res"].float()).to(dt)
            x = out["sum"].float()
        mu = x.mean(1, keepdim=True)
        rstd = 1 / torch.sqrt((x - mu).square().mean(1, keepdim=True) + EPS)
        return {"y": ((x - mu) * rstd * s["gamma"] + s["beta"]).to(dt), "mu": mu[:, 0], "rstd": rstd[:, 0], **out}
    if op == "ln_bwd":
        x, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
        xh = (x - s["mu"][:, None]) * rstd
        w = dy * s["gamma"]
        dx = rstd * (w - w.mean(1, keepdim=True) - xh * (w * xh).mean(1, keepdim=True))
        if c["dres"]:
            dx = dx + s["dres"].float()
        # sums over all rows, whose terms cancel: in 64 bits
        return {"dx": dx.to(DT[c["dtype"]]), "dgamma": (dy * xh).sum(0, dtype=torch.float64).float(),
                "dbeta": dy.sum(0, dtype=torch.float64).float()}
    if op == "glu_fwd":
        F = c["inner"]
        z = (_values(s["x"], "e4m3") @ _values(s["w"], "e4m3").t()) * (s["sx"] * s["sw"])
        h = _act(z[:, :F], c["act"]) * z[:, F:]
        q, amax = _cast(h, "e4m3", s["state"])
        return {"h": q, "amax": amax, **({"gu": z.to(torch.bfloat16)} if c["save"] else {})}
    if op == "glu_bwd":
        F = c["inner"]
        dyv, wv = _values(s["dy"], "e5m2"), _values(s["w"], "e4m3")
        dh = (dyv @ _values(s["wd"], "e4m3")) * (s["sdy"] * s["swd"])
        gate, up = s["gu"][:, :F].float(), s["gu"][:, F:].float()
        dgu = torch.cat([dh * up * _dact(gate, c["act"]), dh * _act(gate, c["act"])], 1)
        q, amax = _cast(dgu, "e5m2", s["state"])
        qv, sdz, b = q.float(), s["state"][H + 1], torch.bfloat16
        dx = ((qv @ wv) * (sdz * s["sw"])).to(b)
        dw = ((qv.t() @ _values(s["x"], "e4m3")) * (sdz * s["sx"])).to(b)
        dwd = ((dyv.t() @ _values(s["h"], "e4m3")) * (s["sdy"] * s["sh"])).to(b)
        return {"dgu": q, "amax": amax, "dx": dx, "dw": dw, "dwd": dwd}
    if op == "act_fwd":
        z = (_values(s["x"], "e4m3") @ _values(s["w"], "e4m3").t()) * (s["sx"] * s["sw"])
        if c["bias"]:
            z = z + s["bias"]
        y = _act(z, c["act"])
        if c["residual"]:
            y = y + s["res"].float()
        if c["out"] != "codes":
            return {"d": y.to(DT[c["out"]])}
        q, amax = _cast(y, "e4m3", s["state"])
        return {"q": q, "amax": amax, "z": z.to(torch.bfloat16)}
    dz = s["dy"].float() * _dact(s["z"].float(), c["act"])
    q, amax = _cast(dz, "e5m2", s["state"])
    return {"dz": q, "amax": amax, "dbias": dz.sum(0, dtype=torch.float64).float()}


# ---------------------------------------------------------------------------------------------------- work, definition
def work(case):
    c, op = case, case["op"]
    if op in ("ln_fwd", "ln_bwd"):
        R, K = c["rows"], c["cols"]
        e = 2 if c["dtype"] == "bf16" else 4
        if op == "ln_fwd":
            return {"bytes": (4 if c["residual"] else 2) * e * R * K + 8 * K + 8 * R, "flops": 8 * R * K}
        return {"bytes": (4 if c["dres"] else 3) * e * R * K + 12 * K + 8 * R, "flops": 14 * R * K}
    if op == "glu_fwd":
        T, d, F = c["tokens"], c["hidden"], c["inner"]
        return {"bytes": T * d + 2 * F * d + T * F + (4 * T * F if c["save"] else 0), "flops": 4 * T * d * F}
    if op == "glu_bwd":
        T, d, F = c["tokens"], c["hidden"], c["inner"]
        # read dy, Wd, W, x, h, [g|u]; write the codes of [dg|du], dx, both weight gradients
        return {"bytes": T * d + d * F + 2 * F * d + T * d + T * F + 4 * T * F + 2 * T * F + 2 * T * d + 6 * d * F,
                "flops": 12 * T * d * F}
    if op == "act_fwd":
        T, K, N = c["tokens"], c["k"], c["n"]
        e = {"bf16": 2, "f32": 4, "codes": 1}[c["out"]]
        return {"bytes": T * K + N * K + e * T * N * (2 if c["residual"] else 1) + (2 * T * N if c["save"] else 0)
                + (4 * N if c["bias"] else 0), "flops": 2 * T * K * N}
    T, N = c["tokens"], c["n"]
    return {"bytes": 5 * T * N + 4 * N, "flops": 12 * T * N}


def _act64(z, act):
    """(act(z), act'(z)) from the definitions with the normal distribution function and the logistic function."""
    if act == "none":
        return z, torch.ones_like(z)
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
    """Codes of 64-bit values: the FP8 numbers nearest to the scaled and clipped values."""
    q = (v * st[H].double()).clamp(-FMAX[fmt], FMAX[fmt]).float().to(F8[fmt])
    return q, torch.maximum(st[:1].double(), v.abs().max().reshape(1))


def exact(case, seed):
    c, op = case, case["op"]
    s = prepare(case, seed)
    val = lambda k, fmt: s[k].view(F8[fmt]).double()                                                # noqa: E731
    sc = lambda a, b: s[a].double() * s[b].double()                                                 # noqa: E731
    if op == "ln_fwd":
        x = s["x"].double()
        total = None
        if c["residual"]:
            total = (s["x"].double() + s["res"].double()).to(DT[c["dtype"]])
            x = total.double()
        var, mu = torch.var_mean(x, dim=1, correction=0)
        rstd = (var + EPS) ** -0.5
        y = torch.addcmul(s["beta"].double(), (x - mu[:, None]) * rstd[:, None], s["gamma"].double())
        return {"y": y, "mu": mu, "rstd": rstd, **({"sum": total} if c["residual"] else {})}
    if op == "ln_bwd":
        x, dy, K = s["x"].double(), s["dy"].double(), c["cols"]
        rstd = s["rstd"].double()
        xh = torch.einsum("rc,r->rc", x - s["mu"].double()[:, None], rstd)
        w = torch.einsum("rc,c->rc", dy, s["gamma"].double())
        a, b = w.sum(1) / K, torch.einsum("rc,rc->r", w, xh) / K
        dx = torch.einsum("rc,r->rc", w - a[:, None] - xh * b[:, None], rstd)
        if c["dres"]:
            dx += s["dres"].double()
        return {"dx": dx, "dgamma": torch.einsum("rc,rc->c", dy, xh), "dbeta": dy.sum(0)}
    if op == "glu_fwd":
        F = c["inner"]
        w = val("w", "e4m3")
        k = sc("sx", "sw")
        x = val("x", "e4m3")
        gate, up = torch.mm(x, w[:F].T) * k, torch.mm(x, w[F:].T) * k
        q, amax = _cast64(_act64(gate, c["act"])[0] * up, "e4m3", s["state"])
        return {"h": q, "amax": amax, **({"gu": torch.cat([gate, up], 1)} if c["save"] else {})}
    if op == "glu_bwd":
        F = c["inner"]
        dh = torch.mm(val("dy", "e5m2"), val("wd", "e4m3")) * sc("sdy", "swd")
        gate, up = s["gu"].double().split(F, 1)
        f, df = _act64(gate, c["act"])
        q, amax = _cast64(torch.cat([dh * up * df, dh * f], 1), "e5m2", s["state"])
        sd = s["state"][H + 1].double()
        qd = q.double()
        return {"dgu": q, "amax": amax, "dx": torch.mm(qd, val("w", "e4m3")) * (sd * s["sw"].double()),
                "dw": torch.mm(qd.T, val("x", "e4m3")) * (sd * s["sx"].double()),
                "dwd": torch.mm(val("dy", "e5m2").T, val("h", "e4m3")) * sc("sdy", "sh")}
    if op == "act_fwd":
        z = torch.mm(val("x", "e4m3"), val("w", "e4m3").T) * sc("sx", "sw")
        if c["bias"]:
            z += s["bias"].double()
        y = _act64(z, c["act"])[0]
        if c["residual"]:
            y = y + s["res"].double()
        if c["out"] != "codes":
            return {"d": y}
        q, amax = _cast64(y, "e4m3", s["state"])
        return {"q": q, "amax": amax, "z": z}
    dz = s["dy"].double() * _act64(s["z"].double(), c["act"])[1]
    q, amax = _cast64(dz, "e5m2", s["state"])
    return {"dz": q, "amax": amax, "dbias": dz.sum(0)}
