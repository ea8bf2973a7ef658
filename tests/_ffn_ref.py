"""The feed-forward operators in 64 bits, and the error bounds their fp32
kernels are held to.

u = 2^-24 is half a step of fp32.  A product accumulates K terms in fp32, 32
per tensor-core instruction, each step rounded (or cut off) within 2 u of the
running magnitude, so |z - z64| <= 2 u (K / 32 + 8) S with S the sum of the
terms' magnitudes.  An elementwise function of fp32 arguments is given 2^-19 of
the magnitudes that enter it: the hardware exponential's argument carries a
rounding of u |x log2 e|, 30 u for the largest arguments here, beside a few
units for exp, the reciprocal and the products.  A stored value adds half a
step of its type: 2^-8 for bf16 (relative), 2^-24 for fp32.  A code has to lie
between the codes of the two ends of the bound.
"""
import math

import torch

U = 2.0 ** -24
ELEM = 2.0 ** -19
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
FMAX = (448.0, 57344.0)
F8 = (torch.float8_e4m3fn, torch.float8_e5m2)
NONE, RELU, GELU, GELU_TANH, SILU = range(5)
ACTS = (NONE, RELU, GELU, GELU_TANH, SILU)
SLOPE = 1.13              # the largest |act'| (gelu's, 1.129)
CURVE = 1.0               # the largest |act''| (gelu_tanh's 0.80, silu's 0.5)


def act64(x, act):
    if act == NONE:
        return x, torch.ones_like(x)
    if act == RELU:
        return x.clamp_min(0), (x > 0).double()
    if act == GELU:
        phi = 0.5 * (1 + torch.erf(x / math.sqrt(2)))
        return x * phi, phi + x * torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
    if act == SILU:
        s = torch.sigmoid(x)
        return x * s, s * (1 + x * (1 - s))
    a = math.sqrt(2 / math.pi)
    t = torch.tanh(a * (x + 0.044715 * x ** 3))
    return 0.5 * x * (1 + t), 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * a * (1 + 3 * 0.044715 * x * x)


def values(codes, fmt):
    return codes.view(F8[fmt]).double()


def product(a, b, s):
    """(z, bound): a b^T s in 64 bits, and the kernel's error bound."""
    K = a.shape[1]
    z = a @ b.T * s
    return z, 2 * U * (K / 32 + 8) * (a.abs() @ b.abs().T * s) + 4 * U * z.abs()


def gated(g, eg, u, eu, act):
    """(h, bound) of h = act(g) u with errors eg, eu on the arguments."""
    f, _ = act64(g, act)
    ef = SLOPE * eg + ELEM * g.abs()
    return f * u, ef * (u.abs() + eu) + f.abs() * eu + ELEM * (f * u).abs()


def assert_within(got, want, bound, what=""):
    """got (stored) against want (64 bits): the bound plus half a step of got's type."""
    g = got.double()
    assert g.shape == want.shape, what
    assert bool(torch.isfinite(g).all()), f"{what}: not finite"
    tiny = 2.0 ** -133 if got.dtype == torch.bfloat16 else 2.0 ** -149
    tol = bound + HALF[got.dtype] * torch.maximum(g.abs(), want.abs()) + tiny
    over = (g - want).abs() - tol
    worst = float(over.max()) if over.numel() else -1.0
    assert worst <= 0, f"{what}: {int((over > 0).sum())} of {over.numel()} beyond the bound, worst by {worst:.3e}"


def round_codes(v, fmt):
    return v.clamp(-FMAX[fmt], FMAX[fmt]).float().to(F8[fmt]).double()


def assert_codes(codes, want, bound, m, fmt, what=""):
    got = values(codes, fmt)
    assert bool(torch.isfinite(got).all()), f"{what}: a NaN code"
    # the product with the multiplier is one more fp32 rounding
    e = bound + 2 * U * want.abs()
    lo, hi = round_codes((want - e) * m, fmt), round_codes((want + e) * m, fmt)
    bad = (got < lo) | (got > hi)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} codes outside their bracket"


def assert_amax(state, before, want, bound, what=""):
    """state[0] holds max(before, max |want|) within the largest bound."""
    w = max(before, float(want.abs().max()) if want.numel() else 0.0)
    tol = (float(bound.max()) if bound.numel() else 0.0) + 4 * U * w
    assert abs(float(state[0]) - w) <= tol, f"{what}: amax {float(state[0])} against {w}"


# ---------------------------------------------------------------- inputs
def gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def randn(g, *shape, device="cuda"):
    return torch.randn(shape, generator=g, device=device)


def to_codes(x, fmt):
    s = float(x.abs().max()) / FMAX[fmt]
    s = s if s > 0 else 1.0
    q = (x / s).clamp(-FMAX[fmt], FMAX[fmt]).to(F8[fmt]).view(torch.uint8).contiguous()
    return q, torch.full((1,), s, device=x.device)


def new_state(H, m, newest=0.0, device="cuda"):
    st = torch.zeros(H + 2, device=device)
    st[0], st[H], st[H + 1] = newest, m, 1.0 / m
    return st
