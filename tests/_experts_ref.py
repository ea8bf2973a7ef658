"""Rows sorted by expert, walked slot by slot, and routings to test them with.

Bounds: u = 2^-24.  A sum of n fp32 terms in any order is within (n - 1) u of the
sum of their magnitudes; each product or addition beside it adds u of its value.
Products on the tensor cores: _ffn_ref.product."""
import torch

import scaled_quantize_gemm_gb300 as sq

PAD, TILE = 32, 256


def walk(ids, E):
    """(row of every slot or -1, offsets [E + 1], counts [E]) of ids [T][k], in plain Python"""
    T, k = ids.shape
    lists = [[] for _ in range(E)]
    for i, e in enumerate(ids.reshape(-1).tolist()):
        if 0 <= e < E:
            lists[e].append(i)
    row, offsets = [-1] * (T * k), [0]
    for a in lists:
        for r, i in enumerate(a):
            row[i] = offsets[-1] + r
        offsets.append(offsets[-1] + -(-len(a) // PAD) * PAD)
    return torch.tensor(row, dtype=torch.int32).reshape(T, k), offsets, [len(a) for a in lists]


def routing(g, T, k, E, how, device="cuda"):
    """ids [T][k]: spread, skewed (most slots want expert 0), one (all of them), masked (some tokens go nowhere, some
    slots name no expert), none (every slot is left out), last (all want the last expert)"""
    rand = lambda *s: torch.rand(s, generator=g, device=device)                                   # noqa: E731
    ids = (rand(T, k) * E).int().clamp_(max=E - 1)
    if how == "skewed":
        ids[rand(T, k) < 0.8] = 0
    elif how == "one":
        ids.fill_(0)
    elif how == "last":
        ids.fill_(E - 1)
    elif how == "masked":
        ids[rand(T) < 0.3] = -1
        ids[rand(T, k) < 0.1] = E
        ids[rand(T, k) < 0.05] = 2 ** 31 - 1
        ids[rand(T, k) < 0.05] = -2 ** 31
    elif how == "none":
        ids.fill_(-1)
    return ids.contiguous()


def make_plan(ids, E):
    T, k = ids.shape
    plan = torch.full((sq.fp8_expert_plan_ints(T, k, E),), -77, dtype=torch.int32, device=ids.device)
    sq.fp8_expert_plan(ids, E, plan)
    return plan


def place(row, values, R, fill=0):
    """[R][K] with values[t] (or values[t][j]) at the row of (t, j)"""
    out = torch.full((R, values.shape[-1]), fill, dtype=values.dtype, device=values.device)
    for j in range(row.shape[1]):
        live = row[:, j] >= 0
        out[row[live, j].long()] = values[live, j] if values.dim() == 3 else values[live]
    return out


ROUTINGS = [(1, 1, 1, "spread"), (1, 8, 64, "spread"), (7, 2, 3, "masked"), (37, 3, 5, "skewed"), (64, 8, 64, "spread"),
            (300, 1, 2, "one"), (333, 4, 7, "masked"), (513, 2, 1024, "spread"), (1000, 2, 16, "last"), (40, 64, 100, "spread"),
            (5, 2, 4, "none"), (5000, 1, 2, "skewed"), (20011, 3, 40, "masked")]
