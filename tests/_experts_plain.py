"""The entry points that ExpertFFN calls, in plain torch arithmetic, so that what the class keeps, shares and overwrites
can be tested without a GPU.  A plan here is offsets, counts and rows as the library documents them."""
import torch

import scaled_quantize_gemm_gb300 as sq
from _experts_ref import PAD, walk
from _ffn_plain import _act, _cast, _use, _val, quantize, scale_init, update_scale


def rows_of(T, k, E):
    n = T * k
    return (n + (PAD - 1) * min(E, n)) // PAD * PAD


def plan_ints(T, k, E):
    return 2 * E + 1 + T * k


def plan(ids, E, out):
    row, offsets, counts = walk(ids.cpu(), E)
    out[:2 * E + 1 + ids.numel()] = torch.tensor(offsets + counts + row.reshape(-1).tolist(), dtype=torch.int32, device=out.device)


def _rows(p, E, T, k):
    return p[2 * E + 1:2 * E + 1 + T * k].view(T, k).long()


def _segments(p, E):
    o = p[:E + 1].tolist()
    return [(e, slice(o[e], o[e + 1])) for e in range(E) if o[e + 1] > o[e]]


def rmsnorm_fwd(x, gamma, eps, y, rstd=None, q_out=None, q_format=0, q_state=None, history_len=0):
    v = x.float()
    r = (v.square().mean(1) + eps).rsqrt()
    if rstd is not None:
        rstd.copy_(r)
    _cast(v * r[:, None] * gamma, q_out, q_format, q_state, history_len)


def rmsnorm_bwd(dy, x, gamma, rstd, dx, dgamma, workspace, dres=None):
    d, xh = dy.float(), x.float() * rstd[:, None]
    w = d * gamma
    dx.copy_(rstd[:, None] * (w - xh * (w * xh).mean(1, keepdim=True)) + dres.float())
    dgamma.copy_((d * xh).sum(0))


def dispatch(x, p, k, E, rows):
    row = _rows(p, E, x.shape[0], k)
    rows[:int(p[E])] = 0
    for j in range(k):
        on = row[:, j] >= 0
        rows[row[on, j]] = x[on]


def combine(rows, p, k, E, y, weights=None, residual=None):
    row = _rows(p, E, y.shape[0], k)
    out = torch.zeros(y.shape, device=y.device)
    for j in range(k):
        on = row[:, j] >= 0
        out[on] += rows[row[on, j]].float() * (1.0 if weights is None else weights[on, j:j + 1])
    y.copy_(out + (0 if residual is None else residual.float()))


def combine_bwd(dy, p, k, E, weights, rows=None, dweights=None, q_out=None, q_format=1, q_state=None, history_len=0):
    row = _rows(p, E, dy.shape[0], k)
    d = torch.zeros((int(p[E]), dy.shape[1]), device=dy.device)
    dweights.zero_()
    for j in range(k):
        on = row[:, j] >= 0
        d[row[on, j]] = dy[on].float() * weights[on, j:j + 1]
        dweights[on, j] = (dy[on].float() * rows[row[on, j]].float()).sum(1)
    _cast(d, q_out[:d.shape[0]], q_format, q_state, history_len)


def glu_fwd(A, fa, sa, W, fw, sw, act, p, T, k, gu_out=None, q_out=None, q_format=0, q_state=None, history_len=0, workspace=None):
    _use(workspace)
    E, F = W.shape[0], W.shape[1] // 2
    for e, r in _segments(p, E):
        z = _val(A[r], fa, sa) @ _val(W[e], fw, sw[e]).T
        if gu_out is not None:
            gu_out[r] = z.to(gu_out.dtype)
        _cast(_act(z[:, :F], act)[0] * z[:, F:], q_out[r], q_format, q_state, history_len)


def gemm(A, fa, sa, B, fb, sb, major, p, T, k, D, workspace=None):
    _use(workspace)
    for e, r in _segments(p, B.shape[0]):
        b = _val(B[e], fb, sb[e])
        D[r] = (_val(A[r], fa, sa) @ (b if major == sq.MN_MAJOR else b.T)).to(D.dtype)


def glu_bwd(dY, fd, sd, Wd, fw, sw, gu, act, p, T, k, q, qf, state, H):
    F = Wd.shape[2]
    for e, r in _segments(p, Wd.shape[0]):
        dh = _val(dY[r], fd, sd) @ _val(Wd[e], fw, sw[e])
        g, u = gu[r, :F].float(), gu[r, F:].float()
        f, d = _act(g, act)
        _cast(torch.cat([dh * u * d, dh * f], 1), q[r], qf, state, H)


def wgrad(A, fa, sa, B, fb, sb, p, T, k, D):
    D.zero_()
    for e, r in _segments(p, D.shape[0]):
        D[e] = _val(A[r], fa, sa).T @ _val(B[r], fb, sb)


def install(monkeypatch):
    for name, f in dict(fp8_scale_init=scale_init, fp8_update_scale=update_scale, fp8_quantize=quantize,
                        fp8_rmsnorm_fwd=rmsnorm_fwd, fp8_rmsnorm_bwd=rmsnorm_bwd, fp8_expert_rows=rows_of,
                        fp8_expert_plan_ints=plan_ints, fp8_expert_plan=plan, fp8_expert_dispatch=dispatch,
                        fp8_expert_combine=combine, fp8_expert_combine_bwd=combine_bwd, fp8_expert_glu_fwd=glu_fwd,
                        fp8_expert_gemm=gemm, fp8_expert_glu_bwd=glu_bwd, fp8_expert_wgrad=wgrad).items():
        monkeypatch.setattr(sq, name, f)
    monkeypatch.setattr(sq, "fp8_expert_workspace_bytes", lambda T, k, E, N, K: 64 * T)
    monkeypatch.setattr(sq, "fp8_rmsnorm_bwd_workspace_bytes", lambda M, K: 4 * K)
