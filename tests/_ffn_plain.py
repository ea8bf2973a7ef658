"""The entry points that GatedFFN calls, in plain torch arithmetic on the CPU, so that what the class keeps, shares and
overwrites can be tested without a GPU.  Their workspace is a byte that has to be found zero and is left zero."""
import torch

import scaled_quantize_gemm_gb300 as sq
from _ffn_ref import F8, FMAX, act64


def _val(q, fmt, scale):
    return q.view(F8[fmt]).float() * scale


def _cast(v, q, fmt, state, H):
    q.copy_((v * state[H]).clamp(-FMAX[fmt], FMAX[fmt]).to(F8[fmt]).view(torch.uint8))
    if v.numel():
        state[0] = torch.maximum(state[0], v.abs().max())


def _act(x, act):
    f, d = act64(x.double(), act)
    return f.float(), d.float()


def _use(workspace):
    assert workspace is None or not bool(workspace.any()), "a workspace that is not zero"


def scale_init(states, n, H):
    b = states.view(n, H + 2)
    b.zero_()
    b[:, H:] = 1.0


def update_scale(states, n, H, formats):
    for b, f in zip(states.view(n, H + 2), formats):
        amax = float(b[:H].max())
        b[1:H] = b[:H - 1].clone()
        b[0] = 0.0
        if amax > 0:
            b[H], b[H + 1] = FMAX[f] / amax, amax / FMAX[f]


def quantize(x, fmt, gran, q, delayed_state=None, history_len=0):
    _cast(x.float(), q.view(x.shape), fmt, delayed_state, history_len)


def layernorm_fwd(x, gamma, beta, eps, y, mu=None, rstd=None, q_out=None, q_format=0, q_state=None, history_len=0):
    v = x.float()
    m = v.mean(1)
    r = ((v - m[:, None]).square().mean(1) + eps).rsqrt()
    if mu is not None:
        mu.copy_(m)
        rstd.copy_(r)
    n = (v - m[:, None]) * r[:, None] * gamma + (0 if beta is None else beta)
    _cast(n, q_out, q_format, q_state, history_len)


def glu_fwd(A, fa, sa, W, fw, sw, act, gu_out=None, q_out=None, q_format=0, q_state=None, history_len=0, workspace=None):
    _use(workspace)
    z = _val(A, fa, sa) @ _val(W, fw, sw).T
    if gu_out is not None:
        gu_out.copy_(z)
    F = W.shape[0] // 2
    _cast(_act(z[:, :F], act)[0] * z[:, F:], q_out, q_format, q_state, history_len)


def gemm_act(A, fa, sa, B, fb, sb, act, D=None, residual=None, workspace=None):
    _use(workspace)
    D.copy_(_val(A, fa, sa) @ _val(B, fb, sb).T + residual.float())


def glu_bwd(dY, fd, sd, Wd, fw, sw, gu, act, q, qf, state, H):
    dh = _val(dY, fd, sd) @ _val(Wd, fw, sw)
    F = Wd.shape[1]
    g, u = gu[:, :F].float(), gu[:, F:].float()
    f, d = _act(g, act)
    _cast(torch.cat([dh * u * d, dh * f], 1), q, qf, state, H)


def gemm_layout(A, fa, sa, ma, B, fb, sb, mb, D, M, N, K):
    a, b = _val(A, fa, sa), _val(B, fb, sb)
    D.copy_((a.T if ma == sq.MN_MAJOR else a) @ (b if mb == sq.MN_MAJOR else b.T))


def layernorm_bwd(dy, x, gamma, mu, rstd, dx, dgamma, dbeta, workspace, dres=None):
    d, xh = dy.float(), (x.float() - mu[:, None]) * rstd[:, None]
    w = d * gamma
    dx.copy_(rstd[:, None] * (w - w.mean(1, keepdim=True) - xh * (w * xh).mean(1, keepdim=True)) + dres.float())
    dgamma.copy_((d * xh).sum(0))
    dbeta.copy_(d.sum(0))


def install(monkeypatch):
    for name, f in dict(fp8_scale_init=scale_init, fp8_update_scale=update_scale, fp8_quantize=quantize,
                        fp8_layernorm_fwd=layernorm_fwd, fp8_glu_fwd=glu_fwd, fp8_gemm_act=gemm_act,
                        fp8_glu_bwd=glu_bwd, fp8_gemm_layout=gemm_layout, fp8_layernorm_bwd=layernorm_bwd).items():
        monkeypatch.setattr(sq, name, f)
    monkeypatch.setattr(sq, "fp8_glu_fwd_workspace_bytes", lambda M, F, K: 64 * M)
    monkeypatch.setattr(sq, "fp8_gemm_act_workspace_bytes", lambda M, N, K: 64 * M)
    monkeypatch.setattr(sq, "fp8_layernorm_bwd_workspace_bytes", lambda M, K: 8 * K)
