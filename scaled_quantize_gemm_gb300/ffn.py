"""A pre-norm gated feed-forward sublayer on the FP8 path (te.LayerNormMLP's
parts, gated):

    n = LayerNorm(x) gamma + beta            cast to E4M3 in the same kernel
    [g | u] = n [W_gate; W_up]^T             one product; h = act(g) u is formed
    h = act(g) u                             and cast in its epilogue
    y = x + h W_down^T                       the residual added in the epilogue

with per-tensor delayed scaling for every cast.  ``forward`` and ``backward``
are a training step (weights cast from bf16 every step, as they change);
``freeze`` casts the weights once and keeps the scales of that moment, and
``decode`` runs a few tokens at a time with both: three kernels, each streaming
its weights once.  Codes are turned back with the steps that they were cast
with, wherever ``update_scales`` falls: between ``freeze`` and ``decode``, or
between ``forward`` and ``backward``.

The backward pass takes dY in E5M2 (HYBRID) and never writes the gradient of
h: its product's epilogue turns it into the codes of [dg | du], which feed the
data and weight gradients as they are.
"""
from __future__ import annotations

import math

import torch

import scaled_quantize_gemm_gb300 as sq

# delayed-scaling states, in the order of GatedFFN.states
N, W_GU, H_, W_DOWN, DY, DGU = range(6)
FORMATS = [sq.E4M3, sq.E4M3, sq.E4M3, sq.E4M3, sq.E5M2, sq.E5M2]


def _capturing() -> bool:
    return torch.cuda.is_available() and torch.cuda.is_current_stream_capturing()


class GatedFFN:
    """One sublayer's weights, scaling states and buffers.

    gamma [K] fp32, beta [K] fp32 or None, w_gate_up [2F][K] bf16 (the gate's
    rows, then the up projection's), w_down [K][F] bf16; K, F multiples of 16.
    A training step takes a number of tokens that is a multiple of 16 (the
    weight gradients contract over them); ``decode`` takes any number.

    The buffers are the block's own, one set for all calls, so its calls follow
    one another on one stream (or in streams that wait for each other), and one
    forward is kept at a time.  Calls may be captured into CUDA graphs, also
    for several numbers of tokens: a buffer that a call was given lives as long
    as the block.
    """

    def __init__(self, gamma, beta, w_gate_up, w_down, act: int = sq.ACT_SILU, eps: float = 1e-5,
                 history_len: int = 16):
        F2, K = w_gate_up.shape
        if F2 % 32 or K % 16 or tuple(w_down.shape) != (K, F2 // 2):
            raise ValueError(f"w_gate_up {tuple(w_gate_up.shape)} and w_down {tuple(w_down.shape)} do not make a "
                             "gated block of sizes that are multiples of 16")
        self.gamma, self.beta, self.w_gate_up, self.w_down = gamma, beta, w_gate_up, w_down
        self.K, self.F, self.act, self.eps, self.H = K, F2 // 2, act, eps, history_len
        dev = w_gate_up.device
        self._states = torch.empty(6 * sq.state_floats(history_len), device=dev)
        sq.fp8_scale_init(self.states, 6, history_len)
        self.q_gate_up = torch.empty((F2, K), dtype=torch.uint8, device=dev)
        self.q_down = torch.empty((K, self.F), dtype=torch.uint8, device=dev)
        self._frozen = torch.empty_like(self.states)     # the states as they were when the weights were last cast
        self._cast = False                   # ... which they have been
        self._live, self._kept_scales = self._split(self.states), self._split(self._frozen)
        self._buffers = {}                   # name -> the largest buffer so far, in bytes
        self._views = {}                     # name -> its last view
        self._kept = []                      # every buffer: a captured graph may replay on it
        self._spaces = []                    # the workspaces among them
        self._saved = None

    # ------------------------------------------------------------ states and scratch
    @property
    def states(self):
        """the six delayed-scaling states, one after another; assigning copies into them (views and graphs hold them)"""
        return self._states

    @states.setter
    def states(self, values):
        self._states.copy_(values)

    def _split(self, states):
        """the six states and the dequantisation steps of their codes (one element each), as views"""
        blocks = states.view(6, sq.state_floats(self.H))
        return list(blocks), list(blocks[:, -1:])

    def _state(self, i):
        return self._live[0][i]

    def _scale(self, i):
        return self._live[1][i]

    def _bytes(self, name, nbytes, zero=False):
        """A buffer of at least `nbytes` that lives as long as the block.  A larger one than before is at least twice
        as large, so all the smaller ones together are no larger than it.  One that is made while a graph is being
        captured belongs to that graph (its memory, and what fills it, come with the replay) and is not handed on."""
        t = self._buffers.get(name)
        if t is None or t.numel() < nbytes:
            n = max(nbytes, 0 if t is None else 2 * t.numel())
            t = (torch.zeros if zero else torch.empty)(n, dtype=torch.uint8, device=self.states.device)
            self._kept.append(t)
            if zero:
                self._spaces.append(t)
            if not _capturing():
                self._buffers[name] = t
        return t

    def _get(self, name, shape, dtype):
        v = self._views.get(name)
        if v is not None and v.shape == shape and v.dtype is dtype:
            return v
        nbytes = math.prod(shape) * dtype.itemsize
        t = self._bytes(name, nbytes)
        v = t[:nbytes].view(dtype).view(shape)
        if t is self._buffers.get(name):
            self._views[name] = v
        return v

    def _workspace(self, name, nbytes):
        """scratch of the split products (zeroed when made, left so by every call)"""
        return self._bytes(name, nbytes, zero=True) if nbytes else None

    def reset_workspaces(self):
        """Zeroes the workspaces: to be called after ``fp8_device_status`` returned ERR_TIMEOUT, as a kernel that gave
        up leaves its counters as they were, and later calls would join their sums too early or never."""
        for t in self._spaces:
            t.zero_()

    def calibrate(self, x):
        """One forward pass that sets the activations' and weights' scales from what it records."""
        for _ in range(2):
            self.forward(x)
            self.update_scales()

    def update_scales(self):
        """The end-of-step update of all states (history maximum)."""
        sq.fp8_update_scale(self.states, 6, self.H, FORMATS)

    def freeze(self):
        """Casts both weights with their current scales and keeps all scales as they are now, for ``decode``."""
        for w, q, i in ((self.w_gate_up, self.q_gate_up, W_GU), (self.w_down, self.q_down, W_DOWN)):
            sq.fp8_quantize(w, FORMATS[i], sq.TENSOR, q, delayed_state=self._state(i), history_len=self.H)
        self._frozen.copy_(self.states)
        self._cast = True

    # ------------------------------------------------------------ one pass
    def _run(self, x, gu, mu, rstd, y, codes, scales):
        """One pass with the activations' states and steps in `scales`; `codes` names the buffers of n's and h's
        codes: a training step's are read again by its backward pass, so nothing else may write them."""
        M, K, F, H = x.shape[0], self.K, self.F, self.H
        state, step = scales
        w_step = self._kept_scales[1]
        qn, qh = self._get("qn" + codes, (M, K), torch.uint8), self._get("qh" + codes, (M, F), torch.uint8)
        sq.fp8_layernorm_fwd(x, self.gamma, self.beta, self.eps, None, mu=mu, rstd=rstd, q_out=qn, q_format=sq.E4M3,
                             q_state=state[N], history_len=H)
        sq.fp8_glu_fwd(qn, sq.E4M3, step[N], self.q_gate_up, sq.E4M3, w_step[W_GU], self.act, gu_out=gu, q_out=qh,
                       q_format=sq.E4M3, q_state=state[H_], history_len=H,
                       workspace=self._workspace("ws_gu", sq.fp8_glu_fwd_workspace_bytes(M, F, K)))
        sq.fp8_gemm_act(qh, sq.E4M3, step[H_], self.q_down, sq.E4M3, w_step[W_DOWN], sq.ACT_NONE, D=y, residual=x,
                        workspace=self._workspace("ws_down", sq.fp8_gemm_act_workspace_bytes(M, K, F)))
        return qn, qh

    def decode(self, x, y=None):
        """y (which may be x itself) for any number of tokens, on the frozen weights and scales; keeps nothing for a
        backward pass and leaves the training step's statistics alone."""
        if not self._cast:
            raise RuntimeError("decode needs the weights' codes: call freeze (or forward) first")
        y = torch.empty_like(x) if y is None else y
        self._run(x, None, None, None, y, "_decode", self._kept_scales)
        return y

    def forward(self, x):
        """y [M][K] bf16 of x [M][K] bf16; keeps what ``backward`` needs, x itself among it."""
        M = x.shape[0]
        self.freeze()
        gu = self._get("gu", (M, 2 * self.F), torch.bfloat16)
        mu, rstd = self._get("mu", (M,), torch.float32), self._get("rstd", (M,), torch.float32)
        y = torch.empty_like(x)
        qn, qh = self._run(x, gu, mu, rstd, y, "", self._live)
        cast = self._get("cast", self.states.shape, torch.float32)       # the scales of qn and qh
        cast.copy_(self.states)
        self._saved = (x, gu, mu, rstd, qn, qh, cast)
        return y

    def backward(self, dy):
        """-> (dx bf16, dgamma, dbeta, dw_gate_up, dw_down, all fp32) of the last forward, on the weights' codes as
        last cast (by it, or by a ``freeze`` since)."""
        if self._saved is None:
            raise RuntimeError("backward without a forward")
        x, gu, mu, rstd, qn, qh, cast = self._saved
        M, K, F, H = x.shape[0], self.K, self.F, self.H
        if M % 16:
            raise ValueError(f"a training step takes a multiple of 16 tokens, got {M}")
        if dy.shape != x.shape or dy.dtype != x.dtype or not dy.is_contiguous():
            raise ValueError(f"dy: {tuple(dy.shape)} {dy.dtype}, the forward had {tuple(x.shape)} {x.dtype} (contiguous)")
        self._saved = None
        dev = x.device
        w_step, step = self._kept_scales[1], self._split(cast)[1]
        qdy, qdgu = self._get("qdy", (M, K), torch.uint8), self._get("qdgu", (M, 2 * F), torch.uint8)
        sq.fp8_quantize(dy, sq.E5M2, sq.TENSOR, qdy, delayed_state=self._state(DY), history_len=H)
        sq.fp8_glu_bwd(qdy, sq.E5M2, self._scale(DY), self.q_down, sq.E4M3, w_step[W_DOWN], gu, self.act, qdgu,
                       sq.E5M2, self._state(DGU), H)
        dn = self._get("dn", (M, K), torch.bfloat16)
        dw_gu = torch.empty((2 * F, K), device=dev)
        dw_down = torch.empty((K, F), device=dev)
        s_dy, s_dgu = self._scale(DY), self._scale(DGU)
        sq.fp8_gemm_layout(qdgu, sq.E5M2, s_dgu, sq.K_MAJOR, self.q_gate_up, sq.E4M3, w_step[W_GU], sq.MN_MAJOR, dn,
                           M, K, 2 * F)
        sq.fp8_gemm_layout(qdgu, sq.E5M2, s_dgu, sq.MN_MAJOR, qn, sq.E4M3, step[N], sq.MN_MAJOR, dw_gu, 2 * F, K, M)
        sq.fp8_gemm_layout(qdy, sq.E5M2, s_dy, sq.MN_MAJOR, qh, sq.E4M3, step[H_], sq.MN_MAJOR, dw_down, K, F, M)
        dx, dgamma, dbeta = torch.empty_like(x), torch.empty(K, device=dev), torch.empty(K, device=dev)
        ws = self._get("ws_ln", (max(16, sq.fp8_layernorm_bwd_workspace_bytes(M, K)),), torch.uint8)
        sq.fp8_layernorm_bwd(dn, x, self.gamma, mu, rstd, dx, dgamma, dbeta, ws, dres=dy)
        return dx, dgamma, dbeta, dw_gu, dw_down
