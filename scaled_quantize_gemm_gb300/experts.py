"""A pre-norm feed-forward sublayer of experts on the FP8 path:

    n = RMSNorm(x) gamma                       cast to E4M3 in the same kernel
    rows of n by expert                        the router's choice ids [T][k], sorted
    [g | u] = n_e [W_gate; W_up]_e^T           one product over all experts' rows; h = act(g) u
    h = act(g) u                               is formed and cast in its epilogue
    o = h_e W_down,e^T                         one product
    y[t] = x[t] + sum_j weights[t][j] o[row of (t, j)]

with per-tensor delayed scaling for the activations and a scale of its own for every
expert's weights.  The router is the caller's: ``ids`` int32 [T][k] (an id outside
[0, experts) leaves a slot out, as for padding) and ``weights`` fp32 [T][k], whose
gradient ``backward`` returns.  A token without any expert still passes through the
norm, its statistics and gamma's gradient: its rows of x and dy hold finite numbers.  Nothing of the routing is read on the host, so a
captured graph follows the ids that are in place when it is replayed.

``forward`` and ``backward`` are a training step (weights cast from bf16 every step,
as they change); ``freeze`` casts the weights once and keeps the scales of that
moment, and ``decode`` runs any number of tokens with both.  Codes are turned back with
the steps that they were cast with, wherever ``update_scales`` falls.
"""
from __future__ import annotations

import torch

import scaled_quantize_gemm_gb300 as sq
from scaled_quantize_gemm_gb300.ffn import Buffers

# delayed-scaling states of the activations, in the order of ExpertFFN.states; the
# experts' follow, E of w_gate_up and E of w_down
N, H_, DY, DGU = range(4)
FORMATS = [sq.E4M3, sq.E4M3, sq.E5M2, sq.E5M2]
MAX_STATES = 1024                        # of one fp8_update_scale


class ExpertFFN(Buffers):
    """One sublayer's weights, scaling states and buffers.

    gamma [K] fp32, w_gate_up [E][2F][K] bf16 (the gate's rows, then the up
    projection's), w_down [E][K][F] bf16; K a multiple of 32, F of 16.  Any number
    of tokens, for training too.

    The buffers are the block's own, one set for all calls, so its calls follow
    one another on one stream (or in streams that wait for each other), and one
    forward is kept at a time.  Calls may be captured into CUDA graphs, also for
    several numbers of tokens: a buffer that a call was given lives as long as the
    block.
    """

    def __init__(self, gamma, w_gate_up, w_down, top_k: int, act: int = sq.ACT_SILU, eps: float = 1e-5,
                 history_len: int = 16):
        E, F2, K = w_gate_up.shape
        if F2 % 32 or K % 32 or tuple(w_down.shape) != (E, K, F2 // 2):
            raise ValueError(f"w_gate_up {tuple(w_gate_up.shape)} and w_down {tuple(w_down.shape)} do not make experts of "
                             "gated blocks, hidden sizes multiples of 32 and inner sizes of 16")
        if not 1 <= top_k <= 64:
            raise ValueError(f"top_k {top_k}")
        super().__init__(w_gate_up.device)
        self.gamma, self.w_gate_up, self.w_down = gamma, w_gate_up, w_down
        self.E, self.K, self.F, self.top_k, self.act, self.eps, self.H = E, K, F2 // 2, top_k, act, eps, history_len
        dev, n = w_gate_up.device, sq.state_floats(history_len)
        self._count = 4 + 2 * E
        self._formats = FORMATS + [sq.E4M3] * (2 * E)
        self._states = torch.empty(self._count * n, device=dev)
        for i in range(0, self._count, MAX_STATES):
            m = min(MAX_STATES, self._count - i)
            sq.fp8_scale_init(self._states[i * n:(i + m) * n], m, history_len)
        self.q_gate_up = torch.empty((E, F2, K), dtype=torch.uint8, device=dev)
        self.q_down = torch.empty((E, K, self.F), dtype=torch.uint8, device=dev)
        self._frozen = torch.empty_like(self._states)    # the states as they were when the weights were last cast
        self._w_steps = torch.empty(2 * E, device=dev)   # their codes' dequantisation steps
        self._cast = False
        self._live, self._kept_scales = self._split(self._states), self._split(self._frozen)
        self._saved = None

    # ------------------------------------------------------------ states
    @property
    def states(self):
        """the delayed-scaling states, one after another; assigning copies into them (views and graphs hold them)"""
        return self._states

    @states.setter
    def states(self, values):
        self._states.copy_(values)

    def _split(self, states):
        """the states and the dequantisation steps of their codes (one element each), as views"""
        blocks = states.view(-1, sq.state_floats(self.H))
        return list(blocks), list(blocks[:, -1:])

    def update_scales(self):
        """The end-of-step update of all states (history maximum)."""
        n = sq.state_floats(self.H)
        for i in range(0, self._count, MAX_STATES):
            m = min(MAX_STATES, self._count - i)
            sq.fp8_update_scale(self._states[i * n:(i + m) * n], m, self.H, self._formats[i:i + m])

    def calibrate(self, x, ids, weights):
        """One forward pass that sets the activations' and weights' scales from what it records."""
        for _ in range(2):
            self.forward(x, ids, weights)
            self.update_scales()

    def freeze(self):
        """Casts the experts' weights with their current scales and keeps all scales as they are now, for ``decode``."""
        states = self._live[0]
        for first, w, q in ((4, self.w_gate_up, self.q_gate_up), (4 + self.E, self.w_down, self.q_down)):
            for e in range(self.E):
                sq.fp8_quantize(w[e], sq.E4M3, sq.TENSOR, q[e], delayed_state=states[first + e], history_len=self.H)
        self._frozen.copy_(self._states)
        self._w_steps.copy_(self._states.view(-1, sq.state_floats(self.H))[4:, -1])
        self._cast = True

    # ------------------------------------------------------------ one pass
    def _check(self, x, ids, weights):
        if ids.shape != (x.shape[0], self.top_k) or weights.shape != ids.shape:
            raise ValueError(f"ids {tuple(ids.shape)} and weights {tuple(weights.shape)}: expected {(x.shape[0], self.top_k)}")

    def _run(self, x, ids, weights, gu, rstd, y, codes, scales):
        """One pass with the activations' states and steps in `scales`; `codes` names the buffers that a training
        step's backward pass reads again, so nothing else may write them."""
        T, E, k, K, F, H = x.shape[0], self.E, self.top_k, self.K, self.F, self.H
        state, step = scales
        R = sq.fp8_expert_rows(T, k, E)
        plan = self._get("plan" + codes, (sq.fp8_expert_plan_ints(T, k, E),), torch.int32)
        qn, qx = self._get("qn", (T, K), torch.uint8), self._get("qx" + codes, (R, K), torch.uint8)
        qh, rows = self._get("qh" + codes, (R, F), torch.uint8), self._get("rows" + codes, (R, K), torch.bfloat16)
        sq.fp8_expert_plan(ids, E, plan)
        sq.fp8_rmsnorm_fwd(x, self.gamma, self.eps, None, rstd=rstd, q_out=qn, q_format=sq.E4M3, q_state=state[N],
                           history_len=H)
        sq.fp8_expert_dispatch(qn, plan, k, E, qx)
        sq.fp8_expert_glu_fwd(qx, sq.E4M3, step[N], self.q_gate_up, sq.E4M3, self._w_steps[:E], self.act, plan, T, k,
                              gu_out=gu, q_out=qh, q_format=sq.E4M3, q_state=state[H_], history_len=H,
                              workspace=self._workspace("ws_gu", sq.fp8_expert_workspace_bytes(T, k, E, 2 * F, K)))
        sq.fp8_expert_gemm(qh, sq.E4M3, step[H_], self.q_down, sq.E4M3, self._w_steps[E:], sq.K_MAJOR, plan, T, k, rows,
                           workspace=self._workspace("ws_down", sq.fp8_expert_workspace_bytes(T, k, E, K, F)))
        sq.fp8_expert_combine(rows, plan, k, E, y, weights=weights, residual=x)
        return plan, qx, qh, rows

    def decode(self, x, ids, weights, y=None):
        """y (which may be x itself) for any number of tokens, on the frozen weights and scales; keeps nothing for a
        backward pass and leaves the training step's statistics alone."""
        if not self._cast:
            raise RuntimeError("decode needs the weights' codes: call freeze (or forward) first")
        self._check(x, ids, weights)
        y = torch.empty_like(x) if y is None else y
        self._run(x, ids, weights, None, None, y, "_decode", self._kept_scales)
        return y

    def forward(self, x, ids, weights):
        """y [T][K] bf16 of x [T][K] bf16; keeps what ``backward`` needs, x and weights themselves among it."""
        self._check(x, ids, weights)
        T = x.shape[0]
        self.freeze()
        gu = self._get("gu", (sq.fp8_expert_rows(T, self.top_k, self.E), 2 * self.F), torch.bfloat16)
        rstd = self._get("rstd", (T,), torch.float32)
        y = torch.empty_like(x)
        plan, qx, qh, rows = self._run(x, ids, weights, gu, rstd, y, "", self._live)
        cast = self._get("cast", self._states.shape, torch.float32)      # the scales of qx and qh
        cast.copy_(self._states)
        self._saved = (x, weights, gu, rstd, plan, qx, qh, rows, cast)
        return y

    def backward(self, dy):
        """-> (dx bf16, dweights, dgamma, dw_gate_up, dw_down, all fp32) of the last forward, on the weights' codes as
        last cast (by it, or by a ``freeze`` since)."""
        if self._saved is None:
            raise RuntimeError("backward without a forward")
        x, weights, gu, rstd, plan, qx, qh, rows, cast = self._saved
        if dy.shape != x.shape or dy.dtype != x.dtype or not dy.is_contiguous():
            raise ValueError(f"dy: {tuple(dy.shape)} {dy.dtype}, the forward had {tuple(x.shape)} {x.dtype} (contiguous)")
        self._saved = None
        T, E, k, K, F, H = x.shape[0], self.E, self.top_k, self.K, self.F, self.H
        R, dev = rows.shape[0], x.device
        state, now = self._live
        step = self._split(cast)[1]
        qdy, qdgu = self._get("qdy", (R, K), torch.uint8), self._get("qdgu", (R, 2 * F), torch.uint8)
        dweights = torch.empty((T, k), device=dev)
        sq.fp8_expert_combine_bwd(dy, plan, k, E, weights, rows=rows, dweights=dweights, q_out=qdy, q_format=sq.E5M2,
                                  q_state=state[DY], history_len=H)
        sq.fp8_expert_glu_bwd(qdy, sq.E5M2, now[DY], self.q_down, sq.E4M3, self._w_steps[E:], gu, self.act, plan, T, k, qdgu,
                              sq.E5M2, state[DGU], H)
        drows, dn = self._get("drows", (R, K), torch.bfloat16), self._get("dn", (T, K), torch.bfloat16)
        dw_gu, dw_down = torch.empty((E, 2 * F, K), device=dev), torch.empty((E, K, F), device=dev)
        sq.fp8_expert_gemm(qdgu, sq.E5M2, now[DGU], self.q_gate_up, sq.E4M3, self._w_steps[:E], sq.MN_MAJOR, plan, T, k, drows)
        sq.fp8_expert_wgrad(qdgu, sq.E5M2, now[DGU], qx, sq.E4M3, step[N], plan, T, k, dw_gu)
        sq.fp8_expert_wgrad(qdy, sq.E5M2, now[DY], qh, sq.E4M3, step[H_], plan, T, k, dw_down)
        sq.fp8_expert_combine(drows, plan, k, E, dn)
        dx, dgamma = torch.empty_like(x), torch.empty(K, device=dev)
        ws = self._get("ws_norm", (max(16, sq.fp8_rmsnorm_bwd_workspace_bytes(T, K)),), torch.uint8)
        sq.fp8_rmsnorm_bwd(dn, x, self.gamma, rstd, dx, dgamma, ws, dres=dy)
        return dx, dweights, dgamma, dw_gu, dw_down
