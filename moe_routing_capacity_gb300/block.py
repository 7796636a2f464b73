"""One training block around the MoE layer: the attention branch, the MoE
branch, the norms around both, and the clipping of their gradients.

    n1 = norm(h) w_pre1                        abi.norm_residual
    q, k, v = n1 W_qkv^T, turned               abi.matmul, abi.rotary
                                               (with head norms: abi.head_norm_rotary)
    b1 = attention(q, k, v) W_o^T              abi.attention, abi.matmul
    h2 = h + gate1 (norm(b1) w_post1),  n2 = norm(h2) w_pre2      (one call)
    b2 = MoE(n2)                               PooledWaveMoE.forward
    h3 = h2 + gate2 (norm(b2) w_post2)

``TrainingBlock`` owns its buffers (allocated once) and runs forward and
backward on one stream with no host synchronisation; the packed sequences of a
batch are given as ``cu_seqlens`` on the device.  Tokens of no sequence pass
the attention branch as zeros.
"""
from __future__ import annotations

import torch

from . import abi
from .workloads import _gen, _normal_bf16

BF, F32 = torch.bfloat16, torch.float32


def draw_block_weights(d_model, n_heads, n_kv_heads, head_dim, device="cpu", seed=0,
                       head_norm=False) -> dict:
    """Seeded weights: projections N(0, 1/fan_in), norms around 1, gates
    around 1/2, all bf16; with head_norm, w_q and w_k of the heads' norms."""
    dev = torch.device(device)
    n_qkv = (n_heads + 2 * n_kv_heads) * head_dim
    w = {"W_qkv": _normal_bf16((n_qkv, d_model), d_model ** -0.5, _gen(dev, seed, "W_qkv"), dev),
         "W_o": _normal_bf16((d_model, n_heads * head_dim), (n_heads * head_dim) ** -0.5,
                             _gen(dev, seed, "W_o"), dev)}
    for n, mean in (("w_pre1", 1.0), ("w_post1", 1.0), ("w_pre2", 1.0), ("w_post2", 1.0),
                    ("gate1", 0.5), ("gate2", 0.5)):
        w[n] = (mean + _normal_bf16((d_model,), 0.1, _gen(dev, seed, n), dev).float()).to(BF)
    if head_norm:
        for n in ("w_q", "w_k"):
            w[n] = (1.0 + _normal_bf16((head_dim,), 0.1, _gen(dev, seed, n), dev).float()).to(BF)
    return w


class TrainingBlock:
    """``layer``: the MoE branch (a PooledWaveMoE); ``weights``: as
    draw_block_weights gives them (with w_q and w_k, every query and key head is
    normalised before it is turned); ``table``: rotary angles [positions,
    rot_dim / 2, 2] fp32 (abi.rotary_table)."""

    def __init__(self, layer, weights, n_heads, n_kv_heads, head_dim, table, n_seqs,
                 interleaved=False, eps=1e-6):
        self.layer, self.table, self.interleaved, self.eps = layer, table, interleaved, eps
        self.T, self.d = layer.cfg.T, layer.cfg.d_model
        self.hq, self.hk, self.D = n_heads, n_kv_heads, head_dim
        dev = layer.device
        self.w = {n: t.to(dev).contiguous() for n, t in weights.items()}
        T, d, hq, hk, D = self.T, self.d, n_heads, n_kv_heads, head_dim
        e = lambda *s, dt=BF: torch.empty(s, dtype=dt, device=dev)  # noqa: E731
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.plan = abi.AttentionPlan(torch.zeros(n_seqs + 1, dtype=torch.int32, device=dev), T,
                                      hq, hk, D, self.status)
        self.pos = None
        self.n1, self.n2, self.h2, self.h3 = e(T, d), e(T, d), e(T, d), e(T, d)
        self.rstd = [e(T, dt=F32) for _ in range(4)]    # n1; b1 and n2; b2
        self.qkv = e(T, hq + 2 * hk, D)
        self.q, self.k, self.v = self.qkv[:, :hq], self.qkv[:, hq:hq + hk], self.qkv[:, hq + hk:]
        # the heads as attention reads them: in place of the projection's, but for the head
        # norms' gradient, which needs those
        self.head_norm = "w_q" in self.w
        if self.head_norm:
            self.qk = e(T, hq + hk, D)
            self.qa, self.ka = self.qk[:, :hq], self.qk[:, hq:]
        else:
            self.qa, self.ka = self.q, self.k
        self.att, self.rest, self.lse = e(T, hq, D), e(T, hq, D), e(hq, T, dt=F32)
        self.b1 = e(T, d)

    def set_batch(self, cu_seqlens, pos, stream=None):
        """The batch's sequences: cu_seqlens [sequences + 1] int32 and the
        tokens' positions [T] int32, both on the device."""
        self.plan.refill(cu_seqlens, stream)
        self.pos = pos

    def forward(self, h, stream=None):
        """h [T, d] bf16 -> h3 [T, d]; intermediates stay for backward()."""
        w, T, d, qd = self.w, self.T, self.d, self.hq * self.D
        self.h = h
        abi.norm_residual(None, h, None, None, w["w_pre1"], None, self.n1, None, self.rstd[0],
                          eps=self.eps, stream=stream)
        abi.matmul(self.n1, w["W_qkv"], T, (self.hq + 2 * self.hk) * self.D, d,
                   self.qkv.view(T, -1), self.status, stream=stream)
        if self.head_norm:
            abi.head_norm_rotary(self.q, self.k, w["w_q"], w["w_k"], self.table, self.pos,
                                 self.qa, self.ka, self.status, eps=self.eps,
                                 interleaved=self.interleaved, stream=stream)
        else:
            abi.rotary(self.q, self.k, self.table, self.pos, self.q, self.k, self.status,
                       interleaved=self.interleaved, stream=stream)
        abi.attention(self.plan, self.qa, self.ka, self.v, self.att, self.lse, self.status,
                      rest=self.rest, stream=stream)
        abi.matmul(self.att.view(T, qd), w["W_o"], T, d, qd, self.b1, self.status, stream=stream)
        abi.norm_residual(self.b1, h, w["gate1"], w["w_post1"], w["w_pre2"], self.h2, self.n2,
                          self.rstd[1], self.rstd[2], eps=self.eps, stream=stream)
        self.b2 = self.layer.forward(self.n2, stream=stream)
        abi.norm_residual(self.b2, self.h2, w["gate2"], w["w_post2"], None, self.h3, None,
                          self.rstd[3], None, eps=self.eps, stream=stream)
        return self.h3

    def backward(self, dh3, stream=None) -> dict:
        """Gradients of the last forward for dh3 [T, d] bf16: {"h": dh (bf16),
        every weight's in fp32, the MoE layer's under "moe."}."""
        w, T, d, hq, hk, D = self.w, self.T, self.d, self.hq, self.hk, self.D
        n_qkv, qd = (hq + 2 * hk) * D, hq * D
        if not hasattr(self, "g"):
            e = lambda *s, dt=F32: torch.empty(s, dtype=dt, device=self.layer.device)  # noqa: E731
            with abi.on_stream(stream):
                self.g = {n: e(*t.shape) for n, t in w.items()}
                self.g["h"] = e(T, d, dt=BF)
                self.db, self.dh2, self.dn1 = (e(T, d, dt=BF) for _ in range(3))
                self.datt, self.dqkv = e(T, hq, D, dt=BF), e(T, hq + 2 * hk, D, dt=BF)
                self.ws_norm = e(abi.norm_residual_workspace(T, d), dt=torch.uint8)
                if self.head_norm:
                    self.ws_heads = e(abi.head_norm_rotary_workspace(T, hq, hk, D), dt=torch.uint8)
                self.ws_att = e(max(1, self.plan.backward_ws_bytes), dt=torch.uint8)
        g = self.g
        abi.norm_residual_backward(None, dh3, self.b2, None, w["gate2"], w["w_post2"], None,
                                   self.rstd[3], None, self.db, self.dh2, g["gate2"],
                                   g["w_post2"], None, self.ws_norm, stream=stream)
        moe = self.layer.backward(self.n2, self.db, stream=stream)
        # dh takes the residual stream's gradient from here on
        abi.norm_residual_backward(moe["x"], self.dh2, self.b1, self.h, w["gate1"], w["w_post1"],
                                   w["w_pre2"], self.rstd[1], self.rstd[2], self.db, self.dh2,
                                   g["gate1"], g["w_post1"], g["w_pre2"], self.ws_norm,
                                   stream=stream)
        abi.matmul(self.db, w["W_o"], T, qd, d, self.datt.view(T, qd), self.status, b_mn=True,
                   stream=stream)
        abi.matmul(self.db, self.att.view(T, qd), d, qd, T, g["W_o"], self.status, a_mn=True,
                   b_mn=True, stream=stream)
        dq, dk, dv = self.dqkv[:, :hq], self.dqkv[:, hq:hq + hk], self.dqkv[:, hq + hk:]
        abi.attention_backward(self.plan, self.qa, self.ka, self.v, self.att, self.rest, self.lse,
                               self.datt, dq, dk, dv, self.ws_att, self.status, stream=stream)
        if self.head_norm:
            abi.head_norm_rotary_backward(dq, dk, self.q, self.k, w["w_q"], w["w_k"], self.table,
                                          self.pos, dq, dk, g["w_q"], g["w_k"], self.ws_heads,
                                          self.status, eps=self.eps, interleaved=self.interleaved,
                                          stream=stream)
        else:
            abi.rotary(dq, dk, self.table, self.pos, dq, dk, self.status,
                       interleaved=self.interleaved, inverse=True, stream=stream)
        flat = self.dqkv.view(T, n_qkv)
        abi.matmul(flat, w["W_qkv"], T, d, n_qkv, self.dn1, self.status, b_mn=True, stream=stream)
        abi.matmul(flat, self.n1, n_qkv, d, T, g["W_qkv"], self.status, a_mn=True, b_mn=True,
                   stream=stream)
        abi.norm_residual_backward(self.dn1, self.dh2, None, self.h, None, None, w["w_pre1"],
                                   None, self.rstd[0], None, g["h"], None, None, g["w_pre1"],
                                   self.ws_norm, stream=stream)
        g.update({"moe." + n: t for n, t in moe.items() if n != "x" and t.numel()})
        return g

    def clip(self, max_norm, norm, stream=None):
        """Scale the weights' gradients of the last backward in place to a
        global 2-norm of at most max_norm; norm [1] fp32 receives it."""
        if not hasattr(self, "grad_set"):
            self.grad_set = abi.GradSet([t for n, t in self.g.items() if n != "h"], stream=stream)
        abi.grad_clip(self.grad_set, max_norm, norm, stream)
