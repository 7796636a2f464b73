"""A training step from token ids to the loss and back: the embedding, training
blocks, the last norm, the head and the loss against a teacher's top logits.

    h0 = scale embed[ids]                      abi.embedding
    h  = blocks(h0)                            TrainingBlock
    z  = norm(h) w_norm head^T                 abi.norm_residual, abi.matmul
    loss = sum_t KL(teacher || softmax z)      abi.distill_loss (one entry: the cross
                                               entropy of a label)

``TrainingModel`` owns its buffers (allocated once) and runs a step on one
stream with no host synchronisation; the loss and the logits' gradient come from
one pass over the logits, whose place the gradient takes.
"""
from __future__ import annotations

import torch

from . import abi
from .workloads import _gen, _normal_bf16

BF, F32 = torch.bfloat16, torch.float32


def draw_model_weights(d_model, vocab, device="cpu", seed=0, tied=False) -> dict:
    """Seeded weights: embed [vocab, d] N(0, 1/d), w_norm around 1 and, unless it
    is tied to embed, head [vocab, d] N(0, 1/d), all bf16."""
    dev = torch.device(device)
    std = d_model ** -0.5
    w = {"embed": _normal_bf16((vocab, d_model), std, _gen(dev, seed, "embed"), dev),
         "w_norm": (1.0 + _normal_bf16((d_model,), 0.1, _gen(dev, seed, "w_norm"), dev).float()).to(BF)}
    if not tied:
        w["head"] = _normal_bf16((vocab, d_model), std, _gen(dev, seed, "head"), dev)
    return w


class TrainingModel:
    """``blocks``: TrainingBlocks of one size; ``weights``: as draw_model_weights
    gives them (without head, the head is embed).  The vocabulary is a multiple of
    8."""

    def __init__(self, blocks, weights, embed_scale=1.0, temperature=1.0, eps=1e-6):
        self.blocks = list(blocks)
        self.T, self.d = blocks[0].T, blocks[0].d
        dev = blocks[0].layer.device
        self.w = {n: t.to(dev).contiguous() for n, t in weights.items()}
        self.vocab = self.w["embed"].shape[0]
        self.tied = "head" not in self.w
        self.embed_scale, self.temperature, self.eps = embed_scale, temperature, eps
        T, d = self.T, self.d
        e = lambda *s, dt=BF: torch.empty(s, dtype=dt, device=dev)  # noqa: E731
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.plan = abi.EmbeddingPlan(torch.full((T,), -1, dtype=torch.int32, device=dev),
                                      self.vocab, d, self.status)
        self.ids = None
        self.batch = torch.empty(2, T, dtype=torch.int32, device=dev)   # its ids and positions
        self.h0, self.n, self.dn, self.dh = e(T, d), e(T, d), e(T, d), e(T, d)
        self.rstd = e(T, dt=F32)
        self.z = e(T, self.vocab)
        self.loss, self.lse, self.total = e(T, dt=F32), e(T, dt=F32), e(1, dt=F32)
        self.g = {n: e(*t.shape, dt=F32) for n, t in self.w.items()}
        self.ws_norm = e(abi.norm_residual_workspace(T, d), dt=torch.uint8)
        self.made = torch.cuda.Event()   # behind what was queued so far, a plan of no words among it
        self.made.record(torch.cuda.current_stream(dev))

    def set_batch(self, ids, cu_seqlens, pos, stream=None):
        """The batch: its tokens' ids [T] int32 (-1: none), packed sequences
        (cu_seqlens [sequences + 1]) and positions [T] (or None: 0, 1, ...), int32 on
        the device.  It is copied on the stream, so that a step looks up the words
        that its plan was made from whatever the caller's tensors hold by then."""
        if pos is not None:
            abi._rows("pos", pos, (self.T,), abi._I32)
        with abi.on_stream(stream):
            # the first batch's stream may be another than the model was made on (a capture
            # begins with the device idle)
            if self.made is not None and not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream(self.batch.device).wait_event(self.made)
                self.made = None
        self.plan.refill(ids, stream)
        with abi.on_stream(stream):
            self.batch[0].copy_(ids)
            if pos is not None:
                self.batch[1].copy_(pos)
        self.ids = self.batch[0]
        for b in self.blocks:
            b.set_batch(cu_seqlens, None if pos is None else self.batch[1], stream)

    def forward(self, stream=None):
        """Logits z [T, vocab] of the batch (the buffer that step() overwrites)."""
        abi.embedding(self.w["embed"], self.ids, self.h0, self.status, scale=self.embed_scale,
                      stream=stream)
        h = self.h0
        for b in self.blocks:
            h = b.forward(h, stream)
        self.h = h
        abi.norm_residual(None, h, None, None, self.w["w_norm"], None, self.n, None, self.rstd,
                          eps=self.eps, stream=stream)
        head = self.w["embed" if self.tied else "head"]
        abi.matmul(self.n, head, self.T, self.vocab, self.d, self.z, self.status, stream=stream)
        return self.z

    def step(self, teacher_ids, teacher, weight=None, scale=1.0, stream=None) -> dict:
        """One step's gradients for scale times the sum of the tokens' losses against
        the teacher's entries (abi.distill_loss): {"embed", "w_norm", "head", and
        "blocks.i.name" for each block}, weights' in fp32; the loss in total[0]."""
        w, T, d, V = self.w, self.T, self.d, self.vocab
        self.forward(stream)
        abi.distill_loss(self.z, teacher_ids, teacher, weight, self.loss, self.lse, self.status,
                         total=self.total, dlogits=self.z, temperature=self.temperature,
                         scale=scale, stream=stream)
        head, dhead = (w["embed"], self.g["embed"]) if self.tied else (w["head"], self.g["head"])
        abi.matmul(self.z, head, T, d, V, self.dn, self.status, b_mn=True, stream=stream)
        abi.matmul(self.z, self.n, V, d, T, dhead, self.status, a_mn=True, b_mn=True, stream=stream)
        abi.norm_residual_backward(self.dn, None, None, self.h, None, None, w["w_norm"], None,
                                   self.rstd, None, self.dh, None, None, self.g["w_norm"],
                                   self.ws_norm, stream=stream)
        got, dh = {}, self.dh
        for i in reversed(range(len(self.blocks))):
            g = self.blocks[i].backward(dh, stream)
            dh = g["h"]
            got.update({f"blocks.{i}.{n}": t for n, t in g.items() if n != "h"})
        # a tied table has the head's gradient already
        abi.embedding_backward(self.plan, dh, self.g["embed"], scale=self.embed_scale,
                               accumulate=self.tied, stream=stream)
        got.update(self.g)
        return got
