"""A training block (attention and MoE branch, their norms, rotary positions,
clipping) against a plain one in 64 bits."""
import math

import pytest
import torch

import block_reference as R
from moe_routing_capacity_gb300 import abi
from moe_routing_capacity_gb300 import workloads as wl
from moe_routing_capacity_gb300.block import TrainingBlock, draw_block_weights
from moe_routing_capacity_gb300.layer import PooledWaveMoE

pytestmark = pytest.mark.gpu


def plain(w, h, lens, table, pos, hq, hk, D, eps):
    """The attention branch and the first residual sum, differentiable."""
    T = h.shape[0]
    _, n1, _, _ = R.norm_forward(None, h, None, None, w["w_pre1"], 1.0, 1.0, eps)
    qkv = (n1 @ w["W_qkv"].T).view(T, hq + 2 * hk, D)
    rot = 2 * table.shape[1]
    cs = table.double()[pos.long()][:, None]

    def turn(x):
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        c, s = cs[..., 0], cs[..., 1]
        return torch.cat((a * c - b * s, b * c + a * s, x[..., rot:]), -1)

    q, k, v = turn(qkv[:, :hq]), turn(qkv[:, hq:hq + hk]), qkv[:, hq + hk:]
    out, at = [], 0
    for n in lens:
        sl = slice(at, at + n)
        at += n
        kk, vv = (t[sl].repeat_interleave(hq // hk, 1) for t in (k, v))
        s = torch.einsum("ihd,jhd->hij", q[sl], kk) * D ** -0.5
        s = s.masked_fill(~torch.ones(n, n, dtype=torch.bool, device=h.device).tril(), -math.inf)
        out.append(torch.einsum("hij,jhd->ihd", torch.softmax(s, -1), vv))
    b1 = torch.cat(out).reshape(T, hq * D) @ w["W_o"].T
    h2, n2, _, _ = R.norm_forward(b1, h, w["gate1"], w["w_post1"], w["w_pre2"], 1.0, 1.0, eps)
    return h2, n2


def rel(got, want):
    return float((got.double() - want).norm() / want.norm())


def test_training_block_forward_backward_clip():
    cfg = wl.TINY
    T, d, hq, hk, D = cfg.T, cfg.d_model, 4, 2, 32
    lens = [100, 1, 155]
    inp = wl.make_inputs(cfg, "cpu")
    layer = PooledWaveMoE(cfg, inp, "cuda")
    w = draw_block_weights(d, hq, hk, D, seed=3)
    table = torch.empty(160, D // 2, 2, device="cuda")
    abi.rotary_table(table)
    blk = TrainingBlock(layer, w, hq, hk, D, table, len(lens))
    cu = torch.tensor([0, 100, 101, 256], device="cuda", dtype=torch.int32)
    pos = torch.cat([torch.arange(n) for n in lens]).to("cuda", torch.int32)
    blk.set_batch(cu, pos)
    h = inp["x"].cuda()
    g = torch.Generator(device="cuda").manual_seed(1)
    dh3 = torch.randn(T, d, generator=g, device="cuda").to(torch.bfloat16)
    h3 = blk.forward(h)
    got = blk.backward(dh3)
    assert int(blk.status) == 0 and int(layer.status) == 0

    w64 = {n: t.cuda().double().requires_grad_() for n, t in w.items()}
    h64 = h.double().requires_grad_()
    h2, n2 = plain(w64, h64, lens, table, pos, hq, hk, D, 1e-6)
    # five bf16 roundings on the way to h2 and n2, each at most 2^-8
    assert rel(blk.h2, h2.detach()) < 5 * R.U and rel(blk.n2, n2.detach()) < 5 * R.U
    # the MoE branch as the layer gave it (its own tests check it)
    b2, dn2 = blk.b2.double(), layer.grads["x"].double()
    y, _, _, _ = R.norm_forward(b2, h2, w64["gate2"], w64["w_post2"], None, 1.0, 1.0, 1e-6)
    assert rel(h3, y.detach()) < 6 * R.U
    loss = (y * dh3.double()).sum() + (n2 * dn2).sum()
    names = list(w64)
    want = dict(zip(names + ["h"], torch.autograd.grad(loss, [w64[n] for n in names] + [h64])))
    for n, t in want.items():
        # the gradients pass about ten such roundings
        assert rel(got[n], t) < 10 * R.U, (n, rel(got[n], t))

    tensors = {n: t for n, t in got.items() if n != "h"}
    total = math.sqrt(sum(float(t.double().square().sum()) for t in tensors.values()))
    before = {n: t.clone() for n, t in tensors.items()}
    norm = torch.empty(1, device="cuda")
    blk.clip(0.25 * total, norm)
    assert abs(float(norm) - total) <= 1e-6 * total
    for n, t in tensors.items():
        R.within(n, t, before[n].double() * 0.25, 1e-5 * before[n].double().abs())


def test_training_block_repeats_bit_for_bit():
    cfg = wl.TINY
    inp = wl.make_inputs(cfg, "cpu")
    layer = PooledWaveMoE(cfg, inp, "cuda")
    table = torch.empty(256, 16, 2, device="cuda")
    abi.rotary_table(table, scaling="linear", factor=2.0)
    blk = TrainingBlock(layer, draw_block_weights(cfg.d_model, 3, 1, 64), 3, 1, 64, table, 1)
    blk.set_batch(torch.tensor([0, 250], device="cuda", dtype=torch.int32), None)
    h = inp["x"].cuda()
    runs = []
    for _ in range(2):
        h3 = blk.forward(h).clone()
        g = {n: t.clone() for n, t in blk.backward(h).items()}
        runs.append({"h3": h3, **g})
    for n in runs[0]:
        assert torch.equal(runs[0][n], runs[1][n]), n
    assert int(blk.status) == 0
