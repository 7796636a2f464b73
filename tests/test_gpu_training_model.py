"""A training step from ids to loss and back (embedding, blocks with head norms and
a routing rule, head, distillation loss), and the layer under a routing rule."""
import math

import pytest
import torch

import model_reference as R
from moe_routing_capacity_gb300 import abi
from moe_routing_capacity_gb300 import workloads as wl
from moe_routing_capacity_gb300.block import TrainingBlock, draw_block_weights
from moe_routing_capacity_gb300.layer import HostPipeline, PooledWaveMoE
from moe_routing_capacity_gb300.model import TrainingModel, draw_model_weights

from test_gpu_training_block import rel

pytestmark = pytest.mark.gpu

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
RULE = dict(score="sigmoid", n_groups=4, groups_kept=2, group_top=2, scale=1.5)


def make_layer(cfg=wl.TINY, rule=RULE, bias=True, **kw):
    inp = wl.make_inputs(cfg, "cpu")
    if bias:
        inp["bias"] = torch.linspace(-0.02, 0.02, cfg.n_experts)
    return PooledWaveMoE(cfg, inp, "cuda", routing=abi.Routing(cfg.n_experts, cfg.top_k, **rule), **kw), inp


@pytest.mark.parametrize("kw", [dict(), dict(pipeline="shared"), dict(pipeline="waves"), dict(dropless=True),
                                dict(dropless=True, pipeline="shared"), dict(expert_bank=False)])
@pytest.mark.parametrize("rule", [RULE, dict(score="softmax", renorm=False, scale=3.0)])
def test_layer_under_a_rule(kw, rule):
    m, inp = make_layer(rule=rule, **kw)
    cfg, x = m.cfg, inp["x"].cuda()
    m.forward(x)
    g = torch.Generator(device="cuda").manual_seed(4)
    dout = torch.randn(cfg.T, cfg.d_model, generator=g, device="cuda").to(BF)
    got = m.backward(x, dout)
    torch.cuda.synchronize()
    assert int(m.status) == 0
    # logits as the product gives them, the choice and the weights as the rule does
    want = x.double() @ inp["Wr"].cuda().double().T
    R.within("logits", m.logits, want, 2.0 ** -16 * (x.double().abs() @ inp["Wr"].cuda().double().abs().T))
    idx, w = R.select(m.logits, m.w["bias"], m.routing)
    assert torch.equal(m.idx.long(), idx)
    R.within("w", m.gate_w, w, 128 * R.STEP * w)
    # dropped assignments have no part in the output, and no gradient
    dw = m.backward_intermediate("dw")[:cfg.T * cfg.top_k * 4].view(F32).view(cfg.T, cfg.top_k)
    dl, _ = R.select_backward(m.logits, idx, dw, m.routing)
    want = dl.T @ x.double()
    bound = (R.U + 2.0 ** -14) * (dl.abs().T @ x.double().abs())
    R.within("dWr", got["Wr"], want, bound + 2.0 ** -18 * bound.max())
    assert all(bool(t.isfinite().all()) for t in got.values())


def test_layer_under_the_layers_own_rule_is_the_layer():
    """Softmax scores renormalised over the chosen, without groups or bias, is what
    the layer does without a rule."""
    a, inp = make_layer(rule=dict(score="softmax"), bias=False)
    b = PooledWaveMoE(wl.TINY, wl.make_inputs(wl.TINY, "cpu"), "cuda")
    x = inp["x"].cuda()
    ya, yb = a.forward(x).clone(), b.forward(x).clone()
    assert torch.equal(a.idx, b.idx) and torch.equal(a.drop, b.drop)
    R.within("w", a.gate_w, b.gate_w.double(), 32 * R.STEP * b.gate_w.double())
    assert rel(ya, yb.double()) < 2.0 ** -9
    ga, gb = a.backward(x, x), b.backward(x, x)
    for n in ga:
        if ga[n].numel():
            assert rel(ga[n], gb[n].double()) < 2.0 ** -8, n
    a.route(x)
    assert torch.equal(a.idx, b.idx)


def test_a_rule_keeps_out_of_the_paths_that_do_not_take_it():
    m, _ = make_layer()
    with pytest.raises(ValueError, match="largest logits"):
        m.forward_native(torch.empty(wl.TINY.T, wl.TINY.d_model, device="cuda", dtype=BF))
    with pytest.raises(ValueError, match="largest logits"):
        HostPipeline(m)


def test_balance_bias_steers_a_rule():
    m, inp = make_layer(bias=False, balance_alpha=5.0)
    x = inp["x"].cuda()
    for _ in range(3):
        m.forward(x)
        idx, _ = R.select(m.logits, None if m.w["bias"] is None else bias_before(m), m.routing)
        assert torch.equal(m.idx.long(), idx)
        m._bias_before = m.w["bias"].clone()
    assert float(m.w["bias"].abs().max()) > 0


def bias_before(m):
    return getattr(m, "_bias_before", torch.zeros_like(m.w["bias"]))


def make_model(tied=False, n_blocks=2, vocab=264, head_norm=True, interleaved=False):
    cfg, hq, hk, D = wl.TINY, 4, 2, 32
    table = torch.empty(cfg.T, D // 2, 2, device="cuda")
    abi.rotary_table(table)
    blocks = []
    for i in range(n_blocks):
        layer, _ = make_layer(cfg.with_(seed=i))
        blocks.append(TrainingBlock(layer, draw_block_weights(cfg.d_model, hq, hk, D, seed=i, head_norm=head_norm),
                                    hq, hk, D, table, 2, interleaved=interleaved))
    w = draw_model_weights(cfg.d_model, vocab, seed=9, tied=tied)
    m = TrainingModel(blocks, w, embed_scale=math.sqrt(cfg.d_model))
    g = torch.Generator(device="cuda").manual_seed(5)
    ids = torch.randint(0, vocab, (cfg.T,), generator=g, device="cuda").to(I32)
    ids[::7] = 3
    ids[-6:] = -1
    cu = torch.tensor([0, 100, 250], device="cuda", dtype=I32)
    pos = torch.cat([torch.arange(100), torch.arange(156)]).to("cuda", I32)
    m.set_batch(ids, cu, pos)
    K = 8
    entries = torch.stack([torch.randperm(vocab, generator=g, device="cuda")[:K] for _ in range(cfg.T)]).to(I32)
    teacher = torch.randn(cfg.T, K, generator=g, device="cuda")
    weight = torch.ones(cfg.T, device="cuda")
    weight[250:] = 0
    return m, ids, entries, teacher, weight


@pytest.mark.parametrize("interleaved", [False, True])
def test_block_with_head_norms(interleaved):
    """The attention branch's heads and their weights' gradients from the block's own
    intermediates."""
    m, *_ = make_model(n_blocks=1, interleaved=interleaved)
    blk = m.blocks[0]
    g = torch.Generator(device="cuda").manual_seed(8)
    h = torch.randn(blk.T, blk.d, generator=g, device="cuda").to(BF)
    blk.forward(h)
    q, k = blk.q.clone(), blk.k.clone()
    for got, x, w in ((blk.qa, q, "w_q"), (blk.ka, k, "w_k")):
        R.within(w, got, *R.head_norm(x, blk.w[w], blk.table, blk.pos, blk.eps, interleaved))
    dq, dk, dv = (torch.empty(blk.T, n, blk.D, device="cuda", dtype=BF) for n in (blk.hq, blk.hk, blk.hk))
    got = blk.backward(h)
    abi.attention_backward(blk.plan, blk.qa, blk.ka, blk.v, blk.att, blk.rest, blk.lse, blk.datt, dq, dk, dv,
                           blk.ws_att, blk.status)
    for d, x, w, out in ((dq, q, "w_q", blk.dqkv[:, :blk.hq]), (dk, k, "w_k", blk.dqkv[:, blk.hq:blk.hq + blk.hk])):
        dx, dx_b, dw, dw_b = R.head_norm_backward(d, x, blk.w[w], blk.table, blk.pos, blk.eps, interleaved)
        R.within("d" + w, got[w], dw, dw_b)
        R.within("dx " + w, out, dx, dx_b)
    assert torch.equal(dv, blk.dqkv[:, blk.hq + blk.hk:])
    assert int(blk.status) == 0


@pytest.mark.parametrize("tied", [False, True])
def test_training_step(tied):
    m, ids, entries, teacher, weight = make_model(tied)
    z = m.forward().clone()
    n = m.n.double().requires_grad_()
    head = m.w["embed" if tied else "head"].double().requires_grad_()
    R.within("logits", z, (n @ head.T).detach(), (R.U + 2.0 ** -16) * (n.abs() @ head.abs().T).detach())
    got = m.step(entries, teacher, weight, scale=1.0 / 250)
    want = R.distill(z, entries, teacher, weight, 1.0, 1.0 / 250)
    R.within("loss", m.loss, *want["loss"])
    R.within("dz", m.z, want["dz"][0], (1 + R.U) * want["dz"][1] + R.U * want["dz"][0].abs())
    assert abs(float(m.total) - float(want["loss"][0].sum())) < 1e-5 * float(want["loss"][0].sum())
    # the two ends from the blocks' gradient, which the blocks' own tests check
    dz, dh = m.z.double(), m.blocks[0].g["h"]
    R.within("h0", m.h0, m.w["embed"].double()[ids.long().clamp(min=0)] * m.embed_scale * (ids >= 0)[:, None],
             (R.U + 2 * R.STEP) * m.h0.double().abs() * (1 + 2 * R.U) + 1e-30)
    dtable, mag, most = R.embedding_backward(ids, dh, m.vocab, m.embed_scale)
    dhead = dz.T @ n.detach()
    slack = 2.0 ** -16 * (dz.abs().T @ n.detach().abs())
    if tied:
        R.within("dembed", got["embed"], dtable + dhead, slack + (most + 4) * R.STEP * mag + 4 * R.STEP * dhead.abs())
    else:
        R.within("dembed", got["embed"], dtable, (most + 4) * R.STEP * mag)
        R.within("dhead", got["head"], dhead, slack)
    assert all(bool(t.isfinite().all()) for t in got.values())
    assert {f"blocks.{i}.{n}" for i in (0, 1) for n in ("w_q", "w_k", "W_qkv", "moe.Wr")} <= set(got)
    assert int(m.status) == 0 and all(int(b.status) == 0 for b in m.blocks)
    norm = torch.empty(1, device="cuda")          # all of them are a GradSet's tensors
    abi.grad_clip(abi.GradSet(list(got.values())), math.inf, norm)
    assert math.isfinite(float(norm)) and float(norm) > 0


def test_training_step_repeats_and_replays():
    m, ids, entries, teacher, weight = make_model()
    first = {n: t.clone() for n, t in m.step(entries, teacher, weight).items()}
    again = {n: t.clone() for n, t in m.step(entries, teacher, weight).items()}
    for n in first:
        assert torch.equal(first[n], again[n]), n
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.step(entries, teacher, weight)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = m.step(entries, teacher, weight)
    for t in got.values():
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for n in first:
        assert torch.equal(first[n], got[n]), n
