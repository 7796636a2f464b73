"""Host-side checks of head norms with rotation, the choice of experts, embedding
and the distillation loss (no GPU needed): struct mirrors, scratch sizes, and
refusals before anything touches the device."""
import ctypes
import math
import os

import pytest
import torch

from moe_routing_capacity_gb300 import abi
from moe_routing_capacity_gb300 import workloads as wl

from test_block_host import built_library, test_struct_mirrors_match_header as mirror  # noqa: F401

P, ODD = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008)
Q2, K2 = ctypes.c_void_p(0x20000), ctypes.c_void_p(0x30000)
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("struct,cls", [("moe_head_norm_t", abi.HeadNorm),
                                        ("moe_routing_t", abi.RoutingConfig),
                                        ("moe_embedding_t", abi.EmbeddingConfig),
                                        ("moe_distill_t", abi.Distill)])
def test_struct_mirrors(struct, cls, tmp_path):
    mirror(struct, cls, tmp_path)


def made(cls, base, kw):
    c = cls(*base)
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)


def heads(**kw):
    #       T  hq hk D  rot il eps   rows q_t  q_h k_t k_h qo      ko      dq      dk
    return made(abi.HeadNorm, (4, 2, 1, 64, 32, 0, 1e-6, 100, 192, 64, 192, 64, 128, 64, 64, 64,
                               128, 64, 64, 64), kw)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(hq=0), dict(hk=-1), dict(D=60), dict(D=8),
                                dict(D=520), dict(rot_dim=8), dict(rot_dim=80), dict(rot_dim=-16),
                                dict(interleaved=2), dict(eps=-1.0), dict(eps=math.nan),
                                dict(table_rows=0), dict(q_t=100), dict(q_h=32), dict(qo_t=64),
                                dict(k_t=0), dict(ko_t=4)])
def test_head_norm_refuses_sizes(kw):
    L = abi.lib()
    assert L.moe_head_norm_rotary(heads(**kw), *[P] * 9, None) == abi.MOE_EINVAL
    assert L.moe_head_norm_rotary_backward(heads(**kw), *[P] * 13, 1 << 40, P, None) == abi.MOE_EINVAL


def test_head_norm_refuses_pointers():
    L = abi.lib()
    good = [P, P, P, P, P, None, Q2, K2, P]   # q k w_q w_k table pos q_out k_out status
    for i, v in ((0, None), (0, ODD), (1, None), (2, None), (3, None), (4, None), (4, ODD),
                 (6, ODD), (7, None), (8, None)):
        a = list(good)
        a[i] = v
        assert L.moe_head_norm_rotary(heads(), *a, None) == abi.MOE_EINVAL, i
    # a table without a rotation, keys where there are none, in place with other strides
    assert L.moe_head_norm_rotary(heads(rot_dim=0), *good, None) == abi.MOE_EINVAL
    assert L.moe_head_norm_rotary(heads(hk=0), *good, None) == abi.MOE_EINVAL
    assert L.moe_head_norm_rotary(heads(), P, Q2, P, P, P, None, P, K2, P, None) == abi.MOE_EINVAL
    assert L.moe_head_norm_rotary(heads(T=0), *[None] * 9, None) == abi.MOE_OK


def test_head_norm_backward_refuses():
    L = abi.lib()
    need = abi.head_norm_rotary_workspace(4, 2, 1, 64)
    # dq dk q k w_q w_k table pos dq_out dk_out dw_q dw_k ws
    good = [P, P, Q2, Q2, P, P, P, None, K2, K2, P, P, P]
    assert L.moe_head_norm_rotary_backward(heads(), *good, need - 1, P, None) == abi.MOE_ENOSPC
    for i in (0, 1, 2, 3, 4, 5, 6, 8, 9, 10, 11, 12):
        a = list(good)
        a[i] = None
        assert L.moe_head_norm_rotary_backward(heads(), *a, need, P, None) == abi.MOE_EINVAL, i
    assert L.moe_head_norm_rotary_backward(heads(), *good, need, None, None) == abi.MOE_EINVAL
    a = list(good)
    a[8] = Q2                                   # over q, whose strides are others
    assert L.moe_head_norm_rotary_backward(heads(), *a, need, P, None) == abi.MOE_EINVAL
    assert L.moe_head_norm_rotary_backward(heads(dq_t=96), *good, need, P, None) == abi.MOE_EINVAL
    assert L.moe_head_norm_rotary_backward(heads(T=0), *[None] * 13, 0, None, None) == abi.MOE_OK
    v = ctypes.c_int64()
    for bad in ((-1, 2, 1, 64), (4, 0, 1, 64), (4, 2, -1, 64), (4, 2, 1, 20), (4, 2, 1, 1024)):
        assert L.moe_head_norm_rotary_workspace(*bad, ctypes.byref(v)) == abi.MOE_EINVAL


def routing(**kw):
    #       T  E   k score groups kept top renorm scale grad reserved
    return made(abi.RoutingConfig, (4, 48, 4, 1, 4, 2, 2, 1, 2.5, 0, 0), kw)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(n_experts=0), dict(n_experts=1028), dict(top_k=0),
                                dict(top_k=33), dict(top_k=25), dict(score=2), dict(n_groups=0),
                                dict(n_groups=5), dict(n_groups=48), dict(groups_kept=0),
                                dict(groups_kept=5), dict(group_top=0), dict(group_top=3),
                                dict(n_experts=4, top_k=2), dict(renorm=2), dict(scale=math.inf),
                                dict(grad_f32=2), dict(reserved=1),
                                dict(n_experts=1020, n_groups=17, groups_kept=3)])
def test_routing_refuses(kw):
    L = abi.lib()
    assert L.moe_router_select(routing(**kw), P, None, P, P, None) == abi.MOE_EINVAL
    assert L.moe_router_select_backward(routing(**kw), P, P, P, P, None) == abi.MOE_EINVAL


def test_routing_refuses_pointers():
    L = abi.lib()
    for i, v in ((0, None), (0, ODD), (1, ODD), (2, None), (3, ODD), (3, None)):
        a = [P, None, P, P]
        a[i] = v
        assert L.moe_router_select(routing(), *a, None) == abi.MOE_EINVAL, i
    for i in range(4):
        a = [P] * 4
        a[i] = None
        assert L.moe_router_select_backward(routing(), *a, None) == abi.MOE_EINVAL, i
    assert L.moe_router_select(routing(T=0), *[None] * 4, None) == abi.MOE_OK
    assert L.moe_router_select_backward(routing(T=0), *[None] * 4, None) == abi.MOE_OK


def test_routed_layer_refuses():
    L = abi.lib()
    cfg = wl.TINY
    c = abi.make_config(cfg)
    args = abi.BackwardArgs()
    rule = abi.Routing(cfg.n_experts, cfg.top_k, score="sigmoid")
    call = lambda r, ragged=0, logits=P: L.moe_layer_backward_routed(  # noqa: E731
        ctypes.byref(c), ragged, ctypes.byref(args), None if r is None else ctypes.byref(r), logits, None)
    assert call(None) == abi.MOE_EINVAL
    assert call(rule.config(cfg.T)) == abi.MOE_EINVAL                       # the layer's own pointers
    assert call(rule.config(cfg.T, True)) == abi.MOE_EINVAL
    assert call(rule.config(cfg.T), ragged=2) == abi.MOE_EINVAL
    assert call(rule.config(cfg.T), logits=None) == abi.MOE_EINVAL
    assert call(abi.Routing(cfg.n_experts, 1).config(cfg.T)) == abi.MOE_EINVAL
    assert L.moe_route_logits(ctypes.byref(c), P, P, P, P, None, P, None) == abi.MOE_EINVAL
    assert L.moe_route_logits(ctypes.byref(c), P, P, None, None, None, P, None) == abi.MOE_EINVAL
    assert L.moe_route_logits(ctypes.byref(c), ODD, P, None, P, None, P, None) == abi.MOE_EINVAL
    with pytest.raises(ValueError):
        abi.Routing(8, 2, score="tanh")


def embedding(**kw):
    return made(abi.EmbeddingConfig, (10, 50, 64, 0, 0, 0, 2.0, 0), kw)   # T V d tab out acc scale


@pytest.mark.parametrize("kw", [dict(T=-1), dict(T=1 << 31), dict(V=0), dict(V=1 << 31), dict(d=4),
                                dict(d=60), dict(d=65544), dict(table_f32=2), dict(out_f32=-1),
                                dict(accumulate=2), dict(scale=math.nan), dict(reserved=1)])
def test_embedding_refuses_sizes(kw):
    L = abi.lib()
    assert L.moe_embedding(embedding(**kw), P, P, P, P, None) == abi.MOE_EINVAL
    assert L.moe_embedding_backward(embedding(**kw), P, 1 << 40, P, P, None) == abi.MOE_EINVAL


def test_embedding_refuses_pointers_and_short_scratch():
    L = abi.lib()
    v = ctypes.c_int64()
    assert L.moe_embedding_workspace(10, 50, 64, ctypes.byref(v)) == abi.MOE_OK and v.value > 0
    for bad in ((-1, 50, 64), (10, 0, 64), (10, 50, 12)):
        assert L.moe_embedding_workspace(*bad, ctypes.byref(v)) == abi.MOE_EINVAL
    need = v.value
    for i, x in ((0, None), (0, ODD), (1, None), (2, ODD), (3, None)):
        a = [P, P, P, P]
        a[i] = x
        assert L.moe_embedding(embedding(), *a, None) == abi.MOE_EINVAL, i
    assert L.moe_embedding_plan(10, 50, 64, P, P, need - 1, P, None) == abi.MOE_ENOSPC
    for a in ([None, P, need, P], [P, None, need, P], [P, ODD, need, P], [P, P, need, None]):
        assert L.moe_embedding_plan(10, 50, 64, *a, None) == abi.MOE_EINVAL
    assert L.moe_embedding_plan(0, 50, 64, None, None, 0, None, None) == abi.MOE_OK
    assert L.moe_embedding_backward(embedding(), P, need - 1, P, P, None) == abi.MOE_ENOSPC
    for i in (0, 2, 3):
        a = [P, need, P, P]
        a[i] = None
        assert L.moe_embedding_backward(embedding(), *a, None) == abi.MOE_EINVAL, i
    assert L.moe_embedding(embedding(T=0), *[None] * 4, None) == abi.MOE_OK
    assert L.moe_embedding_backward(embedding(T=0, accumulate=1), None, 0, None, None, None) == abi.MOE_OK


def distill(**kw):
    return made(abi.Distill, (4, 100, 100, 104, 8, 0, 1, 2.0, 1.0, 0), kw)   # T V ld dld K zf tf tau s


@pytest.mark.parametrize("kw", [dict(T=-1), dict(V=0), dict(V=1 << 31), dict(K=0), dict(K=257),
                                dict(z_f32=2), dict(teacher_f32=2), dict(temperature=0.0),
                                dict(temperature=math.inf), dict(scale=math.nan), dict(reserved=1),
                                dict(z_ld=99), dict(z_ld=1 << 40)])
def test_distill_refuses_sizes(kw):
    L = abi.lib()
    assert L.moe_distill_loss(distill(**kw), P, P, P, None, P, P, None, None, P, None) == abi.MOE_EINVAL
    assert L.moe_distill_loss_backward(distill(**kw), P, P, P, None, P, Q2, P, None) == abi.MOE_EINVAL


def test_distill_refuses_pointers():
    L = abi.lib()
    odd = ctypes.c_void_p(0x10001)
    good = [P, P, P, None, P, P, None, None, P]   # z ids teacher weight loss lse total dlogits status
    for i, v in ((0, None), (0, odd), (1, None), (2, None), (4, None), (5, None), (7, odd), (7, P),
                 (8, None)):                      # dlogits over z with other strides
        a = list(good)
        a[i] = v
        assert L.moe_distill_loss(distill(), *a, None) == abi.MOE_EINVAL, i
    for i in (0, 1, 2, 4, 5, 6):
        a = [P, P, P, None, P, Q2, P]
        a[i] = None
        assert L.moe_distill_loss_backward(distill(), *a, None) == abi.MOE_EINVAL, i
    assert L.moe_distill_loss_backward(distill(dz_ld=50), P, P, P, None, P, Q2, P, None) == abi.MOE_EINVAL
    assert L.moe_distill_loss(distill(T=0), *[None] * 9, None) == abi.MOE_OK
    assert L.moe_distill_loss_backward(distill(T=0), *[None] * 7, None) == abi.MOE_OK


def test_python_argument_checks():
    t = lambda *s, dt=BF: torch.zeros(s, dtype=dt)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="positions"):
        abi.head_norm_rotary(t(4, 2, 64), None, t(64), None, t(8, 32), None, t(4, 2, 64), None, i(1))
    with pytest.raises(ValueError, match="pos"):
        abi.head_norm_rotary(t(4, 2, 64), None, t(64), None, t(8, 32, 2, dt=F32), i(3), t(4, 2, 64),
                             None, i(1))
    with pytest.raises(TypeError, match="q: expected"):
        abi.head_norm_rotary(t(4, 2, 64, dt=F32), None, t(64), None, None, None, t(4, 2, 64), None, i(1))
    with pytest.raises(ValueError, match="heads"):
        abi.head_norm_rotary(t(4, 128), None, t(64), None, None, None, t(4, 128), None, i(1))
    rule = abi.Routing(8, 2)
    with pytest.raises(TypeError, match="logits"):
        abi.router_select(rule, t(4, 8), None, i(4, 2), t(4, 2, dt=F32))
    with pytest.raises(ValueError, match="logits: shape"):
        abi.router_select(rule, t(4, 9, dt=F32), None, i(4, 2), t(4, 2, dt=F32))
    with pytest.raises(ValueError, match="table"):
        abi.embedding(t(50), i(4), t(4, 50), i(1))
    with pytest.raises(ValueError, match="ids"):
        abi.EmbeddingPlan(i(4, 2), 50, 64)
    with pytest.raises(TypeError, match="expected"):
        abi.embedding(t(50, 64, dt=torch.float16), i(4), t(4, 64), i(1))
    with pytest.raises(ValueError, match="logits is"):
        abi.distill_loss(t(4, 50, dt=torch.float16), i(4, 2), t(4, 2), None, t(4, dt=F32), t(4, dt=F32), i(1))
    with pytest.raises(ValueError, match="device tensor"):
        abi.distill_loss(t(4, 50), i(4, 2), t(4, 2), None, t(4, dt=F32), t(4, dt=F32), i(1))
    with pytest.raises(TypeError, match="dlogits"):
        abi._logits("dlogits", t(4, 50, dt=F32), (4, 50), BF)


def test_routed_layer_argument_checks():
    from moe_routing_capacity_gb300.layer import PooledWaveMoE
    with pytest.raises(ValueError, match="other sizes"):
        PooledWaveMoE(wl.TINY, {}, "cpu", routing=abi.Routing(8, 2))
