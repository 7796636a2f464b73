"""Choice of experts where a group has no logit above -inf (all of it masked): its value is
exact, and those of the others are told from it as from any other."""
import pytest
import torch

import model_reference as R
import test_gpu_model_ops as ops
from moe_routing_capacity_gb300 import abi

pytestmark = pytest.mark.gpu

F32, F64, I32 = torch.float32, torch.float64, torch.int32
INF = float("inf")


def choose(rule, logits, bias):
    T = logits.shape[0]
    idx, w = torch.full((T, rule.top_k), -1, device="cuda", dtype=I32), ops.empty(T, rule.top_k, dt=F32)
    abi.router_select(rule, logits, bias, idx, w)
    return idx.long()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("masked", [0, 1])
@pytest.mark.parametrize("kept", [1, 2])
@pytest.mark.parametrize("side,all_by", [(-1, 0.0), (1, 0.0), (-1, -4.0), (1, -4.0)])
def test_a_bias_next_to_another_groups_value(score, top, masked, kept, side, all_by):
    """The masked group's value is its biases', the fp32 value next below or above the
    other's exact value: the larger is kept, whichever way the other's fp32 value rounds.
    With two kept, a third group is far ahead of both.  all_by: a part of every bias."""
    per, groups = 8, kept + 1
    E = per * groups
    rule = abi.Routing(E, 3, score=score, n_groups=groups, groups_kept=kept, group_top=top)
    g = torch.Generator(device="cuda").manual_seed(10 * top + masked)
    mine = slice(per * (1 - masked), per * (2 - masked))
    for _ in range(40):
        logits = torch.full((4, E), -INF, device="cuda")
        logits[:, mine] = ops.randn(g, per, dt=F32)
        bias = torch.full((E,), all_by, device="cuda")
        if kept == 2:                               # two of its experts, the others below any
            logits[:, 2 * per:] = -30.0
            logits[:, 2 * per:2 * per + 2] = 3.0
            bias[2 * per:2 * per + 2] += 4.0
        value = float(R.scores(logits[:1], rule.score == 0)[0, mine].sort(descending=True)[0][:top].sum())
        value += top * all_by
        near = torch.tensor(value, dtype=F32)
        if (float(near) - value) * side <= 0:
            near = torch.nextafter(near, torch.tensor(side * INF))
        assert 0 < (float(near) - value) * side <= 2.0 ** -23 * abs(value)
        bias[per * masked:per * masked + top] = float(near) / top
        want, _ = R.select(logits, bias, rule)
        got = choose(rule, logits, bias)
        lost = masked if side < 0 else 1 - masked
        assert bool((want // per != lost).all())
        assert torch.equal(got, want), (value, float(near), got[0], want[0])


@pytest.mark.parametrize("score,low", [("softmax", -200.0), ("sigmoid", -200.0), ("sigmoid", -100.0)])
@pytest.mark.parametrize("none", [-INF, float("nan")])
@pytest.mark.parametrize("with_bias", [False, True])
def test_scores_that_fp32_does_not_hold_beat_none(score, low, none, with_bias):
    """Three groups: one masked (or NaN, the smallest value of all), one whose scores are
    positive but below what fp32 holds, one with ordinary logits; two are kept, and more
    experts chosen than the last has."""
    if score == "softmax" and none != none:
        pytest.skip("NaN takes the whole row's scores with it")
    E, per = 48, 16
    rule = abi.Routing(E, per + 4, score=score, n_groups=3, groups_kept=2, group_top=2)
    g = torch.Generator(device="cuda").manual_seed(3)
    logits = ops.randn(g, 40, E, dt=F32) * 0.5
    logits[:, :per] = none
    logits[:, per:2 * per] += low
    bias = torch.zeros(E, device="cuda") if with_bias else None
    got = choose(rule, logits, bias)
    assert bool((got >= per).all())
    want, _ = R.select(logits.masked_fill(logits.isnan(), -INF), bias, rule)
    assert torch.equal(got, want)


@pytest.mark.parametrize("score,low", [("softmax", -200.0), ("sigmoid", -200.0), ("sigmoid", -100.0)])
@pytest.mark.parametrize("none", [-INF, float("nan")])
@pytest.mark.parametrize("with_bias", [False, True])
def test_scores_that_fp32_does_not_hold_decide_the_groups(score, low, none, with_bias):
    """The same, with fewer chosen than the ordinary group has experts, of which but two are
    above those of the group with small scores."""
    if score == "softmax" and none != none:
        pytest.skip("NaN takes the whole row's scores with it")
    E, per = 48, 16
    rule = abi.Routing(E, 5, score=score, n_groups=3, groups_kept=2, group_top=2)
    g = torch.Generator(device="cuda").manual_seed(4)
    logits = ops.randn(g, 40, E, dt=F32) * 0.5
    logits[:, :per] = none
    logits[:, per:2 * per] += low
    logits[:, 2 * per + 2:] += 1.5 * low
    bias = torch.zeros(E, device="cuda") if with_bias else None
    got = choose(rule, logits, bias)
    want, _ = R.select(logits.masked_fill(logits.isnan(), -INF), bias, rule)
    assert torch.equal(got, want)
    assert bool(((got // per == 1).sum(1) == 3).all())
