"""GPU tests of the training block's operators where other streams, refused
sequences, values that are not finite, empty batches and long work lists meet
them."""
import math

import pytest
import torch

import block_reference as R
from moe_routing_capacity_gb300 import abi

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture
def rng():
    return torch.Generator(device="cuda").manual_seed(11)


def randn(g, *s, std=1.0, dt=BF):
    return (torch.randn(s, generator=g, device="cuda") * std).to(dt)


def empty(*s, dt=BF):
    return torch.full(s, float("nan"), device="cuda", dtype=dt)


def ints(*v):
    return torch.tensor(v, device="cuda", dtype=torch.int32)


def status():
    return ints(0)


def attention_step(q, k, v, cu, dout, plan=None):
    """out, lse, dq, dk, dv, and the two calls' status words."""
    T, hq, D = q.shape
    hk = k.shape[1]
    plan = abi.AttentionPlan(ints(*cu), T, hq, hk, D) if plan is None else plan
    st = [status(), status()]
    got = {"out": empty(T, hq, D), "lse": empty(hq, T, dt=F32), "dq": empty(T, hq, D),
           "dk": empty(T, hk, D), "dv": empty(T, hk, D)}
    rest = empty(T, hq, D)
    abi.attention(plan, q, k, v, got["out"], got["lse"], st[0], rest=rest)
    ws = torch.empty(plan.backward_ws_bytes, device="cuda", dtype=torch.uint8)
    abi.attention_backward(plan, q, k, v, got["out"], rest, got["lse"], dout, got["dq"],
                           got["dk"], got["dv"], ws, st[1])
    return got, [int(s) for s in st]


# ------------------------------------------------------------------ refused sequences

@pytest.mark.parametrize("hq,hk", [(2, 1), (3, 1)])
def test_calls_on_refused_sequences_say_so(rng, hq, hk):
    """Nothing is written, and the calls' own status tells; sequences that
    are in order again are taken again."""
    T, D = 300, 64
    q, k, v, dout = (randn(rng, T, h, D) for h in (hq, hk, hk, hq))
    plan = abi.AttentionPlan(ints(0, 200, 100), T, hq, hk, D)
    assert int(plan.status) == abi.MOE_EINVAL
    got, st = attention_step(q, k, v, None, dout, plan)
    assert st == [abi.MOE_EINVAL, abi.MOE_EINVAL]
    for n, t in got.items():
        assert bool(t.isnan().all()), n
    plan.refill(ints(0, 200, 300))
    got, st = attention_step(q, k, v, None, dout, plan)
    assert st == [0, 0]
    want = R.attention(q, k, v, [200, 100], D ** -0.5, dout=dout)
    for n in ("out", "dq", "dk", "dv"):
        R.within(n, got[n], want[n][0], want[n][1] + 1e-30)
