"""Distillation of many rows, where the threads a row follow its length alone (a warp and
more a row, in every mode), against the plain 64-bit implementation."""
import pytest
import torch

import model_reference as R
import test_gpu_model_ops as ops
from moe_routing_capacity_gb300 import abi

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
T = 2500    # more than 12 rows an SM


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("V", [900, 1100, 1500, 2049, 3001, 6000, 8191, 12000, 20001])
@pytest.mark.parametrize("shift,dz_shift", [(0, 0), (3, 6)])
def test_many_rows(dt, V, shift, dz_shift):
    """Loss alone, with the gradient, the gradient alone, and over the logits; rows that
    start where they may (one element apart from row to row where V is odd)."""
    g = torch.Generator(device="cuda").manual_seed(V + shift)
    K = 5
    z, ids, teacher, weight = ops.distill_inputs(g, T, V, K, dt, F32, V, shift)
    want = R.distill(z, ids, teacher, weight, 1.3, 0.7)
    kw = dict(temperature=1.3, scale=0.7)
    loss, lse, total, st = ops.empty(T, dt=F32), ops.empty(T, dt=F32), ops.empty(1, dt=F32), ops.status()
    abi.distill_loss(z, ids, teacher, weight, loss, lse, st, total=total, **kw)
    R.within("loss", loss, *want["loss"])
    R.within("lse", lse, *want["lse"])
    R.within("total", total, loss.double().sum().reshape(1), (T / 1024 + 12) * R.STEP * loss.double().abs().sum())
    x, b = want["dz"]
    bound = (1 + R.U) * b + R.round_of(dt) * x.abs()
    room = torch.full((T * V + 64,), 77.0, device="cuda", dtype=dt)
    dz = room[dz_shift:dz_shift + T * V].view(T, V)
    abi.distill_loss_backward(z, ids, teacher, weight, lse, dz, st, **kw)
    R.within("dz from lse", dz, x, bound)
    alone = dz.clone()
    dz.fill_(float("nan"))
    l2, e2 = ops.empty(T, dt=F32), ops.empty(T, dt=F32)
    abi.distill_loss(z, ids, teacher, weight, l2, e2, st, dlogits=dz, **kw)
    R.within("dz", dz, x, bound)
    R.within("loss with the gradient", l2, *want["loss"])
    R.within("lse with the gradient", e2, *want["lse"])
    both = dz.clone()
    assert bool((room[:dz_shift] == 77.0).all()) and bool((room[dz_shift + T * V:] == 77.0).all())
    was = z.clone()
    abi.distill_loss(z, ids, teacher, weight, l2, e2, st, dlogits=z, **kw)
    R.within("dz over the logits", z, x, bound)
    same = shift == dz_shift      # the same code for rows at the same places within 16 bytes
    assert not same or torch.equal(z, both)
    z.copy_(was)
    abi.distill_loss_backward(z, ids, teacher, weight, lse, z, st, **kw)
    R.within("dz over the logits from lse", z, x, bound)
    assert not same or torch.equal(z, alone)
    assert int(st) == 0
