"""Head norms where a group of lanes goes from item to item (several heads an item, several
items a group, query heads and then key heads), and of many heads, against the plain 64-bit
implementation."""
import pytest
import torch

import model_reference as R
import test_gpu_model_ops as ops
from moe_routing_capacity_gb300 import abi

from test_gpu_block_checked import checked_lib  # noqa: F401

pytestmark = pytest.mark.gpu

F32 = torch.float32

#          T     hq   hk   D    rot
# more than 80 heads: runs of neighbours that do not come out even (128 heads in 14 parts
# of 10, 81 in 10 of 9 on 152 SMs); then several items a group
ITEMS = [(2900, 128, 8, 128, 128), (1450, 128, 128, 128, 64), (4001, 81, 8, 128, 128), (300, 200, 3, 64, 64),
         (3, 1000, 1, 64, 32), (8192, 16, 4, 128, 128), (3000, 128, 8, 128, 128), (12001, 6, 2, 128, 64),
         (30011, 3, 1, 64, 64), (30000, 8, 8, 64, 64), (9001, 20, 0, 128, 0), (5003, 7, 5, 264, 16),
         (2503, 9, 3, 512, 512), (20001, 2, 3, 72, 48)]


def inputs(g, T, hq, hk, D, rot):
    """With some positions outside the table: (inputs, tokens whose position is)."""
    x = ops.head_inputs(g, T, hq, hk, D, rot)
    out = torch.zeros(T, dtype=torch.bool, device="cuda")
    if rot and T > 100:
        out = torch.rand(T, generator=g, device="cuda") < 0.01
        out[T - 1] = True
        x["pos"][out] = 50
        x["pos"][T // 2], out[T // 2] = -1, True
    return x, out


def lanes(D):
    units = (D + 15) // 16
    return next(n for n in (4, 8, 16, 32) if units <= n)


@pytest.mark.parametrize("T,hq,hk,D,rot", ITEMS)
@pytest.mark.parametrize("pairs", [False, True])
def test_forward(T, hq, hk, D, rot, pairs):
    g = torch.Generator(device="cuda").manual_seed(T + hq)
    x, out = inputs(g, T, hq, hk, D, rot)
    wide, st = ops.empty(T, hq + hk + 2, D), ops.status()
    ko = wide[:, hq + 1:hq + 1 + hk] if hk else None
    abi.head_norm_rotary(x["q"], x["k"], x["w_q"], x["w_k"], x["table"], x["pos"], wide[:, :hq], ko, st,
                         eps=1e-5, interleaved=pairs)
    assert int(st) == (abi.MOE_EINVAL if bool(out.any()) else 0)
    at = x["pos"].clamp(0, 49)
    for got, n in ((wide[:, :hq], "q"), (ko, "k")):
        if got is None:
            continue
        assert bool(got[out].isnan().all())
        want, bound = R.head_norm(x[n], x["w_" + n], x["table"], at, 1e-5, pairs)
        R.within(n, got[~out], want[~out], bound[~out])
    assert bool(wide[:, hq].isnan().all()) and bool(wide[:, -1].isnan().all())


@pytest.mark.parametrize("T,hq,hk,D,rot", ITEMS)
@pytest.mark.parametrize("pairs,in_place", [(False, False), (True, True)])
def test_backward(T, hq, hk, D, rot, pairs, in_place):
    """dw to the rounding of the sums as they are made: a group of lanes adds up its rows one
    after the other (all resident groups share T x heads rows in parts that differ by an item
    and by a factor of two at most: 2 T heads / groups + heads), a block its groups, 32 runs
    of blocks theirs, and then those."""
    g = torch.Generator(device="cuda").manual_seed(T + hk)
    x, out = inputs(g, T, hq, hk, D, rot)
    at = x["pos"].clamp(0, 49)
    groups = torch.cuda.get_device_properties(0).multi_processor_count * 2 * 256 // lanes(D)
    deep = 32 + (2 * T * (hq + hk) / groups + hq + hk) + 256 / lanes(D) + 10 + 32
    dy = {"q": ops.randn(g, T, hq, D), "k": ops.randn(g, T, hk, D) if hk else None}
    want = {}
    for n in "qk":
        if x[n] is not None:
            dx, dx_b, dw, dw_b = R.head_norm_backward(dy[n], x[n], x["w_" + n], x["table"], at, 1e-5, pairs, out)
            terms = 32 + T * x[n].shape[1]      # what its bound counts
            want[n] = dx, dx_b, dw, dw_b * min(1.0, deep / terms)
    res = {n: None if t is None else t if in_place else ops.empty(*t.shape) for n, t in dy.items()}
    before = {n: None if t is None else t[out].clone() for n, t in res.items()}
    dw = {"q": ops.empty(D, dt=F32), "k": ops.empty(D, dt=F32) if hk else None}
    ws = torch.empty(abi.head_norm_rotary_workspace(T, hq, hk, D), dtype=torch.uint8, device="cuda")
    st = ops.status()
    abi.head_norm_rotary_backward(dy["q"], dy["k"], x["q"], x["k"], x["w_q"], x["w_k"], x["table"], x["pos"],
                                  res["q"], res["k"], dw["q"], dw["k"], ws, st, eps=1e-5, interleaved=pairs)
    assert int(st) == (abi.MOE_EINVAL if bool(out.any()) else 0)
    for n, (dx, dx_b, w, w_b) in want.items():
        same = res[n][out].nan_to_num() == before[n].nan_to_num()
        assert bool(same.all())
        R.within("d" + n, res[n][~out], dx[~out], dx_b[~out])
        R.within("dw_" + n, dw[n], w, w_b)


def test_checked_build(checked_lib, monkeypatch):  # noqa: F811
    """No check of a head fires, and the outputs are the normal build's bit for bit."""
    def run():
        got = []
        for T, hq, hk, D, rot in ITEMS[:8]:
            x, _ = inputs(torch.Generator(device="cuda").manual_seed(T), T, hq, hk, D, rot)
            q, k, st = ops.empty(T, hq, D), ops.empty(T, hk, D), ops.status()
            abi.head_norm_rotary(x["q"], x["k"], x["w_q"], x["w_k"], x["table"], x["pos"], q, k, st)
            got += [q, k]
        torch.cuda.synchronize()
        return got, abi.lib().moe_check_status()

    want, code = run()
    assert code == 0
    monkeypatch.setattr(abi, "_lib", checked_lib)
    got, code = run()
    assert code == 0, f"index check site {code} fired"
    for a, b in zip(want, got):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
