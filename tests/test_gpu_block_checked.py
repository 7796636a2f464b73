"""The checked build (-DMOE_CHECK=1) on the training block and its operators: no
index check fires, the results equal the normal build's bit for bit, and an
entry of a plan that is none is recorded and skipped."""
import os

import pytest
import torch

from moe_routing_capacity_gb300 import abi, build

import test_gpu_block_edges as edges

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def checked_lib():
    if not os.path.exists(build.CHECK_LIB):
        build.build_checked()
    return abi.load_library(build.CHECK_LIB)


def step(lens, hq, hk, D):
    """One training block's forward, backward and clip, and one attention step
    with tokens of no sequence before and after; every result by name."""
    g = torch.Generator(device="cuda").manual_seed(2)
    blk, h = edges.tiny_block(hq, hk, D)
    blk.forward(h)
    got = {"g_" + n: t for n, t in blk.backward(edges.randn(g, *h.shape)).items()}
    got["norm"] = torch.empty(1, device="cuda")
    blk.clip(0.5, got["norm"])
    T = sum(lens) + 300
    cu = [150 + c for c in edges.offsets(lens)]
    q, k, v, dout = (edges.randn(g, T, n, D) for n in (hq, hk, hk, hq))
    att, st = edges.attention_step(q, k, v, cu, dout)
    assert st == [0, 0]
    torch.cuda.synchronize()
    return {**got, **att}, abi.lib().moe_check_status()


@pytest.mark.parametrize("lens,hq,hk,D", [([1, 300, 0, 129], 4, 2, 32), ([900, 1000, 1100], 12, 4, 64),
                                          ([257, 1000], 9, 3, 96)])
def test_checked_build_clean_and_identical(checked_lib, monkeypatch, lens, hq, hk, D):
    want, code = step(lens, hq, hk, D)
    want = {n: t.clone() for n, t in want.items()}
    assert code == 0
    monkeypatch.setattr(abi, "_lib", checked_lib)
    got, code = step(lens, hq, hk, D)
    assert code == 0, f"index check site {code} fired"
    for n, t in want.items():
        assert torch.equal(t.contiguous().view(torch.uint8), got[n].contiguous().view(torch.uint8)), n


def test_an_entry_that_is_none_is_recorded_and_skipped(checked_lib, monkeypatch):
    """A block past its sequence's end (all of its rows are, so that nothing
    would be written without the check either)."""
    monkeypatch.setattr(abi, "_lib", checked_lib)
    g = torch.Generator(device="cuda").manual_seed(2)
    T, D = 300, 64
    q, k, v = (edges.randn(g, T, 2, D) for _ in range(3))
    plan = abi.AttentionPlan(edges.ints(0, T), T, 2, 2, D)
    # group 1: tiles of 256 rows, whose list stands last
    entries = plan.plan[:plan.plan.numel() // 4 * 4].view(torch.int32)
    hits = [i for i in range(8, entries.numel() - 2)
            if entries[i:i + 4].tolist() == [0, T, 1, 0]]
    entries[hits[-1] + 2] = 7
    out, lse, st = edges.empty(T, 2, D), edges.empty(2, T, dt=edges.F32), edges.status()
    abi.attention(plan, q, k, v, out, lse, st)
    torch.cuda.synchronize()
    assert abi.lib().moe_check_status() == 1203 and abi.lib().moe_check_status() == 0
    assert bool(out[:256].isfinite().all()) and bool(out[256:].isnan().all())
