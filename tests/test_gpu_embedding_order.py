"""The embedding's gradient adds up in the order that it says, bit for bit, and its plan of
many tokens captured into a graph."""
import pytest
import torch

import test_gpu_model_ops as ops
from moe_routing_capacity_gb300 import abi

pytestmark = pytest.mark.gpu

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
PIECE = 32


def in_order(ids, dout, V, scale):
    """fp32: a word's tokens ascending, in pieces of 32 that are each added up one after the
    other; a word of several pieces is eight sums of every eighth piece, and then those."""
    ids, dout = ids.cpu().long(), dout.cpu().float()
    got = torch.zeros(V, dout.shape[1])
    for v in range(V):
        rows = dout[ids == v]
        n = rows.shape[0]
        if n == 0:
            continue
        pieces = (n + PIECE - 1) // PIECE
        rows = torch.cat((rows, torch.zeros(pieces * PIECE - n, dout.shape[1]))).view(pieces, PIECE, -1)
        sums = torch.zeros(pieces, dout.shape[1])
        for k in range(PIECE):
            sums = sums + rows[:, k]
        if pieces > 1:
            runs = torch.zeros(8, dout.shape[1])
            for j in range(0, pieces, 8):
                some = sums[j:j + 8]
                runs[:some.shape[0]] += some
            total = runs[0]
            for k in range(1, 8):
                total = total + runs[k]
        else:
            total = sums[0]
        got[v] = total * torch.tensor(scale, dtype=torch.float32)
    return got


@pytest.mark.parametrize("T,V,d", [(20, 3, 24), (1000, 7, 72), (1000, 300, 8), (5000, 3, 1040), (30000, 40, 72),
                                   (270000, 5, 8)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_sums_are_in_the_tokens_order(T, V, d, dt):
    """Values of sizes so different that another order gives another sum."""
    g = torch.Generator(device="cuda").manual_seed(T + V)
    ids = ops.words(g, T, V, "often")
    ids[torch.rand(T, generator=g, device="cuda") < 0.1] = -1
    size = 10.0 ** (8 * torch.rand(T, d, generator=g, device="cuda") - 4)
    dout = (torch.randn(T, d, generator=g, device="cuda") * size).to(dt)
    plan, got = abi.EmbeddingPlan(ids, V, d), ops.empty(V, d, dt=F32)
    abi.embedding_backward(plan, dout, got, scale=0.6)
    want = in_order(ids, dout, V, 0.6).cuda()
    assert torch.equal(got, want)
    if T > 1000:                                    # the values tell it
        other = in_order(ids.flip(0), dout.flip(0), V, 0.6).cuda()
        assert int((other != want).sum()) > V * d // 4


@pytest.mark.parametrize("T", [1500, 20000])
def test_a_plan_of_several_launches_captured_and_replayed(T):
    """refill and gradient in one graph on a stream of its own, replayed for other ids."""
    V, d = 300, 72
    g = torch.Generator(device="cuda").manual_seed(T)
    ids, dout = ops.words(g, T, V, "often"), ops.randn(g, T, d)
    plan, got = abi.EmbeddingPlan(ids, V, d), ops.empty(V, d, dt=F32)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        plan.refill(ids)
        abi.embedding_backward(plan, dout, got)
    for kind in ("often", "one", "none"):
        ids.copy_(ops.words(g, T, V, kind))
        want = ops.empty(V, d, dt=F32)
        abi.embedding_backward(abi.EmbeddingPlan(ids, V, d), dout, want)
        got.fill_(float("nan"))
        graph.replay()
        graph.replay()
        assert torch.equal(got, want)
    assert int(plan.status) == 0
