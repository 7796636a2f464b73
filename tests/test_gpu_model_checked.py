"""The checked build (-DMOE_CHECK=1) on the training model and its operators: no index
check fires, the results equal the normal build's bit for bit, and a plan's entry that
is none is recorded and skipped."""
import pytest
import torch

from moe_routing_capacity_gb300 import abi

import test_gpu_model_ops as ops
from test_gpu_block_checked import checked_lib  # noqa: F401
from test_gpu_training_model import make_model

pytestmark = pytest.mark.gpu


def results():
    """A training step and each operator at sizes of every kernel; by name."""
    m, ids, entries, teacher, weight = make_model()
    got = {"step." + n: t for n, t in m.step(entries, teacher, weight).items()}
    g = torch.Generator(device="cuda").manual_seed(21)
    for T, hq, hk, D, rot in ((70, 4, 2, 64, 32), (9, 3, 1, 264, 16), (600, 12, 4, 128, 64)):
        x = ops.head_inputs(g, T, hq, hk, D, rot)
        q, k, st = ops.empty(T, hq, D), ops.empty(T, hk, D), ops.status()
        abi.head_norm_rotary(x["q"], x["k"], x["w_q"], x["w_k"], x["table"], x["pos"], q, k, st)
        dw = [ops.empty(D, dt=ops.F32) for _ in range(2)]
        ws = torch.empty(abi.head_norm_rotary_workspace(T, hq, hk, D), dtype=torch.uint8, device="cuda")
        dq, dk = ops.empty(T, hq, D), ops.empty(T, hk, D)
        abi.head_norm_rotary_backward(q, k, x["q"], x["k"], x["w_q"], x["w_k"], x["table"], x["pos"], dq, dk,
                                      *dw, ws, st)
        got.update({f"heads{D}.{i}": t for i, t in enumerate((q, k, dq, dk, *dw))})
    for T, E, k, groups, kept in ((300, 384, 8, 8, 4), (65, 100, 7, 5, 2), (9, 1024, 32, 1, 1)):
        rule = abi.Routing(E, k, score="sigmoid", n_groups=groups, groups_kept=kept, group_top=2)
        logits = ops.randn(g, T, E, dt=ops.F32)
        logits[:T // 2] = 0                       # rows that are settled in 64 bits
        idx, w, dl = torch.zeros(T, k, device="cuda", dtype=ops.I32), ops.empty(T, k, dt=ops.F32), ops.empty(T, E)
        abi.router_select(rule, logits, torch.zeros(E, device="cuda"), idx, w)
        abi.router_select_backward(rule, logits, idx, w, dl)
        got.update({f"route{E}.{i}": t for i, t in enumerate((idx, w, dl))})
    for T, V, d in ((20000, 3000, 96), (5000, 4, 1032), (300000, 100, 8)):
        words, dout = ops.words(g, T, V, "often"), ops.randn(g, T, d)
        table = ops.empty(V, d, dt=ops.F32)
        abi.embedding_backward(abi.EmbeddingPlan(words, V, d), dout, table)
        out, st = ops.empty(T, d), ops.status()
        abi.embedding(table, words, out, st)
        got.update({f"embed{T}.{i}": t for i, t in enumerate((table, out))})
    for T, V, K in ((33, 133, 5), (6, 3001, 16), (5, 16001, 40), (7, 50001, 50)):
        z, i, y, wt = ops.distill_inputs(g, T, V, K, ops.BF)
        loss, lse, dz, st = ops.empty(T, dt=ops.F32), ops.empty(T, dt=ops.F32), ops.empty(T, V), ops.status()
        abi.distill_loss(z, i, y, wt, loss, lse, st, dlogits=dz)
        got.update({f"distill{V}.{i}": t for i, t in enumerate((loss, lse, dz))})
    torch.cuda.synchronize()
    return got, abi.lib().moe_check_status()


def test_checked_build_clean_and_identical(checked_lib, monkeypatch):  # noqa: F811
    want, code = results()
    want = {n: t.clone() for n, t in want.items()}
    assert code == 0
    monkeypatch.setattr(abi, "_lib", checked_lib)
    got, code = results()
    assert code == 0, f"index check site {code} fired"
    for n, t in want.items():
        assert torch.equal(t.contiguous().view(torch.uint8), got[n].contiguous().view(torch.uint8)), n


def test_a_piece_of_no_word_is_recorded_and_skipped(checked_lib, monkeypatch):  # noqa: F811
    """A plan whose pieces name a word past the vocabulary: found in the plan by their
    values, changed there; nothing of them is written (to a word that no piece of a small
    plan names zeros are)."""
    monkeypatch.setattr(abi, "_lib", checked_lib)
    V, d = 50, 64
    ids = torch.arange(4, device="cuda", dtype=torch.int32) + 7
    plan = abi.EmbeddingPlan(ids, V, d)
    words = plan.plan[:plan.plan.numel() // 4 * 4].view(torch.int32)
    host = words.cpu()
    hits = [i for i in range(0, host.numel() - 4, 4)
            if 7 <= int(host[i]) < 11 and int(host[i + 2]) == 1 and int(host[i + 3]) == -1]
    assert len(hits) == 4
    words[hits[0]] = V + 3
    out = ops.empty(V, d, dt=ops.F32)
    abi.embedding_backward(plan, torch.ones(4, d, device="cuda", dtype=ops.BF), out)
    torch.cuda.synchronize()
    assert abi.lib().moe_check_status() == 1628 and abi.lib().moe_check_status() == 0
    skipped = int(host[hits[0]])
    want = torch.zeros_like(out)
    want[7:11] = 1
    want[skipped] = 0
    assert torch.equal(out, want)
