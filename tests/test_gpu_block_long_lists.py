"""The training block's operators where a CTA takes one piece of work after
another and a ring of rows or tiles is filled again and again: results against
plain 64-bit implementations, and the same bits as in calls too small for it."""
import pytest
import torch

import block_reference as R
import test_gpu_block_edges as edges
import test_gpu_block_ops as ops
from test_gpu_block_edges import rng  # noqa: F401

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32

# Several times as many pieces of work as a CTA an SM can take at once; blocks
# of one row, of 128 and of 129 next to long ones.
LENS = [100, 257, 1, 128, 640, 33, 0, 512, 129, 300, 90, 700, 5, 1100]


@pytest.mark.parametrize("hq,hk", [(32, 4), (18, 6), (16, 16)])
@pytest.mark.parametrize("D", [40, 64, 80, 128])
def test_attention_with_many_pieces_a_cta(rng, hq, hk, D):  # noqa: F811
    """Tokens of no sequence and a sequence of NaN among them; twice the same
    bits; a sequence alone, in a call of its own, gives the same bits."""
    first, T = 77, 77 + sum(LENS) + 200
    cu = [first + c for c in edges.offsets(LENS)]
    part = slice(first, cu[-1])
    q, k, v, dout = (edges.randn(rng, T, h, D) for h in (hq, hk, hk, hq))
    want = edges.reference(q[part], k[part], v[part], LENS, dout[part])
    for t in (q, k, v, dout):
        t[:first] = t[cu[-1]:] = float("inf")
        t[cu[9]:cu[10]] = float("nan")
    got, st = edges.attention_step(q, k, v, cu, dout)
    assert st == [0, 0]
    sick = torch.zeros(T, dtype=torch.bool, device="cuda")
    sick[cu[9]:cu[10]] = True
    for n in ("out", "dq", "dk", "dv"):
        assert not got[n][:first].any() and not got[n][cu[-1]:].any(), n
        assert bool(got[n][sick].isnan().all()), n
        keep = ~sick[part]
        R.within(n, got[n][part][keep], want[n][0][keep], want[n][1][keep] + 1e-30)
    keep = ~sick[part]
    w = want["lse"][0][:, keep]
    R.within("lse", got["lse"][:, part][:, keep], w, 1e-5 + 1e-5 * w.abs())
    again, _ = edges.attention_step(q, k, v, cu, dout)
    for n in got:
        assert torch.equal(got[n].view(torch.int16), again[n].view(torch.int16)), n
    one = slice(cu[11], cu[12])
    alone, _ = edges.attention_step(q[one], k[one], v[one], [0, LENS[11]], dout[one])
    for n in ("out", "dq"):
        assert torch.equal(got[n][one], alone[n]), n
    assert torch.equal(got["lse"][:, one], alone["lse"])


# rows past five times what the launch has under way: each ring slot is
# filled again, in either direction and in every shape of launch
NORM = [(30011, 64), (26001, 256), (13003, 264), (13001, 512), (7001, 1024), (3600, 1032),
        (3501, 2048), (2001, 2056), (1901, 4096), (1001, 6144), (1003, 8192)]


@pytest.mark.parametrize("T,d", NORM)
@pytest.mark.parametrize("gate,rt", [("none", BF), ("channel", BF), ("token", F32),
                                     ("channel", F32), ("token", BF)])
def test_norm_of_many_rows(rng, T, d, gate, rt):  # noqa: F811
    ops.test_norm_forward(rng, T, d, gate, rt)
    ops.test_norm_backward(rng, T, d, gate, rt)
