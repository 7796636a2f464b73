"""GPU parity of head norms with rotation, the choice of experts, embedding and
the distillation loss against plain 64-bit implementations, at the sizes,
layouts and values where each can go wrong."""
import math

import pytest
import torch

import model_reference as R
from moe_routing_capacity_gb300 import abi

pytestmark = pytest.mark.gpu

BF, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32


@pytest.fixture
def rng():
    return torch.Generator(device="cuda").manual_seed(11)


def randn(g, *s, std=1.0, dt=BF):
    return (torch.randn(s, generator=g, device="cuda") * std).to(dt)


def empty(*s, dt=BF):
    return torch.full(s, float("nan"), device="cuda", dtype=dt)


def status():
    return torch.zeros(1, device="cuda", dtype=I32)


def ints(g, lo, hi, *s):
    return torch.randint(lo, hi, s, generator=g, device="cuda").to(I32)


# ------------------------------------------------------------------ head norms

def angles(rows, rot, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    a = torch.rand(rows, rot // 2, generator=g, device="cuda", dtype=F64) * 2 * math.pi
    return torch.stack((a.cos(), a.sin()), -1).float()


#          T    hq hk D    rot
HEADS = [(1, 1, 0, 16, 16), (1, 16, 4, 128, 128), (3, 5, 1, 24, 16), (70, 4, 2, 64, 32),
         (33, 3, 3, 80, 80), (257, 6, 1, 96, 48), (130, 2, 2, 256, 128), (9, 3, 1, 264, 16),
         (5, 2, 1, 512, 512), (600, 12, 4, 128, 64), (40, 4, 2, 40, 0), (2000, 1, 1, 72, 64)]


def head_inputs(g, T, hq, hk, D, rot):
    qkv = randn(g, T, hq + 2 * hk + 1, D, std=1.5)      # a token's heads among others
    x = {"q": qkv[:, :hq], "w_q": 1 + randn(g, D, std=0.2), "w_k": None, "k": None}
    if hk:
        x.update(k=qkv[:, hq:hq + hk], w_k=1 + randn(g, D, std=0.2))
    x["table"] = angles(50, rot) if rot else None
    x["pos"] = ints(g, 0, 50, T)
    return x


@pytest.mark.parametrize("T,hq,hk,D,rot", HEADS)
@pytest.mark.parametrize("pairs", [False, True])
def test_head_norm_forward(rng, T, hq, hk, D, rot, pairs):
    x = head_inputs(rng, T, hq, hk, D, rot)
    wide = empty(T, hq + hk + 2, D)                       # outputs among others too
    st = status()
    ko = wide[:, hq + 1:hq + 1 + hk] if hk else None
    abi.head_norm_rotary(x["q"], x["k"], x["w_q"], x["w_k"], x["table"], x["pos"], wide[:, :hq], ko,
                         st, eps=1e-5, interleaved=pairs)
    assert int(st) == 0
    for got, name in ((wide[:, :hq], "q"), (ko, "k")):
        if got is not None:
            R.within(name, got, *R.head_norm(x[name], x["w_" + name], x["table"], x["pos"], 1e-5, pairs))
    assert bool(wide[:, hq].isnan().all()) and bool(wide[:, -1].isnan().all())
    # in place, and positions 0, 1, ...
    if T <= 50:
        q, k = x["q"].clone(), None if not hk else x["k"].clone()
        abi.head_norm_rotary(q, k, x["w_q"], x["w_k"], x["table"], None, q, k, st, eps=1e-5, interleaved=pairs)
        at = torch.arange(T, device="cuda")
        R.within("in place", q, *R.head_norm(x["q"], x["w_q"], x["table"], at, 1e-5, pairs))


@pytest.mark.parametrize("T,hq,hk,D,rot", HEADS)
@pytest.mark.parametrize("pairs,place", [(False, "new"), (True, "dy"), (False, "dy"), (True, "x")])
def test_head_norm_backward(rng, T, hq, hk, D, rot, pairs, place):
    x = head_inputs(rng, T, hq, hk, D, rot)
    dy = {"q": randn(rng, T, hq, D), "k": randn(rng, T, hk, D) if hk else None}
    want = {n: R.head_norm_backward(dy[n], x[n], x["w_" + n], x["table"], x["pos"], 1e-5, pairs)
            for n in "qk" if x[n] is not None}
    src = {n: (t if place != "x" or t is None else t.clone()) for n, t in (("q", x["q"]), ("k", x["k"]))}
    out = {n: None if t is None else empty(*t.shape) if place == "new" else t
           for n, t in (dy if place != "x" else src).items()}
    dw = {"q": empty(D, dt=F32), "k": empty(D, dt=F32) if hk else None}
    st = status()
    ws = torch.empty(abi.head_norm_rotary_workspace(T, hq, hk, D), dtype=torch.uint8, device="cuda")
    abi.head_norm_rotary_backward(dy["q"], dy["k"], src["q"], src["k"], x["w_q"], x["w_k"], x["table"],
                                  x["pos"], out["q"], out["k"], dw["q"], dw["k"], ws, st, eps=1e-5,
                                  interleaved=pairs)
    assert int(st) == 0
    for n, (dx, dx_b, w, w_b) in want.items():
        R.within("d" + n, out[n], dx, dx_b)
        R.within("dw_" + n, dw[n], w, w_b)


def test_head_norm_gradient_is_that_of_differences(rng):
    """In 64 bits, the formula of the backward against central differences."""
    T, h, D, rot = 2, 1, 16, 16
    x, w, dy = (randn(rng, *s, dt=F64) for s in ((T, h, D), (D,), (T, h, D)))
    table, pos = angles(9, rot), ints(rng, 0, 9, T)
    dx, _, dw, _ = R.head_norm_backward(dy, x, w, table, pos, 1e-5, False)
    f = lambda x, w: float((R.head_norm(x, w, table, pos, 1e-5, False)[0] * dy).sum())  # noqa: E731
    step = 1e-5
    for t, g, at in ((x, dx, (0, 0, 3)), (x, dx, (1, 0, 15)), (w, dw, (5,))):
        d = torch.zeros_like(t)
        d[at] = step
        hi, lo = (f(x + d, w), f(x - d, w)) if t is x else (f(x, w + d), f(x, w - d))
        assert abs((hi - lo) / (2 * step) - float(g[at])) < 1e-7 * max(1, abs(float(g[at])))


@pytest.mark.parametrize("backward", [False, True])
def test_head_norm_bad_positions(rng, backward):
    T, hq, hk, D = 37, 3, 1, 64
    x = head_inputs(rng, T, hq, hk, D, 64)
    x["pos"][[4, 20]] = torch.tensor([-1, 50], device="cuda", dtype=I32)
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    bad[[4, 20]] = True
    x["pos"] = x["pos"].contiguous()
    fine = x["pos"].clamp(0, 49)
    qo, ko, st = empty(T, hq, D), empty(T, hk, D), status()
    if not backward:
        abi.head_norm_rotary(x["q"], x["k"], x["w_q"], x["w_k"], x["table"], x["pos"], qo, ko, st)
        want = R.head_norm(x["q"], x["w_q"], x["table"], fine, 1e-6, False)
    else:
        dq, dk, dwq, dwk = randn(rng, T, hq, D), randn(rng, T, hk, D), empty(D, dt=F32), empty(D, dt=F32)
        ws = torch.empty(abi.head_norm_rotary_workspace(T, hq, hk, D), dtype=torch.uint8, device="cuda")
        abi.head_norm_rotary_backward(dq, dk, x["q"], x["k"], x["w_q"], x["w_k"], x["table"], x["pos"],
                                      qo, ko, dwq, dwk, ws, st)
        want = R.head_norm_backward(dq, x["q"], x["w_q"], x["table"], fine, 1e-6, False, bad)
        R.within("dw_q", dwq, *want[2:])
    assert int(st) == abi.MOE_EINVAL
    assert bool(qo[bad].isnan().all()) and bool(ko[bad].isnan().all())
    R.within("others", qo[~bad], want[0][~bad], want[1][~bad])


def test_head_norm_zero_rows_and_infinities(rng):
    T, D = 6, 64
    q = randn(rng, T, 2, D)
    q[1, 0] = 0
    q[3, 1, 5] = float("inf")
    out, st = empty(T, 2, D), status()
    w = torch.ones(D, device="cuda", dtype=BF)
    abi.head_norm_rotary(q, None, w, None, angles(9, 64), None, out, None, st)
    assert bool((out[1, 0] == 0).all())
    ok = torch.ones(T, 2, dtype=torch.bool, device="cuda")
    ok[3, 1] = False
    assert bool(out[ok].isfinite().all()) and bool(out[3, 1].isnan().any())


# ------------------------------------------------------------------ choice of experts

#          T    E    k  groups kept top
RULES = [(1, 1, 1, 1, 1, 1), (5, 24, 2, 1, 1, 1), (300, 384, 8, 8, 4, 2), (70, 384, 8, 1, 1, 1),
         (33, 48, 6, 3, 2, 1), (65, 100, 7, 5, 2, 2), (64, 32, 4, 32, 7, 1), (9, 1024, 32, 1, 1, 1),
         (21, 1023, 16, 1, 1, 1), (40, 992, 32, 31, 9, 2), (17, 64, 32, 4, 2, 2), (50, 16, 16, 2, 2, 2),
         (8, 512, 8, 2, 1, 2), (12, 768, 5, 3, 2, 2)]


@pytest.mark.parametrize("T,E,k,groups,kept,top", RULES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias,renorm", [(True, True), (False, False), (True, False), (False, True)])
def test_router_select(rng, T, E, k, groups, kept, top, score, bias, renorm):
    rule = abi.Routing(E, k, score=score, n_groups=groups, groups_kept=kept, group_top=top,
                       renorm=renorm, scale=1.7)
    logits = randn(rng, T, E, std=1.5, dt=F32)
    b = randn(rng, E, std=0.1 if score == "sigmoid" else 0.5 / E, dt=F32) if bias else None
    idx, w = torch.full((T, k), -7, device="cuda", dtype=I32), empty(T, k, dt=F32)
    abi.router_select(rule, logits, b, idx, w)
    want, want_w = R.select(logits, b, rule)
    assert torch.equal(idx.long(), want)
    # fast exponentials in the row's sum: 16 steps and 2 of the largest argument; the rest less
    R.within("w", w, want_w, (64 + 4 * 12 + E / 16) * R.STEP * want_w.abs())
    dw = randn(rng, T, k, dt=F32)
    ref, mag = R.select_backward(logits, want, dw, rule)
    for dt in (BF, F32):
        dl = empty(T, E, dt=dt)
        abi.router_select_backward(rule, logits, idx, dw, dl)
        R.within("dlogits", dl, ref, R.round_of(dt) * ref.abs() + (128 + E / 16) * R.STEP * (1 + R.U) * mag)
        if renorm:
            assert int((dl != 0).sum()) <= T * k


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,kept,top", [(1, 1, 1), (4, 2, 1), (4, 2, 2), (8, 3, 2)])
@pytest.mark.parametrize("bias", ["none", "zero", "steps"])
def test_router_select_ties(rng, score, groups, kept, top, bias):
    """Logits of few values, biases of few steps, rows of one value: equal ones go
    to the lowest expert, and groups likewise."""
    T, E, k = 400, 96, 6
    rule = abi.Routing(E, k, score=score, n_groups=groups, groups_kept=kept, group_top=top)
    logits = ints(rng, -2, 3, T, E).float()
    logits[:50] = logits[:50, :1]
    b = {"none": None, "zero": torch.zeros(E, device="cuda"),
         "steps": ints(rng, -3, 4, E).float() * 2.0 ** -10}[bias]
    idx, w = torch.empty(T, k, device="cuda", dtype=I32), empty(T, k, dt=F32)
    abi.router_select(rule, logits, b, idx, w)
    want, want_w = R.select(logits, b, rule)
    clear = R.told_apart(logits, b, rule)
    assert int(clear.sum()) > T // 2
    assert torch.equal(idx.long()[clear], want[clear])
    R.within("w", w[clear], want_w[clear], 128 * R.STEP * want_w[clear])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_router_select_near_ties(rng, score):
    """Logits one step of fp32 apart, and biases that undo a score's lead to within
    2^-30: the order of the exact values, which fp32 cannot tell."""
    T, E, k = 3000, 64, 8
    rule = abi.Routing(E, k, score=score, n_groups=4, groups_kept=3, group_top=2)
    logits = randn(rng, T, E, dt=F32) * 0.01
    near = ints(rng, 0, 4, T, E).float()
    logits = (1.0 + near * 2.0 ** -23).contiguous()
    b = (ints(rng, -2, 3, E).float() * 2.0 ** -30).contiguous()
    for bb in (None, b):
        idx, w = torch.empty(T, k, device="cuda", dtype=I32), empty(T, k, dt=F32)
        abi.router_select(rule, logits, bb, idx, w)
        s = R.scores(logits, rule.score == 0)
        v = s if bb is None else s + bb.double()
        got = v.gather(1, idx.long())
        want = v.gather(1, R.select(logits, bb, rule)[0])
        # where 64 bits cannot tell either, any of the equal ones
        assert float((got - want).abs().max()) <= 2.0 ** -51


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("k", [6, 32])
def test_router_select_scores_that_64_bits_round_to_one(rng, score, k):
    """Without a bias the logits decide, in the groups as well, also where more experts
    than a warp has lanes reach the k-th logit (several of the same)."""
    T, E = 300, 960
    rule = abi.Routing(E, k, score=score, n_groups=16, groups_kept=6, group_top=1)
    logits = (randn(rng, T, E, dt=F32) * 4).round() * 10.0
    idx, w = torch.empty(T, k, device="cuda", dtype=I32), empty(T, k, dt=F32)
    abi.router_select(rule, logits, None, idx, w)
    want, want_w = R.select(logits, None, rule)
    assert torch.equal(idx.long(), want)
    R.within("w", w, want_w, 128 * R.STEP * want_w + 2.0 ** -120)


def test_router_select_values_that_are_not_finite(rng):
    """Always k different experts; masked experts (-inf) come last; NaN counts as
    the smallest; the weights of rows without NaN are as ever."""
    T, E, k = 64, 40, 5
    for score in ("softmax", "sigmoid"):
        for groups, kept in ((1, 1), (4, 2)):
            for with_bias in (False, True):
                rule = abi.Routing(E, k, score=score, n_groups=groups, groups_kept=kept, group_top=2)
                logits = randn(rng, T, E, dt=F32)
                logits[0] = float("nan")
                logits[1, 3] = float("nan")
                logits[2] = -float("inf")
                logits[3, 4:] = -float("inf")          # fewer than k that can be chosen
                logits[4, :30] = -float("inf")
                logits[5, 7] = float("inf")
                logits[6] = 1e30
                logits[7] = -1e30
                b = randn(rng, E, std=0.01, dt=F32) if with_bias else None
                idx, w = torch.full((T, k), -1, device="cuda", dtype=I32), empty(T, k, dt=F32)
                abi.router_select(rule, logits, b, idx, w)
                s = idx.sort(1)[0]
                assert bool((idx >= 0).all()) and bool((idx < E).all())
                assert bool((s[:, 1:] > s[:, :-1]).all())
                rest = torch.arange(T, device="cuda") >= 8
                want, ww = R.select(logits[rest], b, rule)
                assert torch.equal(idx[rest].long(), want)
                R.within("w", w[rest], ww, 128 * R.STEP * ww)
                if score == "sigmoid" and not with_bias:
                    assert 3 not in idx[1].tolist()
                if groups == 1:
                    assert set(range(4)) <= set(idx[3].tolist())
                    assert bool((idx[4] >= 30).all())
                # the gradient stays in its row
                dl = empty(T, E, dt=F32)
                abi.router_select_backward(rule, logits, idx, randn(rng, T, k, dt=F32), dl)
                assert bool(dl[rest].isfinite().all())


@pytest.mark.parametrize("E", [40, 41])
@pytest.mark.parametrize("bias", [False, True])
def test_router_select_shares_of_small_scores(rng, E, bias):
    """Sigmoids that fp32 does not hold have shares all the same, as long as 64 bits
    hold them, and those have gradients."""
    T, k = 40, 6
    rule = abi.Routing(E, k, score="sigmoid", renorm=True, scale=2.5)
    logits = randn(rng, T, E, dt=F32) - ints(rng, 58, 62, T, 1).float()
    logits[:20] = randn(rng, 20, E, dt=F32) - ints(rng, 85, 600, 20, 1).float()
    logits[0] = -300.0
    logits[1] = -1000.0                                # 0 in 64 bits as well
    logits[2] = -float("inf")
    b = randn(rng, E, std=0.1, dt=F32) if bias else None
    idx, w = torch.empty(T, k, device="cuda", dtype=I32), empty(T, k, dt=F32)
    abi.router_select(rule, logits, b, idx, w)
    want, ww = R.select(logits, b, rule)
    if bias:                                           # 64 bits lose s beside the bias
        want = torch.sort(b.double().expand(T, E), dim=1, descending=True, stable=True)[1][:, :k]
        ww = R.weights(R.scores(logits, False), want, rule)
    assert torch.equal(idx.long(), want)
    assert bool((w[1:3] == 0).all())
    ok = torch.arange(T, device="cuda")
    ok = (ok < 1) | (ok > 2)
    R.within("w", w[ok], ww[ok], 128 * R.STEP * ww[ok])
    dw, dl = randn(rng, T, k, dt=F32), empty(T, E, dt=F32)
    abi.router_select_backward(rule, logits, idx, dw, dl)
    ref, mag = R.select_backward(logits[ok], want[ok], dw[ok], rule)
    R.within("dlogits", dl[ok], ref, (128 + E / 16) * R.STEP * (ref.abs() + mag))
    assert bool((dl[1:3] == 0).all())


@pytest.mark.parametrize("E", [24, 25, 301])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_router_select_backward_skips_other_ids(rng, E, score):
    T, k = 9, 3
    rule = abi.Routing(E, k, score=score, renorm=False)
    logits, dw = randn(rng, T, E, dt=F32), randn(rng, T, k, dt=F32)
    idx = torch.stack([torch.randperm(E, generator=rng, device="cuda")[:k] for _ in range(T)]).to(I32)
    bad = idx.clone()
    bad[2, 1], bad[5, 0] = -1, E
    dl, ref = empty(T, E, dt=F32), empty(T, E, dt=F32)
    abi.router_select_backward(rule, logits, bad, dw, dl)
    zero = dw.clone()
    zero[2, 1] = zero[5, 0] = 0
    abi.router_select_backward(rule, logits, idx, zero, ref)
    if score == "sigmoid":
        assert torch.equal(dl, ref)
    else:   # an expert of the row, or a chosen one without weight: three factors either way round
        R.within("dlogits", dl, ref.double(), 4 * R.STEP * ref.double().abs())


# ------------------------------------------------------------------ embedding

TABLES = [(1, 1, 8), (5, 7, 64), (300, 50, 136), (64, 3, 1024), (65, 2, 1032), (1000, 5000, 256),
          (33, 100, 6144), (2000, 1, 72)]


@pytest.mark.parametrize("T,V,d", TABLES)
@pytest.mark.parametrize("tab,out", [(BF, BF), (F32, BF), (BF, F32), (F32, F32)])
def test_embedding_forward(rng, T, V, d, tab, out):
    table, ids = randn(rng, V, d, dt=tab), ints(rng, 0, V, T)
    ids[T // 2] = -1
    got, st = empty(T, d, dt=out), status()
    abi.embedding(table, ids, got, st, scale=1.7)
    want = table.double()[ids.long().clamp(min=0)] * 1.7 * (ids >= 0)[:, None]
    R.within("out", got, want, (R.round_of(out) + 2 * R.STEP) * want.abs())
    assert int(st) == 0


@pytest.mark.parametrize("T,V,d", TABLES)
@pytest.mark.parametrize("tab,out", [(BF, BF), (F32, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_embedding_backward(rng, T, V, d, tab, out, accumulate):
    ids, dout = ints(rng, 0, V, T), randn(rng, T, d, dt=out)
    ids[T // 2] = -1
    check_embedding_backward(ids, dout, V, tab, accumulate)


def check_embedding_backward(ids, dout, V, tab, accumulate=False, want_status=0):
    T, d = dout.shape
    plan = abi.EmbeddingPlan(ids, V, d)
    start = torch.full((V, d), float("nan"), device="cuda", dtype=tab)
    if accumulate:
        start = torch.randn(V, d, device="cuda").to(tab)
    got = start.clone()
    abi.embedding_backward(plan, dout, got, scale=0.6, accumulate=accumulate)
    want, mag, most = R.embedding_backward(ids, dout, V, 0.6)
    bound = (most + 4) * R.STEP * mag
    if accumulate:
        want = want + start.double()
        bound = bound + 2 * R.STEP * start.double().abs()
    R.within("dtable", got, want, (1 + R.U) * bound + R.round_of(tab) * want.abs())
    assert int(plan.status) == want_status
    absent = torch.ones(V, dtype=torch.bool, device="cuda")
    absent[ids.long()[(ids >= 0) & (ids < V)]] = False
    assert torch.equal(got[absent], start[absent] if accumulate else torch.zeros_like(got[absent]))
    # again on the same plan, bit for bit
    more = start.clone()
    abi.embedding_backward(plan, dout, more, scale=0.6, accumulate=accumulate)
    assert torch.equal(got, more)
    return plan, got


def words(g, T, V, kind):
    if kind == "one":
        return torch.full((T,), V // 2, device="cuda", dtype=I32)
    if kind == "none":
        return torch.full((T,), -1, device="cuda", dtype=I32)
    if kind == "different":
        return torch.randperm(V, generator=g, device="cuda")[:T].to(I32)
    u = torch.rand(T, generator=g, device="cuda", dtype=F64)
    return ((V + 1) ** u - 1).long().clamp(0, V - 1).to(I32)     # a few words most of the time


@pytest.mark.parametrize("T,V,d,kind", [(5000, 9, 64, "one"), (777, 100, 40, "none"),
                                        (3000, 4000, 128, "different"), (20000, 3000, 96, "often"),
                                        (129, 4, 8, "one"), (128, 4, 8, "one"), (64, 1, 2048, "one"),
                                        (40000, 50, 16, "often"), (270000, 300, 8, "often"),
                                        (530000, 2, 8, "one")])
def test_embedding_backward_skewed(rng, T, V, d, kind):
    ids = words(rng, T, V, kind)
    check_embedding_backward(ids, randn(rng, T, d), V, F32)


@pytest.mark.parametrize("T", [31, 32, 33, 63, 65, 257, 1023, 1024, 1025, 1100])
@pytest.mark.parametrize("V,kind", [(1, "even"), (3, "often"), (200, "often"), (70000, "even")])
def test_embedding_backward_of_few_tokens(rng, T, V, kind):
    """Plans of one launch and of several, and one refilled after the other."""
    d, plan = 72, None
    for ids in (ints(rng, 0, V, T) if kind == "even" else words(rng, T, V, kind),
                ints(rng, 0, V, T), torch.full((T,), -1, device="cuda", dtype=I32)):
        ids[T // 3] = -1
        dout = randn(rng, T, d)
        if plan is None:
            plan = abi.EmbeddingPlan(ids, V, d)
        else:
            plan.refill(ids)
        got = torch.full((V, d), 7.0, device="cuda")
        abi.embedding_backward(plan, dout, got, scale=0.6)
        want, mag, most = R.embedding_backward(ids, dout, V, 0.6)
        R.within("dtable", got, want, (most + 4) * R.STEP * (1 + R.U) * mag + R.round_of(F32) * want.abs())


def test_embedding_sums_are_in_the_tokens_order(rng):
    """The plan's order is ascending within each word, whichever way the words are
    found: values whose sum tells the order."""
    T, V, d = 30000, 40, 8
    ids = words(rng, T, V, "often")
    plan, got = check_embedding_backward(ids, randn(rng, T, d, dt=F32), V, F32)
    for _ in range(5):
        plan.refill(ids)
        more = empty(V, d, dt=F32)
        abi.embedding_backward(plan, randn(torch.Generator(device="cuda").manual_seed(3), T, d), more)
        again = empty(V, d, dt=F32)
        plan.refill(ids)
        abi.embedding_backward(plan, randn(torch.Generator(device="cuda").manual_seed(3), T, d), again)
        assert torch.equal(more, again)


def test_embedding_refill_and_bad_ids(rng):
    T, V, d = 500, 60, 64
    a, b = words(rng, T, V, "often"), ints(rng, 0, V, T)
    dout = randn(rng, T, d)
    plan = abi.EmbeddingPlan(a, V, d)
    plan.refill(b)
    got, fresh = empty(V, d, dt=F32), empty(V, d, dt=F32)
    abi.embedding_backward(plan, dout, got)
    abi.embedding_backward(abi.EmbeddingPlan(b, V, d), dout, fresh)
    assert torch.equal(got, fresh)
    b[[3, 400]] = torch.tensor([V, -2], device="cuda", dtype=I32)
    check_embedding_backward(b, dout, V, F32, want_status=abi.MOE_EINVAL)
    out, st = empty(T, d), status()
    abi.embedding(randn(rng, V, d), b, out, st)
    assert int(st) == abi.MOE_EINVAL and bool((out[[3, 400]] == 0).all()) and bool(out.isfinite().all())


def test_embedding_nothing(rng):
    ids = torch.empty(0, device="cuda", dtype=I32)
    for dt in (BF, F32):
        got = empty(9, 24, dt=dt)
        abi.embedding_backward(abi.EmbeddingPlan(ids, 9, 24), torch.empty(0, 24, device="cuda", dtype=BF), got)
        assert bool((got == 0).all())
        abi.embedding_backward(abi.EmbeddingPlan(ids, 9, 24), torch.empty(0, 24, device="cuda", dtype=BF),
                               empty(9, 24, dt=dt), accumulate=True)


# ------------------------------------------------------------------ distillation

def distill_inputs(g, T, V, K, dt, tdt=F32, wide=None, shift=0):
    room = torch.empty(T * (wide or V) + 64, device="cuda", dtype=dt)
    room.fill_(float("nan"))
    z = room[shift:shift + T * (wide or V)].view(T, wide or V)[:, :V]
    z.copy_(randn(g, T, V, std=2.0, dt=dt))
    ids = ints(g, 0, V, T, K)                      # with words that stand twice
    teacher = randn(g, T, K, std=2.0, dt=tdt)
    there = torch.rand(T, K, generator=g, device="cuda") < 0.8
    ids[~there] = -1
    if T > 2:
        ids[1] = -1                                # a row without entries
    weight = torch.rand(T, generator=g, device="cuda") + 0.5
    if T > 3:
        weight[2] = 0
        z[2] = float("nan")                        # a row that is left out
    return z, ids, teacher, weight


#            T     V      K   z dtype
DISTILL = [(1, 1, 1, BF), (1, 7, 3, F32), (9, 64, 64, BF), (33, 133, 5, BF), (17, 2048, 1, BF),
           (5, 2049, 16, BF), (70, 1024, 9, F32), (6, 1025, 33, F32), (3, 16384, 256, BF),
           (4, 16385, 8, BF), (2, 8192, 7, F32), (5, 8193, 100, F32), (7, 50001, 50, BF),
           (4, 50001, 20, F32), (3, 131072, 64, BF), (200, 1000, 128, F32)]


@pytest.mark.parametrize("T,V,K,dt", DISTILL)
@pytest.mark.parametrize("tau,tdt", [(1.0, F32), (2.5, BF)])
def test_distill(rng, T, V, K, dt, tau, tdt):
    z, ids, teacher, weight = distill_inputs(rng, T, V, K, dt, tdt)
    want = R.distill(z, ids, teacher, weight, tau, 0.7)
    loss, lse, total, st = empty(T, dt=F32), empty(T, dt=F32), empty(1, dt=F32), status()
    abi.distill_loss(z, ids, teacher, weight, loss, lse, st, total=total, temperature=tau, scale=0.7)
    R.within("loss", loss, *want["loss"])
    R.within("lse", lse, *want["lse"])
    s = loss.double().sum()
    R.within("total", total, s.reshape(1), (T / 1024 + 12) * R.STEP * loss.double().abs().sum())
    dz, dz_b = want["dz"]
    bound = (1 + R.U) * dz_b + R.round_of(dt) * dz.abs()
    # the gradient alone, in the same pass, and over the logits
    one = empty(T, V, dt=dt)
    abi.distill_loss_backward(z, ids, teacher, weight, lse, one, st, temperature=tau, scale=0.7)
    R.within("dz from lse", one, dz, bound)
    both, l2, e2 = empty(T, V, dt=dt), empty(T, dt=F32), empty(T, dt=F32)
    abi.distill_loss(z, ids, teacher, weight, l2, e2, st, dlogits=both, temperature=tau, scale=0.7)
    R.within("dz", both, dz, bound)
    R.within("loss with the gradient", l2, *want["loss"])
    R.within("lse with the gradient", e2, *want["lse"])
    over = z.clone()
    abi.distill_loss(over, ids, teacher, weight, l2, e2, st, dlogits=over, temperature=tau, scale=0.7)
    assert torch.equal(over, both)
    R.within("loss over the logits", l2, *want["loss"])
    over = z.clone()
    abi.distill_loss_backward(over, ids, teacher, weight, lse, over, st, temperature=tau, scale=0.7)
    assert torch.equal(over, one)
    assert int(st) == 0


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("V,wide,shift,dz_shift", [(1001, 1008, 0, 0), (1001, 1001, 3, 3), (5003, 5010, 1, 2),
                                                   (40009, 40009, 5, 5), (40009, 40016, 0, 7), (3, 5, 1, 1)])
def test_distill_rows_anywhere(rng, dt, V, wide, shift, dz_shift):
    """Rows that start at any element, gradients that start at others, and nothing
    written between the rows."""
    T, K = 6, 4
    z, ids, teacher, weight = distill_inputs(rng, T, V, K, dt, F32, wide, shift)
    want = R.distill(z, ids, teacher, weight, 1.0, 1.0)
    loss, lse, st = empty(T, dt=F32), empty(T, dt=F32), status()
    room = torch.full((T * wide + 64,), 77.0, device="cuda", dtype=dt)
    dz = room[dz_shift:dz_shift + T * wide].view(T, wide)[:, :V]
    abi.distill_loss(z, ids, teacher, weight, loss, lse, st, dlogits=dz)
    R.within("loss", loss, *want["loss"])
    x, b = want["dz"]
    R.within("dz", dz, x, (1 + R.U) * b + R.round_of(dt) * x.abs())
    gone = room.clone()
    gone[dz_shift:dz_shift + T * wide].view(T, wide)[:, :V] = 77.0
    assert bool((gone == 77.0).all())


def test_distill_of_one_entry_is_the_cross_entropy(rng):
    T, V = 50, 777
    z, label = randn(rng, T, V, std=3.0), ints(rng, 0, V, T)
    loss, lse, st = empty(T, dt=F32), empty(T, dt=F32), status()
    abi.distill_loss(z, label[:, None].contiguous(), torch.zeros(T, 1, device="cuda"), None, loss, lse, st)
    want = torch.nn.functional.cross_entropy(z.double(), label.long(), reduction="none")
    R.within("loss", loss, want, 64 * R.STEP * (want + lse.double().abs() + 20))


def test_distill_masked_values(rng):
    """Student words at -inf, teacher entries at -inf, all of them, and ids outside
    the vocabulary."""
    T, V, K = 8, 300, 6
    z, ids = randn(rng, T, V, dt=F32), torch.stack([torch.randperm(V, generator=rng, device="cuda")[:K]
                                                    for _ in range(T)]).to(I32)
    teacher = randn(rng, T, K, dt=F32)
    z[0, :100] = -float("inf")
    ids[0] = torch.arange(100, 106, device="cuda")
    teacher[1, 2:4] = -float("inf")
    teacher[2] = -float("inf")
    ids[3, 0] = V
    ids[4, 1] = -5
    z[5, ids[5, 0].long()] = -float("inf")         # a word that the teacher wants and the student bans
    z[6, ids[6, 0].long()] = -float("inf")         # one that neither wants
    teacher[6, 0] = -float("inf")
    loss, lse, st, dz = empty(T, dt=F32), empty(T, dt=F32), status(), empty(T, V, dt=F32)
    abi.distill_loss(z, ids, teacher, None, loss, lse, st, dlogits=dz)
    assert int(st) == abi.MOE_EINVAL
    want = R.distill(z, ids, teacher, None, 1.0, 1.0)
    fine = torch.tensor([0, 1, 2, 3, 4, 6, 7], device="cuda")
    R.within("loss", loss[fine], want["loss"][0][fine], want["loss"][1][fine])
    x, b = want["dz"]
    R.within("dz", dz[fine], x[fine], b[fine] + R.STEP * x[fine].abs())
    assert float(loss[5]) == float("inf") and bool(dz[5].isfinite().all())
    assert float(loss[2]) == 0 and float(lse[2]) == 0 and bool((dz[2] == 0).all())


def test_distill_gradient_is_that_of_differences(rng):
    T, V, K = 2, 11, 3
    z, ids, teacher = randn(rng, T, V, dt=F64), ints(rng, 0, V, T, K), randn(rng, T, K, dt=F64)
    dz = R.distill(z, ids, teacher, None, 1.5, 0.9)["dz"][0]
    f = lambda z: float(R.distill(z, ids, teacher, None, 1.5, 0.9)["loss"][0].sum())  # noqa: E731
    for at in ((0, 0), (1, 5), (0, int(ids[0, 0]))):
        d = torch.zeros_like(z)
        d[at] = 1e-5
        assert abs((f(z + d) - f(z - d)) / 2e-5 - float(dz[at])) < 1e-8


@pytest.mark.parametrize("V", [700, 5001, 40000])
@pytest.mark.parametrize("shift", [0.0, 512.0, -1024.0])
def test_distill_loss_does_not_feel_a_shift_of_all_logits(rng, V, shift):
    """Logits in whole 2^-10, so that the shift is exact: what is lost is by the
    logits' differences (at most 32 here, 47 as exponents), not by their size."""
    T, K = 33, 4
    z = (randn(rng, T, V, std=2.0, dt=F32) * 1024).round() / 1024
    z[:, 5] += 12.0                                     # a word that is nearly certain
    ids, y = ints(rng, 0, V, T, K), (randn(rng, T, K, dt=F32) * 1024).round() / 1024
    ids[:, 0] = 5
    y[:, 0] += 12.0
    ref = R.distill(z, ids, y, None, 1.0, 1.0)
    loss, lse, dz, st = empty(T, dt=F32), empty(T, dt=F32), empty(T, V, dt=F32), status()
    abi.distill_loss(z + shift, ids, y + shift, None, loss, lse, st, dlogits=dz)
    # differences in one rounding of 47 each, the sums' logarithms, an exponential's 4 and 1.5
    # of its argument, sums in V / 128 + 64 roundings at most
    assert float((loss - ref["loss"][0]).abs().max()) < (4 * 47 + 4 + 1.5 * 47 + V / 128 + 64) * R.STEP
    assert float((dz - ref["dz"][0]).abs().max()) < 2 * (4 + 1.5 * 47 + V / 128 + 64) * R.STEP


# ------------------------------------------------------------------ streams and graphs

def test_captured_on_another_stream_and_replayed(rng):
    """Each operator on a side stream, captured once and replayed on other values."""
    T, hq, hk, D, E, k, V, d, K = 200, 4, 2, 64, 48, 4, 333, 64, 5
    rule = abi.Routing(E, k, score="sigmoid", n_groups=4, groups_kept=2, group_top=2)
    x = head_inputs(rng, T, hq, hk, D, 64)
    logits, bias = randn(rng, T, E, dt=F32), randn(rng, E, std=0.05, dt=F32)
    ids, dout = ints(rng, 0, V, T), randn(rng, T, d)
    z, ti, ty, wt = distill_inputs(rng, T, V, K, BF)
    buf = dict(q=empty(T, hq, D), k=empty(T, hk, D), dq=empty(T, hq, D), dk=empty(T, hk, D), dwq=empty(D, dt=F32),
               dwk=empty(D, dt=F32), idx=torch.zeros(T, k, device="cuda", dtype=I32), w=empty(T, k, dt=F32),
               dl=empty(T, E), dt=empty(V, d, dt=F32), loss=empty(T, dt=F32), lse=empty(T, dt=F32),
               total=empty(1, dt=F32), dz=empty(T, V), st=status())
    ws = torch.empty(abi.head_norm_rotary_workspace(T, hq, hk, D), dtype=torch.uint8, device="cuda")
    plan = abi.EmbeddingPlan(ids, V, d)

    def run(stream=None):
        b = buf
        abi.head_norm_rotary(x["q"], x["k"], x["w_q"], x["w_k"], x["table"], x["pos"], b["q"], b["k"], b["st"],
                             stream=stream)
        abi.head_norm_rotary_backward(b["q"], b["k"], x["q"], x["k"], x["w_q"], x["w_k"], x["table"], x["pos"],
                                      b["dq"], b["dk"], b["dwq"], b["dwk"], ws, b["st"], stream=stream)
        abi.router_select(rule, logits, bias, b["idx"], b["w"], stream=stream)
        abi.router_select_backward(rule, logits, b["idx"], b["w"], b["dl"], stream=stream)
        plan.refill(ids, stream)
        abi.embedding_backward(plan, dout, b["dt"], stream=stream)
        abi.distill_loss(z, ti, ty, wt, b["loss"], b["lse"], b["st"], total=b["total"], dlogits=b["dz"],
                         stream=stream)

    def result():
        run()
        torch.cuda.synchronize()
        return {n: t.clone() for n, t in buf.items()}

    first = result()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for t in buf.values():
        t.zero_()
    torch.cuda.synchronize()
    run(side)                                       # by argument, not as the current stream
    side.synchronize()
    for n in first:
        assert torch.equal(first[n], buf[n]), n
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    logits.copy_(randn(rng, T, E, dt=F32))
    ids.copy_(ints(rng, 0, V, T))
    dout.copy_(randn(rng, T, d))
    x["q"].copy_(randn(rng, T, hq, D))
    z[4:].copy_(randn(rng, T - 4, V))
    want = result()
    for t in buf.values():
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert int(buf["st"]) == 0
    for n in want:
        assert torch.equal(want[n], buf[n]), n


@pytest.mark.parametrize("T", [5, 1500, 6000])
def test_calls_behind_one_another_see_what_came_before(rng, T):
    """Inputs written right before a call and again right behind it, outputs that are
    the next call's inputs, scratch that the next call takes: as with waits between."""
    hq, hk, D, E, k, V, d, K = 6, 2, 64, 64, 4, 900, 136, 7
    rule = abi.Routing(E, k, score="softmax", n_groups=4, groups_kept=2, group_top=2, renorm=False)
    sets = []
    for _ in range(2):
        x = head_inputs(rng, T, hq, hk, D, 64)
        z, ti, ty, wt = distill_inputs(rng, T, V, K, BF)
        sets.append(dict(q=x["q"], pos=x["pos"], wq=x["w_q"], logits=randn(rng, T, E, dt=F32),
                         ids=words(rng, T, V, "often"), table=randn(rng, V, d), z=z, ti=ti, ty=ty, wt=wt))
    key, w_k, table, bias = x["k"], x["w_k"], x["table"], randn(rng, E, std=0.01, dt=F32)
    now = {n: t.clone() for n, t in sets[0].items()}
    buf = dict(q=empty(T, hq, D), k=empty(T, hk, D), dq=empty(T, hq, D), dk=empty(T, hk, D), dwq=empty(D, dt=F32),
               dwk=empty(D, dt=F32), idx=torch.zeros(T, k, device="cuda", dtype=I32), w=empty(T, k, dt=F32),
               dl=empty(T, E, dt=F32), h=empty(T, d), dt=empty(V, d, dt=F32), loss=empty(T, dt=F32),
               lse=empty(T, dt=F32), total=empty(1, dt=F32), dz=empty(T, V), dz2=empty(T, V), st=status())
    ws = torch.empty(abi.head_norm_rotary_workspace(T, hq, hk, D), dtype=torch.uint8, device="cuda")
    plan = abi.EmbeddingPlan(now["ids"], V, d)

    def step(values, wait):
        n, b = now, buf
        for name, t in values.items():
            n[name].copy_(t)
        wait()
        abi.head_norm_rotary(n["q"], key, n["wq"], w_k, table, n["pos"], b["q"], b["k"], b["st"])
        wait()
        abi.head_norm_rotary_backward(b["q"], b["k"], n["q"], key, n["wq"], w_k, table, n["pos"], b["dq"], b["dk"],
                                      b["dwq"], b["dwk"], ws, b["st"])
        wait()
        abi.router_select(rule, n["logits"], bias, b["idx"], b["w"])
        wait()
        abi.router_select_backward(rule, n["logits"], b["idx"], b["w"], b["dl"])
        wait()
        abi.embedding(n["table"], n["ids"], b["h"], b["st"])
        wait()
        plan.refill(n["ids"])
        wait()
        abi.embedding_backward(plan, b["h"], b["dt"])
        wait()
        abi.distill_loss(n["z"], n["ti"], n["ty"], n["wt"], b["loss"], b["lse"], b["st"], total=b["total"],
                         dlogits=b["dz"])
        wait()
        abi.distill_loss_backward(b["dz"], n["ti"], n["ty"], n["wt"], b["lse"], b["dz2"], b["st"])
        wait()

    want = []
    for values in sets:
        step(values, torch.cuda.synchronize)
        want.append({n: t.clone() for n, t in buf.items()})
    got = []
    for i in range(24):
        step(sets[i % 2], lambda: None)
        got.append({n: t.clone() for n, t in buf.items()} if i % 5 == 3 else None)
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        for n in g or ():
            same = torch.equal(g[n].nan_to_num() if g[n].is_floating_point() else g[n],
                               want[i % 2][n].nan_to_num() if g[n].is_floating_point() else want[i % 2][n])
            assert same, (i, n)
