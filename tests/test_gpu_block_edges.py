"""GPU tests of the training block's operators where other streams, refused
sequences, values that are not finite, empty batches and long work lists meet
them."""
import math

import pytest
import torch

import block_reference as R
from moe_routing_capacity_gb300 import abi
from moe_routing_capacity_gb300 import workloads as wl
from moe_routing_capacity_gb300.block import TrainingBlock, draw_block_weights
from moe_routing_capacity_gb300.layer import PooledWaveMoE

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


# ------------------------------------------------------------------ values that are not finite

def offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def reference(q, k, v, lens, dout):
    """R.attention with what its bounds leave out: D of a row past its
    sequence's first 128 comes from the out that the rounded P gave.  With
    weights w~ from P (1 + d), |d| <= U, the row's D is off by
    sum (w~ - w)(dP - D) <= 2 U (1 + 2 U) sum w |dP - D|, and dS by P times it."""
    D = q.shape[2]
    want = R.attention(q, k, v, lens, D ** -0.5, dout=dout)
    group, at = q.shape[1] // k.shape[1], 0
    q, k, v, dout = (t.double() for t in (q, k, v, dout))
    for n in lens:
        sl = slice(at, at + n)
        at += n
        keep = torch.ones(n, n, dtype=torch.bool, device=q.device).tril()
        for h in range(q.shape[1]):
            kv = h // group
            p = torch.softmax((q[sl, h] @ k[sl, kv].T * D ** -0.5).masked_fill(~keep, -math.inf), 1)
            dp = dout[sl, h] @ v[sl, kv].T
            off = (p * (dp - (p * dp).sum(1, keepdim=True)).abs()).sum(1, keepdim=True)
            ds = 2 * R.U * (1 + 2 * R.U) ** 2 * p * off * D ** -0.5
            want["dq"][1][sl, h] += ds @ k[sl, kv].abs()
            want["dk"][1][sl, kv] += ds.T @ q[sl, h].abs()
    return want


# lengths, hq, hk, D: one CTA, two and four a block of keys in the backward;
# second pieces of work a CTA in the last one
NOT_FINITE = [([300, 333, 150], 4, 4, 64), ([300, 211], 2, 1, 128), ([140, 300, 50], 8, 1, 80),
              ([1111, 1300, 900], 16, 8, 128), ([700, 1001, 1499], 9, 3, 96)]


@pytest.mark.parametrize("lens,hq,hk,D", NOT_FINITE)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_token_that_is_not_finite(rng, lens, hq, hk, D, bad):
    """All of one token's q, k, v and gradient: its sequence's earlier rows and
    every other sequence have the values they would have without it (the
    sequence before it ends inside a tile that it shares); with NaN, its own
    row and the later ones are NaN, and so is every key that they see."""
    T, cu = sum(lens), offsets(lens)
    q, k, v, dout = (randn(rng, T, h, D) for h in (hq, hk, hk, hq))
    want = reference(q, k, v, lens, dout)
    clean, _ = attention_step(q, k, v, cu, dout)
    for hit in (cu[1], cu[1] + lens[1] // 2):
        x = [t.clone() for t in (q, k, v, dout)]
        for t in x:
            t[hit] = bad
        got, st = attention_step(*x[:3], cu, x[3])
        assert st == [0, 0]
        rows = torch.ones(T, dtype=torch.bool, device="cuda")
        rows[hit:cu[2]] = False
        keys = torch.ones(T, dtype=torch.bool, device="cuda")
        keys[cu[1]:cu[2]] = False
        for n, some in (("out", rows), ("dq", rows), ("dk", keys), ("dv", keys)):
            R.within(n, got[n][some], want[n][0][some], want[n][1][some] + 1e-30)
            assert torch.equal(got[n][some], clean[n][some]), n    # not a bit of theirs
            if math.isnan(bad):
                assert bool(got[n][~some].isnan().all()), n


@pytest.mark.parametrize("lens,hq,hk,D", NOT_FINITE)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_gradient_that_is_not_finite(rng, lens, hq, hk, D, bad):
    """It reaches its own row and the keys up to it."""
    T, cu = sum(lens), offsets(lens)
    q, k, v, dout = (randn(rng, T, h, D) for h in (hq, hk, hk, hq))
    want = reference(q, k, v, lens, dout)
    clean, _ = attention_step(q, k, v, cu, dout)
    hit = cu[1] + lens[1] // 2
    d = dout.clone()
    d[hit] = bad
    got, st = attention_step(q, k, v, cu, d)
    assert st == [0, 0]
    rows = torch.ones(T, dtype=torch.bool, device="cuda")
    rows[hit] = False
    keys = torch.ones(T, dtype=torch.bool, device="cuda")
    keys[cu[1]:hit + 1] = False
    for n, some in (("out", rows | True), ("dq", rows), ("dk", keys), ("dv", keys)):
        R.within(n, got[n][some], want[n][0][some], want[n][1][some] + 1e-30)
        assert torch.equal(got[n][some], clean[n][some]), n
        assert not bool(got[n][~some].isfinite().any()), n


@pytest.mark.parametrize("D", [64, 128])
def test_a_channel_that_is_not_finite(rng, D):
    """NaN in one channel of every value stays in that channel of out; an
    infinity that a row sees and one that it does not are told apart."""
    lens, hq, hk = [300, 500], 4, 2
    T, cu = 800, [0, 300, 800]
    q, k, v, dout = (randn(rng, T, h, D) for h in (hq, hk, hk, hq))
    want = R.attention(q, k, v, lens, D ** -0.5)["out"]
    x = v.clone()
    x[:, :, 5] = float("nan")
    x[310, :, 7] = float("inf")      # seen by the rows from there on
    x[340, :, 7] = float("inf")      # hidden from the rows before it
    got, st = attention_step(q, k, x, cu, dout)
    assert st == [0, 0]
    assert bool(got["out"][:, :, 5].isnan().all())
    keep = torch.ones(D, dtype=torch.bool, device="cuda")
    keep[5] = keep[7] = False
    R.within("out", got["out"][..., keep], want[0][..., keep], want[1][..., keep] + 1e-30)
    R.within("before", got["out"][:310, :, 7], want[0][:310, :, 7], want[1][:310, :, 7] + 1e-30)
    assert bool((got["out"][310:, :, 7] == float("inf")).all())


@pytest.mark.parametrize("what", ["first value", "every value", "every gradient", "first key",
                                  "a token amid", "a value a block", "infinite values"])
def test_what_is_not_finite_costs_little(rng, what):
    """The step takes no more than three times a finite one's time."""
    T, hq, hk, D = 16384, 4, 1, 128
    x = {n: randn(rng, T, h, D) for n, h in (("q", hq), ("k", hk), ("v", hk), ("d", hq))}
    bad = {n: t.clone() for n, t in x.items()}
    if what == "first value":
        bad["v"][0] = math.nan
    elif what == "every value":
        bad["v"].fill_(math.nan)
    elif what == "every gradient":
        bad["d"].fill_(math.nan)
    elif what == "first key":
        bad["k"][0] = math.nan
    elif what == "a token amid":
        for t in bad.values():
            t[T // 2 + 64] = math.nan
    elif what == "a value a block":
        for i in range(64, T, 128):
            bad["v"][i, 0, i // 128] = math.nan
    else:
        bad["v"].fill_(math.inf)
    plan = abi.AttentionPlan(ints(0, T), T, hq, hk, D)
    times = []
    for t in (x, bad, x, bad):
        best = math.inf
        for _ in range(3):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            _, st = attention_step(t["q"], t["k"], t["v"], None, t["d"], plan)
            b.record()
            b.synchronize()
            assert st == [0, 0]
            best = min(best, a.elapsed_time(b))
        times.append(best)
    assert min(times[1::2]) <= 3 * min(times[::2]), times


@pytest.mark.parametrize("hq,hk", [(2, 1), (3, 1)])
def test_keys_without_weight(rng, hq, hk):
    """Keys whose scores are -infinity have weight 0, a sequence's first 128 or
    more among them: the later rows are the softmax over the others."""
    T, D, dead = 700, 64, 260
    q, k, v = randn(rng, T, hq, D), randn(rng, T, hk, D), randn(rng, T, hk, D)
    q[..., 0] = q[..., 0].abs() + 1
    k[:dead, :, 0] = -math.inf
    plan = abi.AttentionPlan(ints(0, T), T, hq, hk, D)
    out, lse, st = empty(T, hq, D), empty(hq, T, dt=F32), status()
    abi.attention(plan, q, k, v, out, lse, st)
    assert int(st) == 0
    assert bool(out[:dead].isnan().all()) and bool((lse[:, :dead] == -math.inf).all())
    keep = torch.ones(T, T, dtype=torch.bool, device="cuda").tril()
    for h in range(hq):
        s = (q[dead:, h].double() @ k[:, h * hk // hq].double().T * D ** -0.5)
        s = s.masked_fill(~keep[dead:], -math.inf)
        p, x = torch.softmax(s, 1), v[:, h * hk // hq].double()
        R.within("out", out[dead:, h], p @ x, (R.U + R.EPS) * (p @ x.abs()) + R.U * (p @ x).abs())
        want = torch.logsumexp(s, 1)
        R.within("lse", lse[h, dead:], want, 1e-5 + 1e-5 * want.abs())


# ------------------------------------------------------------------ other streams

def test_a_plan_on_another_stream_clears_its_status_there():
    """Not on the current one, whose queued work would put the clear behind the
    plan and its error."""
    cu, side = ints(0, 50, 40), torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    plan = abi.AttentionPlan(cu, 100, 2, 1, 64, stream=side)
    side.synchronize()
    assert int(plan.status.cpu()) == abi.MOE_EINVAL
    torch.cuda.synchronize()
    assert int(plan.status.cpu()) == abi.MOE_EINVAL


def tiny_block(heads=4, kv_heads=2, D=32):
    """A training block at the tiny layer's size, two sequences, its input."""
    cfg = wl.TINY
    inp = wl.make_inputs(cfg, "cpu")
    table = empty(cfg.T, D // 2, 2, dt=F32)
    abi.rotary_table(table)
    blk = TrainingBlock(PooledWaveMoE(cfg, inp, "cuda"),
                        draw_block_weights(cfg.d_model, heads, kv_heads, D, seed=5), heads,
                        kv_heads, D, table, 2)
    blk.set_batch(ints(0, 101, cfg.T), None)
    return blk, inp["x"].cuda()


def test_a_block_on_another_stream_takes_its_memory_there(rng):
    """backward() and clip() allocate what they use on their stream: memory
    that work queued on the current stream still writes is not theirs."""
    runs = []
    for side in (None, torch.cuda.Stream()):
        blk, h = tiny_block()
        dh = randn(torch.Generator(device="cuda").manual_seed(3), *h.shape)
        norm = empty(1, dt=F32)
        torch.cuda.synchronize()
        blk.forward(h, stream=side)
        if side:
            # freed at once, written once the current stream gets there
            junk = [empty(n) for t in (blk.qkv, blk.n1, blk.rstd[0], *blk.w.values())
                    for n in {t.numel(), 2 * t.numel(), 4096}]
            junk.append(empty(1 << 24))
            torch.cuda.synchronize()
            torch.cuda._sleep(200_000_000)
            for t in junk:
                t.fill_(float("nan"))
            del t, junk
        g = blk.backward(dh, stream=side)
        blk.clip(0.5, norm, stream=side)
        torch.cuda.synchronize()
        assert int(blk.status) == 0
        runs.append({n: t.clone() for n, t in g.items()} | {"norm": norm})
    for n, t in runs[0].items():
        assert torch.equal(t, runs[1][n]), n


# ------------------------------------------------------------------ nothing to sum

@pytest.mark.parametrize("gate", ["none", "channel", "token"])
def test_norm_gradients_of_no_token_are_zero(rng, gate):
    T, d = 0, 64
    w = randn(rng, d)
    g = {"none": None, "channel": w, "token": empty(T, d)}[gate]
    dgate = {"none": None, "channel": empty(d, dt=F32), "token": empty(T, d)}[gate]
    dw_post, dw_pre = empty(d, dt=F32), empty(d, dt=F32)
    x, s = empty(T, d), empty(T, dt=F32)
    ws = torch.empty(max(1, abi.norm_residual_workspace(T, d)), device="cuda", dtype=torch.uint8)
    abi.norm_residual_backward(x, x, x, x, g, w, w, s, s, empty(T, d), empty(T, d), dgate,
                               dw_post, dw_pre, ws)
    for t in (dw_post, dw_pre, dgate):
        assert t is None or not t.any()


def test_norm_of_no_gradients_is_zero():
    norm = empty(1, dt=F32)
    abi.grad_clip(abi.GradSet([]), 1.0, norm)
    assert float(norm) == 0.0
    norm = empty(1, dt=F32)
    abi.grad_clip(abi.GradSet([empty(0, dt=F32), empty(0)]), 1.0, norm)
    assert float(norm) == 0.0


# ------------------------------------------------------------------ gradients of zero and near it

def best_ms(f, n=5):
    best = math.inf
    for _ in range(n):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        f()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("size", [0.0, -0.0, 1e-11])
def test_zero_and_small_gradients_take_no_longer(rng, dt, size):
    """Experts that met no token have gradients of exactly zero."""
    n = 100_000_000
    x, out, norm = randn(rng, n, dt=dt), empty(n, dt=dt), empty(1, dt=F32)
    small = x * size
    sets = [abi.GradSet([t], [out]) for t in (x, small)]
    ms = [best_ms(lambda s=s: abi.grad_clip(s, 1.0, norm)) for s in sets]
    want = math.sqrt(float(small.double().square().sum()))
    assert abs(float(norm) - want) <= 1e-6 * want
    assert torch.equal(out, small)
    assert ms[1] <= 1.2 * ms[0], ms


@pytest.mark.parametrize("size", [1e-13, 1e-15, 1e-16, 1e-18])
def test_norm_of_small_gradients(rng, size):
    """About where the squares leave fp32's normal numbers."""
    x = torch.randn(300_001, generator=rng, device="cuda") * size
    norm = empty(1, dt=F32)
    abi.grad_clip(abi.GradSet([x]), 1.0, norm)
    want = math.sqrt(float(x.double().square().sum()))
    assert abs(float(norm) - want) <= 1e-6 * want


# ------------------------------------------------------------------ what the block hands on

def test_the_moe_branch_gets_its_own_gradient(rng):
    """The gradient that the block gives the MoE layer is the second residual
    norm's; dx of that call, and its weights' gradients, are what it uses and
    returns."""
    blk, h = tiny_block()
    dh3 = randn(rng, *h.shape)
    blk.forward(h)
    seen, plain = {}, blk.layer.backward

    def backward(x, dout, stream=None):
        seen.update(x=x.clone(), dout=dout.clone())
        got = plain(x, dout, stream=stream)
        seen["dx"] = got["x"].clone()
        return got

    blk.layer.backward = backward
    got = {n: t.clone() for n, t in blk.backward(dh3).items()}
    assert torch.equal(seen["x"], blk.n2)
    w = blk.w
    want = R.norm_backward(None, dh3, blk.b2, blk.h2, w["gate2"], w["w_post2"], None, 1.0, 1.0,
                           1e-6)
    # rows cancel (dp - p mean(dp p)): bounded against the tensor's size
    R.within("db2", seen["dout"], want["db"],
             2e-5 * float(want["db"].abs().max()) + R.U * want["db"].abs())
    alone = plain(blk.n2, seen["dout"])
    assert torch.equal(alone["x"], seen["dx"])
    names = [n for n, t in alone.items() if n != "x" and t.numel()]
    assert names and sorted("moe." + n for n in names) == sorted(n for n in got if n.startswith("moe."))
    for n in names:
        assert torch.equal(got["moe." + n], alone[n]), n
    # dn2, used in the first residual norm's backward: dgate1 depends on it
    du = R.norm_backward(seen["dx"], dh3, blk.b1, h, w["gate1"], w["w_post1"], w["w_pre2"], 1.0, 1.0,
                         1e-6)
    size = float(du["dgate"].abs().max())
    # dy of that call is the stream's gradient, dh3 itself (alpha 1, no norm behind h3)
    R.within("dgate1", got["gate1"], du["dgate"], 2e-5 * size)
    R.within("dw_pre2", got["w_pre2"], du["dw_pre"], 2e-5 * float(du["dw_pre"].abs().max()))


@pytest.mark.parametrize("hq,hk", [(4, 2), (3, 1)])
def test_gradients_with_keys_without_weight(rng, hq, hk):
    """Keys at -infinity in one channel: 0 times that is NaN in that channel of
    dq, for the rows that see them, and nothing anywhere else."""
    T, D, dead = 700, 64, 260
    q, k, v, dout = (randn(rng, T, h, D) for h in (hq, hk, hk, hq))
    q[..., 0] = q[..., 0].abs() + 1
    k[:dead, :, 0] = -math.inf
    got, st = attention_step(q, k, v, [0, T], dout)
    assert st == [0, 0]
    for n in ("out", "dq", "dk", "dv"):
        assert bool(got[n][:dead].isnan().all()), n
    assert bool(got["dq"][dead:, :, 0].isnan().all())
    # the others' gradients: what the live keys alone give
    live = slice(dead, T)
    want = reference(q[live], k[live], v[live], [T - dead], dout[live])
    for n in ("out", "dk", "dv"):
        R.within(n, got[n][live], want[n][0], want[n][1] + 1e-30)
    R.within("dq", got["dq"][live, :, 1:], want["dq"][0][..., 1:], want["dq"][1][..., 1:] + 1e-30)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hq,hk", [(4, 2), (3, 1), (8, 1)])
def test_infinities_that_are_seen_come_out(rng, hq, hk, D):
    """Single infinite values and gradients, of either sign, some in one block and
    some in the next: out and dv hold their signs, or NaN where both meet."""
    T = 600
    q, k, v, dout = (randn(rng, T, h, D) for h in (hq, hk, hk, hq))
    clean, _ = attention_step(q, k, v, [0, T], dout)
    x, d = v.clone(), dout.clone()
    x[130, :, 3] = math.inf
    x[140, :, 3] = -math.inf
    x[300, :, 9] = -math.inf
    got, st = attention_step(q, k, x, [0, T], dout)
    want = clean["out"].clone()
    want[130:, :, 3] = math.inf
    want[140:, :, 3] = math.nan
    want[300:, :, 9] = -math.inf
    assert torch.equal(got["out"].nan_to_num(7e5), want.nan_to_num(7e5))
    d[130, :, 3] = math.inf
    d[140, :, 3] = -math.inf
    d[300, 0, 9] = -math.inf
    got, st = attention_step(q, k, v, [0, T], d)
    want = clean["dv"].clone()
    want[:141, :, 3] = -math.inf
    want[:131, :, 3] = math.nan
    want[:301, 0, 9] = -math.inf
    assert torch.equal(got["dv"].nan_to_num(7e5), want.nan_to_num(7e5))
