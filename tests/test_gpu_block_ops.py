"""GPU parity of the training block's operators against plain 64-bit
implementations, at the sizes, layouts and values where each can go wrong."""
import math

import pytest
import torch

import block_reference as R
from moe_routing_capacity_gb300 import abi

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture
def rng():
    return torch.Generator(device="cuda").manual_seed(7)


def randn(g, *s, std=1.0, dt=BF):
    return (torch.randn(s, generator=g, device="cuda") * std).to(dt)


def empty(*s, dt=BF):
    return torch.full(s, float("nan"), device="cuda", dtype=dt)


def status():
    return torch.zeros(1, device="cuda", dtype=torch.int32)


# ------------------------------------------------------------------ norm

NORM_SIZES = [(1, 8), (3, 64), (9, 264), (17, 512), (300, 1000), (5, 1024), (33, 1032), (7, 2048),
              (450, 2056), (2, 4104), (331, 6144), (3, 8192)]


def norm_inputs(g, T, d, gate, rt):
    x = dict(b=randn(g, T, d), r=randn(g, T, d, std=2.0, dt=rt), w_post=1 + randn(g, d, std=0.1),
             w_pre=1 + randn(g, d, std=0.1))
    x["gate"] = {"none": None, "channel": randn(g, d, std=0.5),
                 "token": randn(g, T, d, std=0.5)}[gate]
    return x


@pytest.mark.parametrize("T,d", NORM_SIZES)
@pytest.mark.parametrize("gate,rt", [("none", BF), ("channel", BF), ("token", F32),
                                     ("channel", F32), ("token", BF)])
def test_norm_forward(rng, T, d, gate, rt):
    x = norm_inputs(rng, T, d, gate, rt)
    y, n = empty(T, d, dt=rt), empty(T, d)
    rb, ry = empty(T, dt=F32), empty(T, dt=F32)
    abi.norm_residual(x["b"], x["r"], x["gate"], x["w_post"], x["w_pre"], y, n, rb, ry,
                      alpha=0.9, beta=0.7, eps=1e-5)
    wy, wn, wb, wr = R.norm_forward(x["b"], x["r"], x["gate"], x["w_post"], x["w_pre"], 0.9, 0.7,
                                    1e-5)
    # fp32 sums relative to the terms' magnitudes, one rounding to bf16
    mag = (0.9 * x["r"].double()).abs() + (wy - 0.9 * x["r"].double()).abs()
    R.within("y", y, wy, R.EPS * mag + (R.U * wy.abs() if rt == BF else 0))
    R.within("n", n, wn, R.EPS * (mag * wr[:, None] * x["w_pre"].double().abs()) + (R.U + R.EPS) * wn.abs())
    R.within("rstd_post", rb, wb, R.EPS * wb)
    R.within("rstd_pre", ry, wr, R.EPS * wr)


@pytest.mark.parametrize("d", [96, 2048])
def test_norm_forward_parts_and_in_place(rng, d):
    """No branch, no next norm, no statistics; y over r and n over b."""
    T = 37
    x = norm_inputs(rng, T, d, "channel", BF)
    n, y = empty(T, d), empty(T, d)
    abi.norm_residual(None, x["r"], None, None, x["w_pre"], None, n)
    _, wn, _, _ = R.norm_forward(None, x["r"], None, None, x["w_pre"], 1.0, 1.0, 1e-6)
    R.within("n", n, wn, (R.U + R.EPS) * wn.abs())
    abi.norm_residual(x["b"], x["r"], x["gate"], x["w_post"], None, y, None)
    wy = R.norm_forward(x["b"], x["r"], x["gate"], x["w_post"], None, 1.0, 1.0, 1e-6)[0]
    mag = x["r"].double().abs() + (wy - x["r"].double()).abs()
    R.within("y", y, wy, R.U * wy.abs() + R.EPS * mag)
    abi.norm_residual(x["b"], x["r"], x["gate"], x["w_post"], x["w_pre"], y, n)
    r, b = x["r"].clone(), x["b"].clone()
    abi.norm_residual(b, r, x["gate"], x["w_post"], x["w_pre"], r, b)
    assert torch.equal(r, y) and torch.equal(b, n)


def test_norm_rows_of_zeros_and_of_huge_values(rng):
    """A zero row gives zeros (eps); a row's NaN or infinity stays in its row."""
    T, d = 6, 256
    x = norm_inputs(rng, T, d, "none", BF)
    x["b"][1] = 0
    x["r"][1] = 0
    x["b"][3, 5] = float("nan")
    x["r"][4, 7] = float("inf")
    y, n = empty(T, d), empty(T, d)
    abi.norm_residual(x["b"], x["r"], None, x["w_post"], x["w_pre"], y, n)
    assert not y[1].any() and not n[1].any()
    assert bool(n[3].isnan().any())
    for t in (0, 1, 2, 5):
        assert bool(y[t].isfinite().all()) and bool(n[t].isfinite().all())


def norm_grads(x, dn, dy, alpha=0.9, beta=0.7, eps=1e-5, dr=None):
    T, d = dn.shape if dn is not None else dy.shape
    rt = x["r"].dtype
    y, n = empty(T, d, dt=rt), empty(T, d) if dn is not None else None
    has_b = x["b"] is not None
    rb = empty(T, dt=F32) if has_b else None
    ry = empty(T, dt=F32) if dn is not None else None
    w_pre = x["w_pre"] if dn is not None else None
    abi.norm_residual(x["b"], x["r"], x["gate"], x["w_post"], w_pre, y, n, rb, ry, alpha=alpha,
                      beta=beta, eps=eps)
    got = dict(db=empty(T, d) if has_b else None, dr=empty(T, d, dt=rt) if dr is None else dr,
               dw_post=empty(d, dt=F32) if has_b else None,
               dw_pre=empty(d, dt=F32) if dn is not None else None)
    gate = x["gate"]
    got["dgate"] = None if gate is None else empty(d, dt=F32) if gate.dim() == 1 else empty(T, d)
    ws = torch.empty(abi.norm_residual_workspace(T, d), device="cuda", dtype=torch.uint8)
    abi.norm_residual_backward(dn, dy, x["b"], x["r"], gate, x["w_post"], w_pre, rb, ry,
                               got["db"], got["dr"], got["dgate"], got["dw_post"], got["dw_pre"],
                               ws, alpha=alpha, beta=beta)
    return got


def check_norm_grads(got, want):
    for name, w in want.items():
        if w is None:
            continue
        # rows cancel (x - q mean(x q)): bounded against the tensor's size
        size = float(w.abs().max())
        bound = 2e-5 * size + (R.U * w.abs() if got[name].dtype == BF else 0)
        R.within(name, got[name], w, bound)


@pytest.mark.parametrize("T,d", NORM_SIZES)
@pytest.mark.parametrize("gate,rt", [("none", BF), ("channel", BF), ("token", F32),
                                     ("channel", F32), ("token", BF)])
def test_norm_backward(rng, T, d, gate, rt):
    x = norm_inputs(rng, T, d, gate, rt)
    dn, dy = randn(rng, T, d), randn(rng, T, d, dt=rt)
    got = norm_grads(x, dn, dy)
    check_norm_grads(got, R.norm_backward(dn, dy, x["b"], x["r"], x["gate"], x["w_post"],
                                          x["w_pre"], 0.9, 0.7, 1e-5))


@pytest.mark.parametrize("d", [64, 1024, 3000])
def test_norm_backward_parts(rng, d):
    """No branch; no next norm; no dy; dr over dy; the same bits twice."""
    T = 41
    x = norm_inputs(rng, T, d, "channel", F32)
    dn, dy = randn(rng, T, d), randn(rng, T, d, dt=F32)
    args = (x["w_post"], x["w_pre"], 0.9, 0.7, 1e-5)
    check_norm_grads(norm_grads(x, dn, None),
                     R.norm_backward(dn, None, x["b"], x["r"], x["gate"], *args))
    only = dict(x, b=None, gate=None, w_post=None)
    check_norm_grads(norm_grads(only, dn, dy),
                     R.norm_backward(dn, dy, None, x["r"], None, None, *args[1:]))
    check_norm_grads(norm_grads(x, None, dy),
                     R.norm_backward(None, dy, x["b"], x["r"], x["gate"], args[0], None, *args[2:]))
    a = norm_grads(x, dn, dy)
    over = dy.clone()
    b = norm_grads(x, dn, over, dr=over)
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_norm_backward_against_differences(rng):
    """Directional derivatives of a 64-bit loss."""
    T, d = 5, 72
    x = norm_inputs(rng, T, d, "channel", F32)
    dn, dy = randn(rng, T, d), randn(rng, T, d, dt=F32)
    got = norm_grads(x, dn, dy)

    def loss(z):
        y, n, _, _ = R.norm_forward(z["b"], z["r"], z["gate"], z["w_post"], z["w_pre"], 0.9, 0.7, 1e-5)
        return float((n * dn.double()).sum() + (y * dy.double()).sum())

    h = 1e-5
    for name, grad in (("b", "db"), ("r", "dr"), ("gate", "dgate"), ("w_post", "dw_post"),
                       ("w_pre", "dw_pre")):
        v = torch.randn(x[name].shape, generator=rng, device="cuda", dtype=torch.float64)
        up, down = ({**x, name: x[name].double() + s * h * v} for s in (1, -1))
        diff = (loss(up) - loss(down)) / (2 * h)
        dot = float((got[grad].double() * v).sum())
        size = float((got[grad].double().abs() * v.abs()).sum())
        assert abs(diff - dot) <= (R.U if got[grad].dtype == BF else 1e-4) * size, name


# ------------------------------------------------------------------ rotary

@pytest.mark.parametrize("kw", [dict(), dict(scaling="linear", factor=4.0),
                                dict(scaling="base", factor=8.0, base=500000.0),
                                dict(scaling="by_parts", factor=16.0, orig_len=4096.0)])
def test_rotary_table(kw):
    rows, rot = 70001, 96
    t = empty(rows, rot // 2, 2, dt=F32)
    abi.rotary_table(t, **kw)
    a = R.rotary_angles(rows, rot, **kw)
    want = torch.stack((a.cos(), a.sin()), -1).cuda()
    # the angle in 64 bits (its own rounding grows with the position), one
    # rounding to fp32
    R.within("table", t, want, 2.0 ** -23 + 70001 * 2.0 ** -50)


def test_rotary_table_magnitude():
    t, u = empty(9, 8, 2, dt=F32), empty(9, 8, 2, dt=F32)
    abi.rotary_table(t, magnitude=1.0)
    abi.rotary_table(u, magnitude=2.0)
    assert torch.equal(2 * t, u)


@pytest.mark.parametrize("T,hq,hk,D,rot", [(1, 1, 1, 64, 64), (1, 48, 8, 128, 128),
                                           (5, 3, 1, 128, 32), (77, 6, 2, 72, 48),
                                           (1001, 5, 5, 96, 96), (3000, 16, 4, 128, 64),
                                           (13, 2, 0, 40, 16), (4, 1, 1, 256, 256)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_rotary(rng, T, hq, hk, D, rot, interleaved, inverse):
    """Heads of one projection's output (strided) to tensors of their own, and
    in place."""
    table = torch.randn(512, rot // 2, 2, generator=rng, device="cuda")
    pos = torch.randint(0, 512, (T,), generator=rng, device="cuda", dtype=torch.int32)
    qkv = randn(rng, T, hq + 2 * max(1, hk), D)
    q, k = qkv[:, :hq], qkv[:, hq:hq + hk] if hk else None
    qo, ko = empty(T, hq, D), empty(T, hk, D) if hk else None
    st = status()
    abi.rotary(q, k, table, pos, qo, ko, st, interleaved=interleaved, inverse=inverse)
    before = qkv.clone()
    abi.rotary(q, k, table, pos, q, k, st, interleaved=interleaved, inverse=inverse)
    assert int(st) == 0
    for name, x, got, now in (("q", before[:, :hq], qo, q),
                              ("k", before[:, hq:hq + hk], ko, k))[:2 if hk else 1]:
        want = R.rotary(x, table, pos, rot, interleaved, inverse)
        # the products' magnitudes: in either direction one of a pair's two
        # outputs is their sum
        mag = sum(R.rotary(x.double().abs(), table.abs(), pos, rot, interleaved, e).abs()
                  for e in (False, True))
        R.within(name, got, want, R.U * want.abs() + 8 * R.EPS * mag)
        assert torch.equal(got, now), name
        assert torch.equal(got[..., rot:], x[..., rot:])
    assert torch.equal(before[:, hq + hk:], qkv[:, hq + hk:])


def test_rotary_default_positions_and_inverse(rng):
    T, D = 40, 64
    table = empty(64, 32, 2, dt=F32)
    abi.rotary_table(table)
    q = randn(rng, T, 2, D)
    a, b = empty(T, 2, D), empty(T, 2, D)
    st = status()
    abi.rotary(q, None, table, None, a, None, st)
    abi.rotary(q, None, table, torch.arange(T, device="cuda", dtype=torch.int32), b, None, st)
    assert torch.equal(a, b)
    abi.rotary(a, None, table, None, b, None, st, inverse=True)
    R.within("there and back", b, q, 3 * R.U * q.double().abs().amax(-1, keepdim=True))


def test_rotary_position_outside_the_table(rng):
    """That token's outputs stay as they were, and the status says so."""
    table = torch.ones(8, 8, 2, device="cuda")
    q = randn(rng, 4, 1, 16)
    out = torch.zeros_like(q)
    st = status()
    pos = torch.tensor([0, 8, -1, 7], device="cuda", dtype=torch.int32)
    abi.rotary(q, None, table, pos, out, None, st)
    assert int(st) == abi.MOE_EINVAL
    assert not out[1].any() and not out[2].any() and bool(out[0].any()) and bool(out[3].any())


# ------------------------------------------------------------------ attention

def run_attention(q, k, v, cu, dout=None, scale=None):
    T, hq, D = q.shape
    hk = k.shape[1]
    plan = abi.AttentionPlan(torch.tensor(cu, device="cuda", dtype=torch.int32), T, hq, hk, D)
    st = status()
    out, rest, lse = empty(T, hq, D), empty(T, hq, D), empty(hq, T, dt=F32)
    abi.attention(plan, q, k, v, out, lse, st, scale=scale, rest=rest if dout is not None else None)
    got = {"out": out, "lse": lse}
    if dout is not None:
        got.update(dq=empty(T, hq, D), dk=empty(T, hk, D), dv=empty(T, hk, D))
        ws = torch.empty(plan.backward_ws_bytes, device="cuda", dtype=torch.uint8)
        abi.attention_backward(plan, q, k, v, out, rest, lse, dout, got["dq"], got["dk"],
                               got["dv"], ws, st, scale=scale)
    assert int(st) == 0 and int(plan.status) == 0
    return got


def check_attention(got, want):
    for name, (w, bound) in want.items():
        if name == "lse":
            some = torch.isfinite(w)
            assert torch.equal(torch.isfinite(got["lse"]), some)
            R.within("lse", got["lse"][some], w[some], 1e-5 + 1e-5 * w[some].abs())
        else:
            # a value below bf16's smallest normal number may round to it
            R.within(name, got[name], w, bound + 1e-30)


ATT = [  # lengths, hq, hk, D
    ([1], 1, 1, 64), ([2], 2, 1, 128), ([127], 2, 2, 64), ([128], 2, 1, 128), ([129], 1, 1, 128),
    ([256], 3, 1, 64), ([257], 2, 1, 128), ([1, 1, 1], 4, 2, 64), ([0, 5, 0, 130, 1], 6, 2, 128),
    ([300, 1, 511], 4, 1, 80), ([640], 5, 5, 128), ([1000], 8, 2, 96), ([385, 77], 3, 1, 128),
    ([200], 2, 1, 8), ([150, 300], 4, 4, 40), ([1537], 2, 1, 128), ([2000], 1, 1, 64),
]


@pytest.mark.parametrize("lens,hq,hk,D", ATT)
def test_attention(rng, lens, hq, hk, D):
    T = sum(lens)
    q, k, v = randn(rng, T, hq, D, std=2.0), randn(rng, T, hk, D), randn(rng, T, hk, D)
    dout = randn(rng, T, hq, D)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    got = run_attention(q, k, v, cu, dout)
    check_attention(got, R.attention(q, k, v, lens, D ** -0.5, dout=dout))
    again = run_attention(q, k, v, cu, dout)
    for n in got:
        assert torch.equal(got[n], again[n]), n
    assert torch.equal(run_attention(q, k, v, cu)["out"], got["out"])


def test_attention_strided_views(rng):
    """Heads of one projection's output; head-major tensors; out with gaps."""
    T, hq, hk, D = 210, 4, 2, 64
    lens = [130, 80]
    qkv = randn(rng, T, hq + 2 * hk, D)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    want = run_attention(q.contiguous(), k.contiguous(), v.contiguous(), [0, 130, 210])["out"]
    assert torch.equal(run_attention(q, k, v, [0, 130, 210])["out"], want)
    qm, km, vm = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v))
    dout = randn(rng, hq, T, D).transpose(0, 1)
    plan = abi.AttentionPlan(torch.tensor([0, 130, 210], device="cuda", dtype=torch.int32), T, hq,
                             hk, D)
    st = status()
    wide = torch.zeros(T, 2 * hq, D, device="cuda", dtype=BF)
    rest = torch.zeros_like(wide)[:, ::2]
    lse = empty(hq, T, dt=F32)
    abi.attention(plan, qm, km, vm, wide[:, ::2], lse, st, rest=rest)
    assert torch.equal(wide[:, ::2], want) and not wide[:, 1::2].any()
    grads = torch.zeros(T, hq + 2 * hk, D, device="cuda", dtype=BF)
    ws = torch.empty(plan.backward_ws_bytes, device="cuda", dtype=torch.uint8)
    dq, dk, dv = grads[:, :hq], grads[:, hq:hq + hk], grads[:, hq + hk:]
    abi.attention_backward(plan, qm, km, vm, wide[:, ::2], rest, lse, dout, dq, dk, dv, ws, st)
    ref = R.attention(q, k, v, lens, D ** -0.5, dout=dout)
    check_attention({"out": wide[:, ::2], "lse": lse, "dq": dq, "dk": dk, "dv": dv}, ref)
    assert int(st) == 0


@pytest.mark.parametrize("hq,hk", [(4, 2), (3, 1)])
def test_attention_tokens_of_no_sequence(rng, hq, hk):
    """Before the first and after the last sequence: zeros and lse -inf, and
    whatever stands there (NaN here) reaches no other token."""
    T, D, first, lens = 700, 128, 37, [200, 0, 133]
    q, k, v, dout = (randn(rng, T, h, D) for h in (hq, hk, hk, hq))
    cu = [37, 237, 237, 370]
    for t in (q, k, v, dout):
        t[:37] = float("nan")
        t[370:] = float("nan")
    got = run_attention(q, k, v, cu, dout)
    part = slice(37, 370)
    want = R.attention(q[part], k[part], v[part], lens, D ** -0.5, dout=dout[part])
    for n in ("out", "dq", "dk", "dv"):
        assert not got[n][:37].any() and not got[n][370:].any(), n
    assert bool((got["lse"][:, :37] == -math.inf).all()) and bool((got["lse"][:, 370:] == -math.inf).all())
    check_attention({n: (t[part] if n != "lse" else t[:, part]) for n, t in got.items()}, want)


def test_attention_no_sequence_and_no_token(rng):
    q = randn(rng, 5, 2, 64)
    got = run_attention(q, q, q, [0], q)
    for n in ("out", "dq", "dk", "dv"):
        assert not got[n].any()
    run_attention(q[:0], q[:0], q[:0], [0, 0], q[:0])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("hq,hk,D", [(2, 1, 128), (1, 1, 64)])
def test_attention_hidden_values_stay_hidden(rng, bad, hq, hk, D):
    """A non-finite key, value or gradient reaches the tokens that see it and
    no other: rows before it, other sequences, keys after its query."""
    lens, T, hit = [140, 300, 50], 490, 140 + 170
    q, k, v, dout = (randn(rng, T, h, D) for h in (hq, hk, hk, hq))
    cu = [0, 140, 440, 490]
    clean = run_attention(q, k, v, cu, dout)
    kb, vb, db = k.clone(), v.clone(), dout.clone()
    kb[hit, 0, 3] = bad
    vb[hit, 0, 5] = bad
    free = torch.ones(T, dtype=torch.bool, device="cuda")
    free[hit:440] = False                      # tokens that attend to it
    got = run_attention(q, kb, vb, cu, dout)
    for n in ("out", "dq"):
        R.within(n, got[n][free], clean[n][free], 2 * R.U * clean[n][free].double().abs() + 1e-2)
    assert torch.equal(got["lse"][:, free], clean["lse"][:, free])
    other = torch.ones(T, dtype=torch.bool, device="cuda")
    other[140:440] = False                     # its sequence's keys share its rows
    for n in ("dk", "dv"):
        assert torch.equal(got[n][other], clean[n][other]), n
    # a query's gradient reaches the keys up to it
    db[hit] = bad
    got = run_attention(q, k, v, cu, db)
    later = torch.ones(T, dtype=torch.bool, device="cuda")
    later[140:hit + 1] = False
    for n in ("dk", "dv"):
        R.within(n, got[n][later], clean[n][later], 2 * R.U * clean[n][later].double().abs() + 1e-2)
    rows = torch.ones(T, dtype=torch.bool, device="cuda")
    rows[hit] = False
    R.within("dq", got["dq"][rows], clean["dq"][rows], 2 * R.U * clean["dq"][rows].double().abs() + 1e-2)


def test_attention_large_scores_and_scale(rng):
    """Rows of one key, maxima that rise block after block, a given scale."""
    T, D = 515, 64
    q, k, v, dout = (randn(rng, T, 1, D) for _ in range(4))
    k = (k.float() * torch.linspace(0.1, 12, T, device="cuda")[:, None, None]).to(BF)
    got = run_attention(q, k, v, [0, T], dout, scale=0.5)
    check_attention(got, R.attention(q, k, v, [T], 0.5, dout=dout))


def test_attention_plan_refuses_bad_sequences():
    for cu in ([0, 50, 40], [-1, 10], [0, 200]):
        plan = abi.AttentionPlan(torch.tensor(cu, device="cuda", dtype=torch.int32), 100, 2, 1, 64)
        assert int(plan.status) == abi.MOE_EINVAL, cu


def test_attention_plan_refill(rng):
    q, k, v = (randn(rng, 300, 2, 64) for _ in range(3))
    dev = lambda *cu: torch.tensor(cu, device="cuda", dtype=torch.int32)  # noqa: E731
    plan = abi.AttentionPlan(dev(0, 10, 300), 300, 2, 2, 64)
    plan.refill(dev(0, 222, 300))
    out, lse = empty(300, 2, 64), empty(2, 300, dt=F32)
    abi.attention(plan, q, k, v, out, lse, status())
    assert torch.equal(out, run_attention(q, k, v, [0, 222, 300])["out"])


def test_attention_gradient_against_differences(rng):
    """Directional derivatives of a 64-bit loss."""
    lens, hq, hk, D = [70, 3], 4, 2, 16
    T = sum(lens)
    x = {n: randn(rng, T, h, D) for n, h in (("q", hq), ("k", hk), ("v", hk))}
    dout = randn(rng, T, hq, D)
    got = run_attention(x["q"], x["k"], x["v"], [0, 70, 73], dout)

    def loss(z):
        return float((R.attention(z["q"], z["k"], z["v"], lens, D ** -0.5)["out"][0] * dout.double()).sum())

    for name in x:
        u = torch.randn(x[name].shape, generator=rng, device="cuda", dtype=torch.float64)
        up, down = ({**x, name: x[name].double() + s * 1e-5 * u} for s in (1, -1))
        diff = (loss(up) - loss(down)) / 2e-5
        g = got["d" + name].double()
        # three roundings to bf16 on the way to a gradient
        assert abs(diff - float((g * u).sum())) <= 3 * R.U * float((g.abs() * u.abs()).sum()), name


def test_attention_in_a_graph_and_on_another_stream(rng):
    T, hq, hk, D = 333, 4, 2, 128
    q, k, v, dout = (randn(rng, T, h, D) for h in (hq, hk, hk, hq))
    want = run_attention(q, k, v, [0, 333], dout)
    cu = torch.tensor([0, 333], device="cuda", dtype=torch.int32)
    plan = abi.AttentionPlan(cu, T, hq, hk, D)
    st = status()
    out, rest, lse = empty(T, hq, D), empty(T, hq, D), empty(hq, T, dt=F32)
    dq, dk, dv = empty(T, hq, D), empty(T, hk, D), empty(T, hk, D)
    ws = torch.empty(plan.backward_ws_bytes, device="cuda", dtype=torch.uint8)

    def step():
        plan.refill(cu)
        abi.attention(plan, q, k, v, out, lse, st, rest=rest)
        abi.attention_backward(plan, q, k, v, out, rest, lse, dout, dq, dk, dv, ws, st)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(dk, want["dk"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for t in (out, dq, dk, dv):
        t.fill_(float("nan"))
    g.replay()
    for n, t in (("out", out), ("dq", dq), ("dk", dk), ("dv", dv)):
        assert torch.equal(t, want[n]), n


# ------------------------------------------------------------------ gradient clipping

def run_clip(tensors, max_norm, outs=None):
    norm = empty(1, dt=F32)
    s = abi.GradSet(tensors, outs)
    abi.grad_clip(s, max_norm, norm)
    return float(norm)


@pytest.mark.parametrize("sizes", [[1], [7], [16384], [16385, 1, 3], [0, 5, 0], [100000, 0, 12, 65536, 8],
                                   [3] * 64, [5] * 65, [1000] * 700])
@pytest.mark.parametrize("kinds", ["f32", "bf16", "mixed"])
@pytest.mark.parametrize("share", [0.3, 2.0])
def test_grad_clip(rng, sizes, kinds, share):
    kind = lambda i: {"f32": F32, "bf16": BF, "mixed": (F32, BF)[i % 2]}[kinds]  # noqa: E731
    x = [randn(rng, n, dt=kind(i)) for i, n in enumerate(sizes)]
    want = math.sqrt(sum(float(t.double().square().sum()) for t in x))
    outs = [empty(n, dt=kind(i)) for i, n in enumerate(sizes)]
    norm = run_clip(x, share * want, outs)
    assert abs(norm - want) <= 1e-6 * want
    c = min(1.0, share * want / (want + 1e-6))
    for i, (a, b) in enumerate(zip(x, outs)):
        w = a.double() * c
        R.within(f"tensor {i}", b, w, 1e-6 * w.abs() + (R.U * w.abs() if b.dtype == BF else 0))
        if c == 1.0:
            assert torch.equal(a, b)
    norm2 = run_clip(x, share * want)          # in place
    assert norm2 == norm
    for a, b in zip(x, outs):
        assert torch.equal(a, b)


def test_grad_clip_alignment(rng):
    """Views that start off a 16-byte boundary."""
    base, out = randn(rng, 50001, dt=F32), empty(50003, dt=F32)
    b16 = randn(rng, 40001)
    x, o = [base[1:], b16[3:]], [out[3:], torch.zeros(39998 + 1, device="cuda", dtype=BF)[1:]]
    want = math.sqrt(sum(float(t.double().square().sum()) for t in x))
    assert abs(run_clip(x, 0.5 * want, o) - want) <= 1e-6 * want
    c = 0.5 * want / (want + 1e-6)
    R.within("f32", o[0], x[0].double() * c, 1e-6 * x[0].double().abs())
    R.within("bf16", o[1], x[1].double() * c, (R.U + 1e-6) * x[1].double().abs())
    assert bool(out[:3].isnan().all())


@pytest.mark.parametrize("size", [1e-30, 1e-22, 3e19, 1e30])
def test_grad_clip_far_from_one(rng, size):
    """Squares that leave fp32's range; zeros among them."""
    x = [(torch.randn(40000, generator=rng, device="cuda", dtype=torch.float64) * size).float(),
         torch.zeros(30000, device="cuda")]
    want = math.sqrt(float(x[0].double().square().sum()))
    c = min(1.0, want * 0.5 / (want + 1e-6))
    before = x[0].double()
    assert abs(run_clip(x, want * 0.5) - want) <= 1e-6 * want
    R.within("x", x[0], before * c, 1e-6 * before.abs() * c + 1e-44)
    assert not x[1].any()


def test_grad_clip_zero_and_not_finite(rng):
    z = [torch.zeros(100, device="cuda")]
    assert run_clip(z, 1.0) == 0.0 and not z[0].any()
    for bad in (float("nan"), float("inf")):
        x = [randn(rng, 20000, dt=F32), randn(rng, 50)]
        x[0][12345] = bad
        keep = [t.clone() for t in x]
        outs = [empty(20000, dt=F32), empty(50)]
        assert not math.isfinite(run_clip(x, 1.0, outs))
        for a, b, o in zip(keep, x, outs):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
            assert torch.equal(a.isnan(), o.isnan()) and torch.equal(a[~a.isnan()], o[~o.isnan()])


def test_norm_and_clip_in_a_graph(rng):
    """Captured, replayed on new values: as called."""
    T, d = 70, 2048
    x = norm_inputs(rng, T, d, "channel", BF)
    dn, dy = randn(rng, T, d), randn(rng, T, d)
    st = torch.empty(2, T, device="cuda")
    y, n, db, dr = (empty(T, d) for _ in range(4))
    dg, dq, dp = (empty(d, dt=F32) for _ in range(3))
    ws = torch.empty(abi.norm_residual_workspace(T, d), device="cuda", dtype=torch.uint8)
    grads = abi.GradSet([dg, dq, dp, db])
    norm = empty(1, dt=F32)

    def step():
        abi.norm_residual(x["b"], x["r"], x["gate"], x["w_post"], x["w_pre"], y, n, st[0], st[1])
        abi.norm_residual_backward(dn, dy, x["b"], x["r"], x["gate"], x["w_post"], x["w_pre"],
                                   st[0], st[1], db, dr, dg, dq, dp, ws)
        abi.grad_clip(grads, 0.5, norm)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for t in x.values():
        t.copy_(t * 0.75)
    step()
    want = [t.clone() for t in (y, n, db, dr, dg, dq, dp, norm)]
    for t in (y, n, db, dr, dg, dq, dp, norm):
        t.fill_(float("nan"))
    g.replay()
    for a, b in zip((y, n, db, dr, dg, dq, dp, norm), want):
        assert torch.equal(a, b)
