"""Cases and plain forms of the operators around the MoE layer in a training block.

Four operators: ``norm`` (norm after a branch, gate, residual sum, norm before
the next branch; forward and backward), ``rotary`` (positions turned into the
query and key heads, forward and inverse), ``attention`` (causal, packed
sequences, grouped heads; forward, and a training step of forward and
backward) and ``clip`` (the global gradient norm over many tensors, and
clipping).  ``own`` chooses between the plain forms, in 32 bits from
elementary torch operations, and the framework's kernels.
"""
import math
import random

import numpy as np
import torch

own = False

BF, F32 = torch.bfloat16, torch.float32


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of a served batch at the mid layer's width: all latency
        {"name": "norm one token", "op": "norm", "dir": "forward", "T": 1, "d": 2048, "gate": "channel", "res": "bf16"},
        # the full layer's batch and width, one gate value a channel
        {"name": "norm full", "op": "norm", "dir": "forward", "T": 16384, "d": 6144, "gate": "channel", "res": "bf16"},
        # its backward: three sums over all tokens beside the rows
        {"name": "norm full backward", "op": "norm", "dir": "backward", "T": 16384, "d": 6144, "gate": "channel", "res": "bf16"},
        # the mid layer with an odd batch, a gate value for each token and channel, a residual stream in 32 bits
        {"name": "norm mid backward", "op": "norm", "dir": "backward", "T": 8191, "d": 2048, "gate": "token", "res": "f32"},
        # the mid layer's two sequences, heads side by side in one q, k, v tensor
        {"name": "rotary mid", "op": "rotary", "dir": "forward", "T": 8192, "seq": 4096, "hq": 16, "hk": 4, "D": 128, "rot": 128, "layout": "half"},
        # one long sequence, half of each head turned, pairs side by side, the gradient's direction
        {"name": "rotary long backward", "op": "rotary", "dir": "backward", "T": 65536, "seq": 65536, "hq": 48, "hk": 8, "D": 128, "rot": 64, "layout": "pairs"},
        # a handful of short prompts of odd lengths: latency
        {"name": "attention short", "op": "attention", "dir": "forward", "T": 301, "seqs": 5, "cut": 1, "spread": 1.0, "hq": 8, "hk": 2, "D": 64},
        # the full layer's batch: sequences of different lengths packed into 16384 tokens
        {"name": "attention full", "op": "attention", "dir": "forward", "T": 16384, "seqs": 7, "cut": 2, "spread": 0.4, "hq": 48, "hk": 8, "D": 128},
        # one long prompt, few heads
        {"name": "attention long", "op": "attention", "dir": "forward", "T": 32768, "seqs": 1, "cut": 3, "spread": 1.0, "hq": 8, "hk": 2, "D": 128},
        # a training step of the mid layer's batch: forward and gradients
        {"name": "attention step mid", "op": "attention", "dir": "step", "T": 8192, "seqs": 4, "cut": 4, "spread": 0.4, "hq": 16, "hk": 4, "D": 128},
        # the gradients of the tiny layer, in 32 bits: latency
        {"name": "clip tiny", "op": "clip", "n": 700_000, "tensors": 9, "cut": 5, "mixed": False, "clipped": True},
        # the gradients of a layer of the mid layer's size, in 32 bits and bf16
        {"name": "clip mid", "op": "clip", "n": 180_000_000, "tensors": 10, "cut": 6, "mixed": True, "clipped": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "rotary", "attention", "attention", "clip"))
    if op == "norm":
        d = 8 * _log(rng, 8, 1024)
        return {"op": op, "dir": rng.choice(("forward", "backward")), "T": _log(rng, 1, min(65536, 16384 * 6144 // d)), "d": d,
                "gate": rng.choice(("channel", "token", "none")), "res": rng.choice(("bf16", "f32"))}
    if op == "rotary":
        D, hk = rng.choice((64, 96, 128)), rng.choice((1, 2, 4, 8))
        hq = hk * rng.choice((1, 2, 3, 4, 6))
        T = _log(rng, 1, 65536)
        return {"op": op, "dir": rng.choice(("forward", "backward")), "T": T, "seq": max(1, T // rng.randint(1, 4)), "hq": hq, "hk": hk, "D": D,
                "rot": rng.choice((D, D // 2)), "layout": rng.choice(("half", "pairs"))}
    if op == "attention":
        while True:
            D, hk = rng.choice((64, 80, 96, 128)), rng.choice((1, 2, 4, 8))
            T = _log(rng, 1, 16384)
            c = {"op": op, "dir": rng.choice(("forward", "step")), "T": T, "seqs": min(T, _log(rng, 1, 24)), "cut": rng.randint(0, 10**6),
                 "spread": rng.choice((0.3, 1.0)), "hq": hk * rng.choice((1, 2, 3, 4, 6)), "hk": hk, "D": D}
            most = max(lengths(c))
            # within the longest listed prompt's work, and within memory in its plain form
            if work(c)["flops"] <= 4 * 128 * 8 * 32768 * 32768 / 2 and c["seqs"] * c["hq"] * most * most * 4 <= 20e9:
                return c
    return {"op": op, "n": _log(rng, 100, 180_000_000), "tensors": rng.randint(1, 48), "cut": rng.randint(0, 10**6), "mixed": rng.random() < 0.5,
            "clipped": rng.random() < 0.75}


def lengths(case):
    """The packed sequences' lengths: odd, of very different sizes, one of them a single token where there are several."""
    T, n = case["T"], case["seqs"]
    if n == 1:
        return [T]
    rng = random.Random(case["cut"])
    w = [math.exp(rng.gauss(0, case["spread"])) for _ in range(n - 1)]
    got = [max(1, int((T - 1) * v / sum(w))) for v in w] + [1]
    while sum(got) > T:
        got[got.index(max(got))] -= 1
    got[0] += T - sum(got)
    return got


def sizes(case):
    """Elements of each gradient: from vectors to a tensor that holds most of them, odd ones among them."""
    n, k = case["n"], min(case["tensors"], case["n"])
    rng = random.Random(case["cut"])
    w = [math.exp(rng.gauss(0, 2)) for _ in range(k)]
    got = [max(1, int(n * v / sum(w))) for v in w]
    while sum(got) > n and max(got) > 1:
        got[got.index(max(got))] -= min(sum(got) - n, max(got) - 1)
    return got


def _pairs(case):
    return sum(n * (n + 1) // 2 for n in lengths(case))


def work(case):
    op = case["op"]
    if op == "norm":
        T, d, r = case["T"], case["d"], 2 if case["res"] == "bf16" else 4
        g = 2 * T * d if case["gate"] == "token" else 0
        if case["dir"] == "forward":
            return {"bytes": T * d * (4 + 2 * r) + g, "flops": 10 * T * d}
        return {"bytes": T * d * (6 + 3 * r) + 2 * g, "flops": 24 * T * d}
    if op == "rotary":
        return {"bytes": 4 * case["T"] * (case["hq"] + case["hk"]) * case["D"], "flops": 3 * case["T"] * (case["hq"] + case["hk"]) * case["rot"]}
    if op == "attention":
        T, hq, hk, D = case["T"], case["hq"], case["hk"], case["D"]
        step = case["dir"] == "step"
        return {"bytes": 2 * T * D * ((2 * hq + 2 * hk) + (3 * hq + 2 * hk if step else 0)), "flops": (14 if step else 4) * D * hq * _pairs(case)}
    kinds = _kinds(case)
    return {"bytes": sum(2 * n * (2 if k == BF else 4) for n, k in zip(sizes(case), kinds)), "flops": 3 * case["n"]}


def _kinds(case):
    return [BF if case["mixed"] and i % 3 == 2 else F32 for i in range(len(sizes(case)))]


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    draw_ = lambda *s, std=1.0, dt=BF: (torch.randn(s, generator=g, device=dev, dtype=F32) * std).to(dt)  # noqa: E731
    out = lambda *s, dt=BF: torch.empty(s, device=dev, dtype=dt)  # noqa: E731
    s = dict(case=case, op=case["op"])
    if case["op"] == "norm":
        T, d, rt = case["T"], case["d"], BF if case["res"] == "bf16" else F32
        s.update(b=draw_(T, d), r=draw_(T, d, std=2.0, dt=rt), w_post=1 + draw_(d, std=0.1), w_pre=1 + draw_(d, std=0.1), alpha=0.97, beta=0.5, eps=1e-6)
        s["gate"] = {"none": lambda: None, "channel": lambda: draw_(d, std=0.5), "token": lambda: draw_(T, d, std=0.5)}[case["gate"]]()
        s["rstd_post"], s["rstd_pre"] = out(T, dt=F32), out(T, dt=F32)
        if case["dir"] == "forward":
            s.update(y=out(T, d, dt=rt), n=out(T, d))
        else:  # the forward's statistics are in hand, as a training step keeps them
            s.update(dn=draw_(T, d, std=1e-2), dy=draw_(T, d, std=1e-2, dt=rt))
            for a in range(0, T, 4096):
                at = slice(a, a + 4096)
                b, r = s["b"][at].double(), s["r"][at].double()
                rb = torch.rsqrt((b * b).mean(1) + s["eps"])
                gate = 1.0 if s["gate"] is None else (s["gate"] if s["gate"].dim() == 1 else s["gate"][at]).double()
                y = s["alpha"] * r + s["beta"] * gate * (b * rb[:, None] * s["w_post"].double())
                s["rstd_post"][at], s["rstd_pre"][at] = rb.float(), torch.rsqrt((y * y).mean(1) + s["eps"]).float()
            s.update(db=out(T, d), dr=out(T, d, dt=rt), dw_post=out(d, dt=F32), dw_pre=out(d, dt=F32))
            s["dgate"] = None if s["gate"] is None else out(d, dt=F32) if s["gate"].dim() == 1 else out(T, d)
            if own:
                from moe_routing_capacity_gb300 import abi
                s["ws"] = out(abi.norm_residual_workspace(T, d), dt=torch.uint8)
    elif case["op"] == "rotary":
        T, hq, hk, D = case["T"], case["hq"], case["hk"], case["D"]
        s["pos"] = (torch.arange(T, device=dev) % case["seq"]).to(torch.int32)
        f = 10000.0 ** (-torch.arange(0, case["rot"], 2, device=dev, dtype=torch.float64) / case["rot"])
        a = torch.arange(case["seq"], device=dev, dtype=torch.float64)[:, None] * f
        s["table"] = torch.stack((a.cos(), a.sin()), -1).float()  # [positions, rot / 2, 2], made once
        if case["dir"] == "forward":  # heads of one projection's output
            qkv = draw_(T, hq + 2 * hk, D)
            s.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hk])
        else:
            s.update(q=draw_(T, hq, D, std=1e-2), k=draw_(T, hk, D, std=1e-2))
        s.update(q_out=out(T, hq, D), k_out=out(T, hk, D))
        s["status"] = torch.zeros(1, device=dev, dtype=torch.int32)
    elif case["op"] == "attention":
        T, hq, hk, D, n = case["T"], case["hq"], case["hk"], case["D"], lengths(case)
        s.update(q=draw_(T, hq, D, std=2.0), k=draw_(T, hk, D), v=draw_(T, hk, D), scale=D ** -0.5, lens=n)
        at = np.concatenate([[0], np.cumsum(n)])
        s["cu"] = torch.tensor(at, dtype=torch.int32, device=dev)
        s.update(out=out(T, hq, D))
        if case["dir"] == "step":
            s.update(dout=draw_(T, hq, D, std=1e-2), dq=out(T, hq, D), dk=out(T, hk, D), dv=out(T, hk, D))
        # where the packed tokens stand in [sequences, longest], for the plain form's products
        s["rows"] = torch.tensor(np.concatenate([np.arange(m) + i * max(n) for i, m in enumerate(n)]), device=dev)
        if own:
            from moe_routing_capacity_gb300 import abi
            s["plan"] = abi.AttentionPlan(s["cu"], T, hq, hk, D)
            s["lse"] = out(hq, T, dt=F32)
            s["status"] = torch.zeros(1, device=dev, dtype=torch.int32)
            if case["dir"] == "step":
                s["rest"], s["ws"] = out(T, hq, D), out(s["plan"].backward_ws_bytes, dt=torch.uint8)
    else:
        n, kinds = sizes(case), _kinds(case)
        s["grads"] = [draw_(m, std=1e-3 * (1 + i % 3), dt=k) for i, (m, k) in enumerate(zip(n, kinds))]
        s["outs"] = [torch.empty_like(x) for x in s["grads"]]
        s["norm"] = out(1, dt=F32)
        # about a third of what the norm comes to, or twice
        s["max_norm"] = (0.37 if case["clipped"] else 2.0) * 1e-3 * math.sqrt(sum(m * (1 + i % 3) ** 2 for i, m in enumerate(n)))
        if own:
            from moe_routing_capacity_gb300 import abi
            s["set"] = abi.GradSet(s["grads"], s["outs"])
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    if own:
        return _OWN[s["op"]](s, case)
    return _PLAIN[s["op"]](s, case)


def _own_norm(s, case):
    from moe_routing_capacity_gb300 import abi
    if case["dir"] == "forward":
        abi.norm_residual(s["b"], s["r"], s["gate"], s["w_post"], s["w_pre"], s["y"], s["n"], s["rstd_post"], s["rstd_pre"],
                          alpha=s["alpha"], beta=s["beta"], eps=s["eps"])
        return {"y": s["y"], "n": s["n"]}
    abi.norm_residual_backward(s["dn"], s["dy"], s["b"], s["r"], s["gate"], s["w_post"], s["w_pre"], s["rstd_post"], s["rstd_pre"], s["db"], s["dr"],
                               s["dgate"], s["dw_post"], s["dw_pre"], s["ws"], alpha=s["alpha"], beta=s["beta"])
    got = {"db": s["db"], "dr": s["dr"], "dw_post": s["dw_post"], "dw_pre": s["dw_pre"]}
    return got if s["dgate"] is None else {**got, "dgate": s["dgate"]}


def _own_rotary(s, case):
    from moe_routing_capacity_gb300 import abi
    abi.rotary(s["q"], s["k"], s["table"], s["pos"], s["q_out"], s["k_out"], s["status"], interleaved=case["layout"] == "pairs",
               inverse=case["dir"] == "backward")
    return {"q": s["q_out"], "k": s["k_out"]}


def _own_attention(s, case):
    from moe_routing_capacity_gb300 import abi
    step = case["dir"] == "step"
    abi.attention(s["plan"], s["q"], s["k"], s["v"], s["out"], s["lse"], s["status"], scale=s["scale"], rest=s["rest"] if step else None)
    if not step:
        return {"out": s["out"]}
    abi.attention_backward(s["plan"], s["q"], s["k"], s["v"], s["out"], s["rest"], s["lse"], s["dout"], s["dq"], s["dk"], s["dv"], s["ws"], s["status"],
                           scale=s["scale"])
    return {"out": s["out"], "dq": s["dq"], "dk": s["dk"], "dv": s["dv"]}


def _own_clip(s, case):
    from moe_routing_capacity_gb300 import abi
    abi.grad_clip(s["set"], s["max_norm"], s["norm"])
    return {"norm": s["norm"], "grads": s["outs"]}


def _plain_norm(s, case):
    b, r, wq, wp = s["b"].float(), s["r"].float(), s["w_post"].float(), s["w_pre"].float()
    g = 1.0 if s["gate"] is None else s["gate"].float()
    if case["dir"] == "forward":
        p = b * torch.rsqrt((b * b).mean(1, keepdim=True) + s["eps"])
        y = s["alpha"] * r + s["beta"] * g * (p * wq)
        n = y * torch.rsqrt((y * y).mean(1, keepdim=True) + s["eps"]) * wp
        return {"y": y.to(s["r"].dtype), "n": n.to(BF)}
    dn, dy, rb, ry = s["dn"].float(), s["dy"].float(), s["rstd_post"][:, None], s["rstd_pre"][:, None]
    p = b * rb
    m = p * wq
    q = (s["alpha"] * r + s["beta"] * g * m) * ry
    dq = dn * wp
    du = dy + ry * (dq - q * (dq * q).mean(1, keepdim=True))
    dm = s["beta"] * g * du
    dp = dm * wq
    got = {"db": (rb * (dp - p * (dp * p).mean(1, keepdim=True))).to(BF), "dr": (s["alpha"] * du).to(s["r"].dtype), "dw_post": (dm * p).sum(0),
           "dw_pre": (dn * q).sum(0)}
    if s["gate"] is not None:
        dg = s["beta"] * m * du
        got["dgate"] = dg.sum(0) if s["gate"].dim() == 1 else dg.to(BF)
    return got


def _plain_rotary(s, case):
    cs = s["table"][s["pos"].long()]
    c, t = cs[..., 0][:, None], cs[..., 1][:, None]
    if case["dir"] == "backward":
        t = -t
    rot, half = case["rot"], case["rot"] // 2

    def turn(x):
        f = x.float()
        if case["layout"] == "half":
            x1, x2 = f[..., :half], f[..., half:rot]
            y = torch.cat((x1 * c - x2 * t, x2 * c + x1 * t, f[..., rot:]), -1)
        else:
            x1, x2 = f[..., 0:rot:2], f[..., 1:rot:2]
            y = torch.cat((torch.stack((x1 * c - x2 * t, x2 * c + x1 * t), -1).flatten(-2), f[..., rot:]), -1)
        return y.to(BF)

    return {"q": turn(s["q"]), "k": turn(s["k"])}


def _plain_attention(s, case):
    n, hq, hk, D = s["lens"], case["hq"], case["hk"], case["D"]
    B, L, G = len(n), max(n), hq // hk

    def padded(x):  # [T, h, D] -> [B, hk, h / hk, L, D]
        h = x.shape[1]
        f = torch.zeros(B * L, h, D, device=x.device)
        f[s["rows"]] = x.float()
        return f.view(B, L, hk, h // hk, D).permute(0, 2, 3, 1, 4)

    def packed(f):  # back
        f = f.permute(0, 3, 1, 2, 4).reshape(B * L, -1, D)
        return f[s["rows"]].to(BF)

    q, k, v = padded(s["q"]), padded(s["k"]), padded(s["v"])
    rows = q.reshape(B, hk, G * L, D)  # the group's heads are rows of one product
    ban = torch.ones(L, L, dtype=torch.bool, device=q.device).triu(1)
    p = (rows @ k[:, :, 0].transpose(-1, -2)).view(B, hk, G, L, L)
    p.mul_(s["scale"]).masked_fill_(ban, -math.inf)
    p.sub_(p.amax(-1, keepdim=True)).exp_()
    p.div_(p.sum(-1, keepdim=True))
    flat = p.view(B, hk, G * L, L)
    o = (flat @ v[:, :, 0]).view(B, hk, G, L, D)
    if case["dir"] != "step":
        return {"out": packed(o)}
    do = padded(s["dout"])
    do_rows = do.reshape(B, hk, G * L, D)
    dv = flat.transpose(-1, -2) @ do_rows
    ds = (do_rows @ v[:, :, 0].transpose(-1, -2)).view(B, hk, G, L, L)
    ds.sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(s["scale"])
    ds = ds.view(B, hk, G * L, L)
    dq = (ds @ k[:, :, 0]).view(B, hk, G, L, D)
    dk = ds.transpose(-1, -2) @ rows
    return {"out": packed(o), "dq": packed(dq), "dk": packed(dk[:, :, None]), "dv": packed(dv[:, :, None])}


def _plain_clip(s, case):
    f = [x.float() for x in s["grads"]]
    norm = torch.stack([(x * x).sum() for x in f]).sum().sqrt()
    c = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    return {"norm": norm.reshape(1), "grads": [(x * c).to(g.dtype) for x, g in zip(f, s["grads"])]}


_OWN = {"norm": _own_norm, "rotary": _own_rotary, "attention": _own_attention, "clip": _own_clip}
_PLAIN = {"norm": _plain_norm, "rotary": _plain_rotary, "attention": _plain_attention, "clip": _plain_clip}


# ------------------------------------------------------------------ in 64 bits, from the definitions

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s, case)
    if case["op"] == "rotary":
        return _exact_rotary(s, case)
    if case["op"] == "attention":
        return _exact_attention(s, case)
    total = math.sqrt(math.fsum(float(g.double().square().sum()) for g in s["grads"]))
    c = min(1.0, s["max_norm"] / (total + 1e-6))
    return {"norm": np.array([total]), "grads": [g.double() * c for g in s["grads"]]}


def _exact_norm(s, case):
    """In blocks of tokens; the backward from the Jacobians of x -> x rstd(x)."""
    T, d = case["T"], case["d"]
    back = case["dir"] == "backward"
    new = lambda *shape: torch.zeros(shape, dtype=torch.float64, device=s["b"].device)  # noqa: E731
    per_token = s["gate"] is not None and s["gate"].dim() == 2
    got = {"db": new(T, d), "dr": new(T, d), "dw_post": new(d), "dw_pre": new(d)} if back else {"y": new(T, d), "n": new(T, d)}
    if back and s["gate"] is not None:
        got["dgate"] = new(T, d) if per_token else new(d)
    wq, wp = s["w_post"].double(), s["w_pre"].double()
    for a in range(0, T, 2048):
        at = slice(a, min(T, a + 2048))
        b, r = s["b"][at].double(), s["r"][at].double()
        gate = torch.ones_like(b) if s["gate"] is None else (s["gate"][at] if per_token else s["gate"].expand(b.shape)).double()
        if back:
            rb, ry = s["rstd_post"][at].double().unsqueeze(1), s["rstd_pre"][at].double().unsqueeze(1)
        else:
            rb = 1.0 / torch.sqrt(torch.einsum("td,td->t", b, b) / d + s["eps"]).unsqueeze(1)
        y = r.mul(s["alpha"]) + gate * wq * b * rb * s["beta"]
        if not back:
            ry = 1.0 / torch.sqrt(torch.einsum("td,td->t", y, y) / d + s["eps"]).unsqueeze(1)
            got["y"][at], got["n"][at] = y, wp * y * ry
            continue
        dn = s["dn"][at].double()
        into_y = dn * wp
        along = torch.einsum("td,td->t", into_y, y).unsqueeze(1) / d
        du = s["dy"][at].double() + into_y * ry - y * along * ry ** 3
        got["dr"][at] = du * s["alpha"]
        into_b = du * s["beta"] * gate * wq
        along = torch.einsum("td,td->t", into_b, b).unsqueeze(1) / d
        got["db"][at] = into_b * rb - b * along * rb ** 3
        got["dw_post"] += torch.einsum("td,td->d", du * gate, b * rb) * s["beta"]
        got["dw_pre"] += torch.einsum("td,td->d", dn, y * ry)
        if s["gate"] is not None:
            dg = du * b * rb * wq * s["beta"]
            if per_token:
                got["dgate"][at] = dg
            else:
                got["dgate"] += dg.sum(0)
    return got


def _exact_rotary(s, case):
    """As a product of complex numbers with the table's."""
    T, rot = case["T"], case["rot"]
    z = torch.view_as_complex(s["table"].double().contiguous())[s["pos"].long()].unsqueeze(1)
    if case["dir"] == "backward":
        z = z.conj()
    got = {}
    for name in ("q", "k"):
        y = s[name].double()
        x = y[..., :rot].clone()
        pair = x.unflatten(-1, (2, rot // 2)).transpose(-1, -2) if case["layout"] == "half" else x.unflatten(-1, (rot // 2, 2))
        turned = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
        y[..., :rot] = turned.transpose(-1, -2).reshape(T, -1, rot) if case["layout"] == "half" else turned.reshape(T, -1, rot)
        got[name] = y
    return got


def _exact_attention(s, case):
    """Head by head and sequence by sequence, in blocks of query rows."""
    T, hq, hk, D = case["T"], case["hq"], case["hk"], case["D"]
    step = case["dir"] == "step"
    if work(case)["flops"] > 6e12:
        return None
    new = lambda h: torch.zeros(T, h, D, dtype=torch.float64, device=s["q"].device)  # noqa: E731
    got = {"out": new(hq)}
    if step:
        got.update(dq=new(hq), dk=new(hk), dv=new(hk))
    at = 0
    for n in s["lens"]:
        for h in range(hq):
            kv = h // (hq // hk)
            k, v = s["k"][at:at + n, kv].double(), s["v"][at:at + n, kv].double()
            for a in range(0, n, 2048):
                e = min(n, a + 2048)
                q = s["q"][at + a:at + e, h].double()
                logits = torch.einsum("id,jd->ij", q, k[:e]) * s["scale"]
                keep = torch.arange(e, device=q.device)[None, :] <= torch.arange(a, e, device=q.device)[:, None]
                p = torch.softmax(torch.where(keep, logits, torch.full_like(logits, -math.inf)), dim=1)
                o = p @ v[:e]
                got["out"][at + a:at + e, h] = o
                if step:
                    do = s["dout"][at + a:at + e, h].double()
                    dp = do @ v[:e].T
                    ds = p * (dp - torch.einsum("ij,ij->i", p, dp)[:, None])
                    got["dq"][at + a:at + e, h] = ds @ k[:e] * s["scale"]
                    got["dk"][at:at + e, kv] += ds.T @ q * s["scale"]
                    got["dv"][at:at + e, kv] += p.T @ do
        at += n
    return got
