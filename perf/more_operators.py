"""Cases and plain forms of what a training step runs between token ids and loss.

Four operators: ``heads`` (norm of each query and key head and the rotation to
its position in one pass; forward and backward), ``route`` (softmax or sigmoid
scores, a bias for balance, groups, top-k, weights; forward and backward),
``embed`` (lookup with scaling; its gradient by sorted tokens) and ``distill``
(the loss against a teacher's top logits; forward, backward, and a step that
gives the loss and the gradient).  ``own`` chooses between the plain forms, in
32 bits from elementary torch operations (in 64 where a choice hangs on it),
and the framework's kernels.
"""
import math

import numpy as np
import torch

own = False

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one new token of a served sequence: all latency
        {"name": "heads one token", "op": "heads", "dir": "forward", "T": 1, "seq": 4096, "hq": 16, "hk": 4, "D": 128, "rot": 128, "layout": "half"},
        # the mid layer's batch, heads side by side in one projection's output
        {"name": "heads mid", "op": "heads", "dir": "forward", "T": 8192, "seq": 4096, "hq": 16, "hk": 4, "D": 128, "rot": 128, "layout": "half"},
        # the gradient over one long sequence, half of each head turned, pairs side by side
        {"name": "heads long backward", "op": "heads", "dir": "backward", "T": 65536, "seq": 65536, "hq": 48, "hk": 8, "D": 128, "rot": 64, "layout": "pairs"},
        # the tiny layer's router: latency
        {"name": "route tiny", "op": "route", "dir": "forward", "T": 256, "groups": 1, "per": 24, "kept": 1, "top": 1, "k": 2, "score": "softmax", "bias": False, "renorm": True, "grad": "bf16"},
        # the full layer's router: eight groups of 48 experts, four of them kept, a bias that keeps the load even
        {"name": "route full", "op": "route", "dir": "forward", "T": 16384, "groups": 8, "per": 48, "kept": 4, "top": 2, "k": 8, "score": "sigmoid", "bias": True, "renorm": True, "grad": "bf16"},
        # the gradient of the long batch's logits, every expert's part of the softmax among them
        {"name": "route long backward", "op": "route", "dir": "backward", "T": 65536, "groups": 1, "per": 384, "kept": 1, "top": 1, "k": 8, "score": "softmax", "bias": False, "renorm": False, "grad": "bf16"},
        # a served batch's last tokens
        {"name": "embed few", "op": "embed", "dir": "forward", "T": 37, "d": 2048, "V": 50001, "table": "bf16", "out": "bf16"},
        # an odd batch of the mid layer, gradients summed in 32 bits and kept in bf16, a vocabulary of odd size
        {"name": "embed mid backward", "op": "embed", "dir": "backward", "T": 8191, "d": 2048, "V": 50001, "table": "bf16", "out": "bf16"},
        # the full layer's batch and width: every row of the gradient is written
        {"name": "embed full backward", "op": "embed", "dir": "backward", "T": 16384, "d": 6144, "V": 131072, "table": "f32", "out": "bf16"},
        # a few answers scored against a teacher, vocabulary of odd size in 32 bits
        {"name": "distill few", "op": "distill", "dir": "forward", "T": 5, "V": 50001, "K": 16, "z": "f32", "pad": False, "tau": 1.0},
        # a batch whose loss is kept for later, rows that start at odd places
        {"name": "distill mid backward", "op": "distill", "dir": "backward", "T": 2047, "V": 50001, "K": 50, "z": "bf16", "pad": False, "tau": 2.0},
        # a training step of a long batch: the loss and the gradient of all logits
        {"name": "distill full step", "op": "distill", "dir": "step", "T": 8192, "V": 131072, "K": 64, "z": "bf16", "pad": False, "tau": 1.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("heads", "route", "embed", "distill"))
    if op == "heads":
        D, hk = rng.choice((64, 80, 96, 128, 256)), rng.choice((1, 2, 4, 8))
        hq = hk * rng.choice((1, 2, 3, 4, 6))
        T = _log(rng, 1, min(65536, 65536 * 56 * 128 // ((hq + hk) * D)))
        return {"op": op, "dir": rng.choice(("forward", "backward")), "T": T, "seq": max(1, T // rng.randint(1, 4)), "hq": hq, "hk": hk, "D": D,
                "rot": rng.choice((D, D // 32 * 16)), "layout": rng.choice(("half", "pairs"))}
    if op == "route":
        groups = rng.choice((1, 1, 2, 4, 8, 16))
        per = _log(rng, max(2, 16 // groups), 512 // groups)
        k = rng.randint(1, min(16, groups * per))
        kept = rng.randint(-(-k // per), groups)
        return {"op": op, "dir": rng.choice(("forward", "backward")), "T": _log(rng, 1, min(65536, 65536 * 384 // (groups * per))), "groups": groups, "per": per,
                "kept": kept, "top": rng.choice((1, 2)), "k": k, "score": rng.choice(("sigmoid", "softmax")), "bias": rng.random() < 0.6,
                "renorm": rng.random() < 0.6, "grad": rng.choice(("bf16", "f32"))}
    if op == "embed":
        d = 8 * _log(rng, 8, 768)
        V = _log(rng, 2, min(200000, 131072 * 6144 // d))
        return {"op": op, "dir": rng.choice(("forward", "backward")), "T": _log(rng, 1, min(65536, 16384 * 6144 // d)), "d": d, "V": V,
                "table": rng.choice(("bf16", "f32")), "out": rng.choice(("bf16", "bf16", "f32"))}
    V, z = _log(rng, 64, 200000), rng.choice(("bf16", "bf16", "f32"))
    return {"op": op, "dir": rng.choice(("forward", "backward", "step")), "T": _log(rng, 1, min(16384, 8192 * 131072 // V // (2 if z == "f32" else 1))), "V": V,
            "K": _log(rng, 1, min(V, 128)), "z": z, "pad": rng.random() < 0.5, "tau": rng.choice((1.0, 2.0, 0.7))}


def _type(name):
    return BF if name == "bf16" else F32


def _size(name):
    return 2 if name == "bf16" else 4


def work(case):
    op, T = case["op"], case["T"]
    if op == "heads":
        n = T * (case["hq"] + case["hk"]) * case["D"]
        return {"bytes": n * (4 if case["dir"] == "forward" else 6), "flops": n * (6 if case["dir"] == "forward" else 14)}
    if op == "route":
        n, k = T * case["groups"] * case["per"], case["k"]
        if case["dir"] == "forward":
            return {"bytes": 4 * n + 8 * T * k, "flops": 6 * n}
        dense = case["score"] == "softmax" and not case["renorm"]  # only there every logit is needed
        return {"bytes": (4 * n if dense else 4 * T * k) + _size(case["grad"]) * n + 8 * T * k, "flops": (6 * n if dense else 8 * T * k)}
    if op == "embed":
        n = T * case["d"]
        if case["dir"] == "forward":  # rows that occur several times are read once at best
            return {"bytes": min(T, case["V"]) * case["d"] * _size(case["table"]) + n * _size(case["out"]) + 4 * T, "flops": n}
        return {"bytes": n * _size(case["out"]) + case["V"] * case["d"] * _size(case["table"]) + 4 * T, "flops": n}
    # rows without weight or entries, about one in ten, are not read; their gradient is written
    n, e, live = T * case["V"], _size(case["z"]), 0.9 * (0.8 + 0.2 * case["K"] / (case["K"] + 1))
    return {"bytes": n * e * (live if case["dir"] == "forward" else 1 + live) + T * case["K"] * 8, "flops": n * live * (4 if case["dir"] == "forward" else 8)}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    draw_ = lambda *s, std=1.0, dt=BF: (torch.randn(s, generator=g, device=dev, dtype=F32) * std).to(dt)  # noqa: E731
    rand = lambda *s: torch.rand(s, generator=g, device=dev, dtype=F64)  # noqa: E731
    out = lambda *s, dt=BF: torch.empty(s, device=dev, dtype=dt)  # noqa: E731
    s = dict(case=case, op=case["op"], status=torch.zeros(1, device=dev, dtype=torch.int32))
    if own:
        from moe_routing_capacity_gb300 import abi
    T = case["T"]
    if case["op"] == "heads":
        hq, hk, D = case["hq"], case["hk"], case["D"]
        s["pos"] = ((torch.arange(T, device=dev) + (int(rand(1)[0] * case["seq"]) if T == 1 else 0)) % case["seq"]).to(torch.int32)
        f = 10000.0 ** (-torch.arange(0, case["rot"], 2, device=dev, dtype=F64) / case["rot"])
        a = torch.arange(case["seq"], device=dev, dtype=F64)[:, None] * f
        s["table"] = torch.stack((a.cos(), a.sin()), -1).float()  # [positions, rot / 2, 2], made once
        qkv = draw_(T, hq + 2 * hk, D, std=1.5)  # heads of one projection's output
        s.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hk], w_q=1 + draw_(D, std=0.1), w_k=1 + draw_(D, std=0.1), eps=1e-6, q_out=out(T, hq, D), k_out=out(T, hk, D))
        if case["dir"] == "backward":
            s.update(dq=draw_(T, hq, D, std=1e-2), dk=draw_(T, hk, D, std=1e-2), dw_q=out(D, dt=F32), dw_k=out(D, dt=F32))
            if own:
                s["ws"] = out(abi.head_norm_rotary_workspace(T, hq, hk, D), dt=torch.uint8)
    elif case["op"] == "route":
        E, k = case["groups"] * case["per"], case["k"]
        s.update(logits=draw_(T, E, dt=F32) + draw_(E, std=0.3, dt=F32), idx=out(T, k, dt=torch.int32), w=out(T, k, dt=F32), scale=2.5)
        s["bias"] = draw_(E, std=0.05 if case["score"] == "sigmoid" else 0.3 / E, dt=F32) if case["bias"] else None
        if case["dir"] == "backward":  # the choice is the forward's
            s["idx"] = _choose(s, case).to(torch.int32)
            s.update(dw=draw_(T, k, std=1e-2, dt=F32), dlogits=out(T, E, dt=_type(case["grad"])))
        if own:
            s["cfg"] = abi.Routing(E, k, score=case["score"], n_groups=case["groups"], groups_kept=case["kept"], group_top=case["top"], renorm=case["renorm"],
                                   scale=s["scale"])
    elif case["op"] == "embed":
        d, V = case["d"], case["V"]
        # words as often as their rank's inverse, the ranks spread over the vocabulary, one place in fifty padding
        rank = ((V + 1) ** rand(T) - 1).long().clamp(0, V - 1)
        s["ids"] = torch.where(rand(T) < 0.02, -1, torch.randperm(V, generator=g, device=dev)[rank]).to(torch.int32)
        s["scale"] = math.sqrt(d)
        if case["dir"] == "forward":
            s.update(table=draw_(V, d, std=0.02, dt=_type(case["table"])), out=out(T, d, dt=_type(case["out"])))
        else:
            s.update(dout=draw_(T, d, std=1e-2, dt=_type(case["out"])), dtable=out(V, d, dt=_type(case["table"])))
            if own:
                s["plan"] = abi.EmbeddingPlan(s["ids"], V, d)
    else:
        V, K, zt = case["V"], case["K"], _type(case["z"])
        wide = -(-V // 128) * 128 if case["pad"] else V  # the head product's rows, padded to whole tiles or not
        z = out(T, wide, dt=zt)
        for a in range(0, T, 1024):
            z[a:a + 1024] = draw_(min(1024, T - a), wide, std=2.0, dt=zt)
        z = z[:, :V]
        # distinct words, and as many entries as the teacher gave: all, or fewer, or none
        step = (rand(T, 1) * (V // K)).long().clamp(0, V // K - 1) + 1
        ids = ((rand(T, 1) * V).long().clamp(0, V - 1) + step * torch.arange(K, device=dev)) % V
        given = torch.where(rand(T) < 0.8, K, (rand(T) * (K + 1)).long())
        s["ids"] = torch.where(torch.arange(K, device=dev) < given[:, None], ids, -1).to(torch.int32)
        s["teacher"] = draw_(T, K, std=2.0, dt=F32).sort(dim=1, descending=True)[0]
        z.scatter_add_(1, ids, (s["teacher"] + 6.0).to(zt))  # a student that has learnt something
        s.update(z=z, weight=torch.where(rand(T) < 0.9, 1.0, 0.0).float(), scale=1.0 / T, loss=out(T, dt=F32), lse=out(T, dt=F32), total=out(1, dt=F32))
        if case["dir"] != "forward":
            s["dz"] = out(T, wide, dt=zt)[:, :V]
        if case["dir"] == "backward":  # the forward's, in hand
            for a in range(0, T, 256):
                s["lse"][a:a + 256] = torch.logsumexp(z[a:a + 256].double() / case["tau"], 1).float()
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    if own:
        return _OWN[s["op"]](s, case)
    return _PLAIN[s["op"]](s, case)


def _own_heads(s, case):
    from moe_routing_capacity_gb300 import abi
    pairs = case["layout"] == "pairs"
    if case["dir"] == "forward":
        abi.head_norm_rotary(s["q"], s["k"], s["w_q"], s["w_k"], s["table"], s["pos"], s["q_out"], s["k_out"], s["status"], eps=s["eps"], interleaved=pairs)
        return {"q": s["q_out"], "k": s["k_out"]}
    abi.head_norm_rotary_backward(s["dq"], s["dk"], s["q"], s["k"], s["w_q"], s["w_k"], s["table"], s["pos"], s["q_out"], s["k_out"], s["dw_q"], s["dw_k"], s["ws"],
                                  s["status"], eps=s["eps"], interleaved=pairs)
    return {"q": s["q_out"], "k": s["k_out"], "dw_q": s["dw_q"], "dw_k": s["dw_k"]}


def _own_route(s, case):
    from moe_routing_capacity_gb300 import abi
    if case["dir"] == "forward":
        abi.router_select(s["cfg"], s["logits"], s["bias"], s["idx"], s["w"])
        return {"idx": s["idx"], "w": s["w"]}
    abi.router_select_backward(s["cfg"], s["logits"], s["idx"], s["dw"], s["dlogits"])
    return {"dlogits": s["dlogits"]}


def _own_embed(s, case):
    from moe_routing_capacity_gb300 import abi
    if case["dir"] == "forward":
        abi.embedding(s["table"], s["ids"], s["out"], s["status"], scale=s["scale"])
        return {"out": s["out"]}
    s["plan"].refill(s["ids"])
    abi.embedding_backward(s["plan"], s["dout"], s["dtable"], scale=s["scale"])
    return {"dtable": s["dtable"]}


def _own_distill(s, case):
    from moe_routing_capacity_gb300 import abi
    if case["dir"] == "backward":
        abi.distill_loss_backward(s["z"], s["ids"], s["teacher"], s["weight"], s["lse"], s["dz"], s["status"], temperature=case["tau"], scale=s["scale"])
        return {"dz": s["dz"]}
    abi.distill_loss(s["z"], s["ids"], s["teacher"], s["weight"], s["loss"], s["lse"], s["status"], total=s["total"],
                     dlogits=s["dz"] if case["dir"] == "step" else None, temperature=case["tau"], scale=s["scale"])
    got = {"loss": s["loss"], "lse": s["lse"], "total": s["total"]}
    return {**got, "dz": s["dz"]} if case["dir"] == "step" else got


def _turn(x, cs, rot, pairs, back):
    c, t = cs[..., 0][:, None], cs[..., 1][:, None]
    if back:
        t = -t
    if pairs:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * c - b * t, b * c + a * t), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * c - b * t, b * c + a * t), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _plain_heads(s, case):
    cs, rot, pairs = s["table"][s["pos"].long()], case["rot"], case["layout"] == "pairs"

    def forward(x, w):
        f = x.float()
        n = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + s["eps"]) * w.float()
        return _turn(n, cs, rot, pairs, False).to(BF)

    def backward(dy, x, w):
        f, dn = x.float(), _turn(dy.float(), cs, rot, pairs, True)
        r = torch.rsqrt((f * f).mean(-1, keepdim=True) + s["eps"])
        u, h = dn * w.float(), f * r
        return (r * (u - h * (u * h).mean(-1, keepdim=True))).to(BF), (dn * h).sum((0, 1))

    if case["dir"] == "forward":
        return {"q": forward(s["q"], s["w_q"]), "k": forward(s["k"], s["w_k"])}
    dq, dw_q = backward(s["dq"], s["q"], s["w_q"])
    dk, dw_k = backward(s["dk"], s["k"], s["w_k"])
    return {"q": dq, "k": dk, "dw_q": dw_q, "dw_k": dw_k}


def _scores(logits, case):
    if case["score"] == "sigmoid":
        return 1 / (1 + torch.exp(-logits))
    e = torch.exp(logits - logits.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _choose(s, case):
    """The k experts, in 64 bits: next to a border 32 bits choose by chance."""
    v = _scores(s["logits"].double(), case)
    if s["bias"] is not None:
        v = v + s["bias"].double()
    if case["kept"] < case["groups"]:
        of = v.unflatten(1, (case["groups"], case["per"]))
        best = of.sort(dim=2, descending=True, stable=True)[0][..., :case["top"]].sum(2).sort(dim=1, descending=True, stable=True)[1][:, :case["kept"]]
        keep = torch.zeros(v.shape[0], case["groups"], dtype=torch.bool, device=v.device).scatter_(1, best, True)
        v = torch.where(keep[..., None], of, -math.inf).flatten(1)
    return v.sort(dim=1, descending=True, stable=True)[1][:, :case["k"]]


def _plain_route(s, case):
    if case["dir"] == "forward":
        idx = _choose(s, case)
        w = _scores(s["logits"], case).gather(1, idx)
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True)
        return {"idx": idx.to(torch.int32), "w": w * s["scale"]}
    idx, g = s["idx"].long(), s["dw"] * s["scale"]
    p = _scores(s["logits"], case)
    ps = p.gather(1, idx)
    if case["renorm"]:
        total = ps.sum(1, keepdim=True)
        g = (g - (g * ps).sum(1, keepdim=True) / total) / total
    if case["score"] == "sigmoid":
        got = torch.zeros_like(p).scatter_(1, idx, g * ps * (1 - ps))
    else:
        got = torch.zeros_like(p).scatter_(1, idx, g)
        got = p * (got - (g * ps).sum(1, keepdim=True))
        if case["renorm"]:  # what the others get is exactly zero
            got = torch.zeros_like(p).scatter_(1, idx, got.gather(1, idx))
    return {"dlogits": got.to(s["dlogits"].dtype)}


def _plain_embed(s, case):
    ids = s["ids"].long()
    if case["dir"] == "forward":
        rows = s["table"][ids.clamp(min=0)].float() * s["scale"]
        return {"out": torch.where((ids >= 0)[:, None], rows, 0.0).to(s["out"].dtype)}
    got = torch.zeros(case["V"] + 1, case["d"], device=ids.device)
    got.index_add_(0, torch.where(ids < 0, case["V"], ids), s["dout"].float())
    return {"dtable": (got[:case["V"]] * s["scale"]).to(s["dtable"].dtype)}


def _plain_distill(s, case):
    tau, ids = case["tau"], s["ids"].long()
    there, at = ids >= 0, ids.clamp(min=0)
    live = (s["weight"] != 0) & there.any(1)
    y = torch.where(there, s["teacher"].float() / tau, -math.inf)
    y = torch.where(live[:, None], y, 0.0)
    e = torch.exp(y - y.amax(1, keepdim=True))
    p = e / e.sum(1, keepdim=True)
    z = s["z"].float() / tau
    if case["dir"] == "backward":
        lse = s["lse"]
    else:
        top = z.amax(1)
        lse = top + torch.log(torch.exp(z - top[:, None]).sum(1))
    got = {}
    if case["dir"] != "backward":
        logq = z.gather(1, at) - lse[:, None]
        loss = torch.where(p > 0, p * (torch.log(torch.where(p > 0, p, 1.0)) - logq), 0.0).sum(1)
        loss = torch.where(live, loss * (tau * tau) * s["weight"] * s["scale"], 0.0)
        got = {"loss": loss, "lse": torch.where(live, lse, 0.0), "total": loss.sum().reshape(1)}
    if case["dir"] != "forward":
        f = torch.where(live, s["weight"] * (s["scale"] * tau), 0.0)[:, None]
        dz = z.sub_(lse[:, None]).exp_().mul_(f)
        dz.scatter_add_(1, at, torch.where(there, -p * f, 0.0))
        got["dz"] = dz.to(s["z"].dtype)
    return got


_OWN = {"heads": _own_heads, "route": _own_route, "embed": _own_embed, "distill": _own_distill}
_PLAIN = {"heads": _plain_heads, "route": _plain_route, "embed": _plain_embed, "distill": _plain_distill}


# ------------------------------------------------------------------ in 64 bits, from the definitions

def exact(case, seed):
    s = prepare(case, seed)
    return {"heads": _exact_heads, "route": _exact_route, "embed": _exact_embed, "distill": _exact_distill}[case["op"]](s, case)


def _exact_heads(s, case):
    """Blocks of tokens; the rotation as a product of complex numbers, the norm's gradient from its Jacobian."""
    T, D, rot, back = case["T"], case["D"], case["rot"], case["dir"] == "backward"
    table = torch.view_as_complex(s["table"].double())
    got = {}

    def spin(x, z):
        pair = x[..., :rot].unflatten(-1, (rot // 2, 2)) if case["layout"] == "pairs" else x[..., :rot].unflatten(-1, (2, rot // 2)).transpose(-1, -2)
        y = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z[:, None])
        y = y.flatten(-2) if case["layout"] == "pairs" else y.transpose(-1, -2).flatten(-2)
        return torch.cat((y, x[..., rot:]), -1)

    for name in ("q", "k"):
        x, w = s[name], s["w_" + name].double()
        y = torch.empty(x.shape, dtype=F64, device=x.device)
        dw = torch.zeros(D, dtype=F64, device=x.device)
        for a in range(0, T, 2048):
            at = slice(a, min(T, a + 2048))
            f, z = x[at].double(), table[s["pos"][at].long()]
            ms = torch.einsum("thd,thd->th", f, f)[..., None] / D + s["eps"]
            if not back:
                y[at] = spin(f * w / ms.sqrt(), z)
                continue
            dn = spin(s["d" + name][at].double(), z.conj())
            along = torch.einsum("thd,thd->th", dn * w, f)[..., None]
            y[at] = dn * w / ms.sqrt() - f * along / (D * ms * ms.sqrt())
            dw += torch.einsum("thd,thd->d", dn, f / ms.sqrt())
        got[name] = y
        if back:
            got["dw_" + name] = dw
    return got


def _exact_route(s, case):
    """The choice by selecting the best group and the best expert one after the other."""
    logits = s["logits"].double()
    T, E = logits.shape
    p = torch.sigmoid(logits) if case["score"] == "sigmoid" else torch.softmax(logits, 1)
    row = torch.arange(T, device=logits.device)
    first = lambda v: (v == v.amax(1, keepdim=True)).to(torch.uint8).argmax(1)  # noqa: E731  the lowest index of the largest
    if case["dir"] == "forward":
        v = p if s["bias"] is None else p + s["bias"].double()
        if case["kept"] < case["groups"]:
            of = v.reshape(T, case["groups"], case["per"])
            value, rest = of.amax(2), of.clone()
            for _ in range(case["top"] - 1):
                at = first(rest.flatten(0, 1)).view(T, case["groups"], 1)
                rest.scatter_(2, at, -math.inf)
                value = value + rest.amax(2)
            open_ = torch.zeros(T, case["groups"], dtype=torch.bool, device=v.device)
            for _ in range(case["kept"]):
                at = first(value)
                open_[row, at] = True
                value[row, at] = -math.inf
            v = torch.where(open_.repeat_interleave(case["per"], 1), v, -math.inf)
        else:
            v = v.clone()
        idx = torch.empty(T, case["k"], dtype=torch.int64, device=v.device)
        for j in range(case["k"]):
            idx[:, j] = first(v)
            v[row, idx[:, j]] = -math.inf
        w = torch.take_along_dim(p, idx, 1)
        return {"idx": idx.to(torch.int32), "w": w * (s["scale"] / (w.sum(1, keepdim=True) if case["renorm"] else 1.0))}
    idx, g = s["idx"].long(), s["dw"].double() * s["scale"]
    w = torch.take_along_dim(p, idx, 1)
    if case["renorm"]:
        g = g / w.sum(1, keepdim=True) - torch.einsum("tk,tk->t", g, w)[:, None] / w.sum(1, keepdim=True) ** 2
    dp = torch.zeros_like(p)
    dp[row[:, None], idx] = g
    if case["score"] == "sigmoid":
        return {"dlogits": dp * p * (1 - p)}
    got = p * dp - p * torch.einsum("te,te->t", p, dp)[:, None]
    if case["renorm"]:
        held = torch.zeros_like(p)
        held[row[:, None], idx] = got[row[:, None], idx]
        return {"dlogits": held}
    return {"dlogits": got}


def _exact_embed(s, case):
    ids, d = s["ids"].long(), case["d"]
    if case["dir"] == "forward":
        got = s["table"][ids.clamp(min=0)].double() * s["scale"]
        got[ids < 0] = 0
        return {"out": got}
    # word by word, over its rows side by side
    order = torch.argsort(ids, stable=True)
    word, count = torch.unique_consecutive(ids[order], return_counts=True)
    got = torch.zeros(case["V"], d, dtype=F64, device=ids.device)
    at = 0
    for w, n in zip(word.tolist(), count.tolist()):
        if w >= 0:
            got[w] = s["dout"][order[at:at + n]].double().sum(0) * s["scale"]
        at += n
    return {"dtable": got}


def _exact_distill(s, case):
    T, V, tau, ids = case["T"], case["V"], case["tau"], s["ids"].long()
    dev = ids.device
    step, back = case["dir"] == "step", case["dir"] == "backward"
    loss, lses = torch.zeros(T, dtype=F64, device=dev), torch.zeros(T, dtype=F64, device=dev)
    dz = None if case["dir"] == "forward" else torch.zeros(T, V, dtype=F64, device=dev)
    weight = s["weight"].double() * s["scale"]
    for a in range(0, T, 512):
        at = slice(a, min(T, a + 512))
        z, i = s["z"][at].double() / tau, ids[at]
        lse = s["lse"][at].double() if back else torch.logsumexp(z, 1)
        there = (i >= 0) & (weight[at] != 0)[:, None]
        empty = ~there.any(1)
        lses[at] = lse.masked_fill(empty, 0)
        logp = torch.log_softmax(torch.where(there, s["teacher"][at].double() / tau, -math.inf), 1)
        logp = torch.where(there, logp, -math.inf)
        p = logp.exp()
        gap = torch.where(there, logp - (torch.take_along_dim(z, i.clamp(min=0), 1) - lse[:, None]), 0.0)
        loss[at] = (p * gap).sum(1) * weight[at] * tau ** 2
        if dz is not None:
            q = (z - lse[:, None]).exp()
            q[empty] = 0
            row = torch.arange(q.shape[0], device=dev)[:, None].expand_as(i)[there]
            q.index_put_((row, i[there]), -p[there], accumulate=True)
            dz[at] = q * (weight[at] * tau)[:, None]
    if back:
        return {"dz": dz}
    got = {"loss": loss, "lse": lses, "total": np.array([math.fsum(loss.tolist())])}
    return {**got, "dz": dz} if step else got
