"""Plain 64-bit implementations of head norms with rotation, the choice of
experts, embedding and the distillation loss, with the elementwise bounds that
the kernels' roundings allow.

U is the largest relative error of one rounding to bf16, STEP of one to fp32.
"""
import math

import torch

from block_reference import U, rotary, within  # noqa: F401

STEP = 2.0 ** -24


def round_of(dtype):
    return U if dtype == torch.bfloat16 else STEP


# ------------------------------------------------------------------ head norms

def head_norm(x, w, table, pos, eps, interleaved):
    """Outputs and their bound.  fp32: up to 512 squares in 16 + 5 steps, the
    inverse root within 4 steps, three products and a sum a channel: under 32
    steps of the pair that is turned."""
    f = x.double()
    n = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + eps) * w.double()
    rot = 0 if table is None else 2 * table.shape[1]
    y = n if not rot else rotary(n, table, pos, rot, interleaved, False)
    mag = n.abs()
    if rot:
        mag = rotary_abs(n, table, pos, rot, interleaved)
    return y, U * y.abs() + 32 * STEP * (1 + U) * mag


def rotary_abs(x, table, pos, rot, interleaved):
    """|a c| + |b s| of each rotated channel."""
    x = x.double().abs().clone()
    c, s = (table.double()[pos.long()][:, None, :, e].abs() for e in (0, 1))
    at = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = x[..., at[0]].clone(), x[..., at[1]].clone()
    x[..., at[0]], x[..., at[1]] = a * c + b * s, b * c + a * s
    return x


def head_norm_backward(dy, x, w, table, pos, eps, interleaved, skip=None):
    """(dx, bound, dw, bound); skip [T]: tokens that add nothing to dw."""
    f, wd, D = x.double(), w.double(), x.shape[-1]
    rot = 0 if table is None else 2 * table.shape[1]
    dn = dy.double() if not rot else rotary(dy, table, pos, rot, interleaved, True)
    mag = dn.abs() if not rot else rotary_abs(dy, table, pos, rot, interleaved)
    r = torch.rsqrt((f * f).mean(-1, keepdim=True) + eps)
    u = dn * wd
    dx = r * (u - f * r * r * (u * f).mean(-1, keepdim=True))
    big = r * (mag * wd.abs() + f.abs() * r * r * (mag * wd.abs() * f.abs()).mean(-1, keepdim=True))
    dx_b = U * dx.abs() + 64 * STEP * (1 + U) * big
    keep = 1.0 if skip is None else (~skip).double()[:, None, None]
    terms = (dn * f * r * keep), (mag * f.abs() * r * keep)
    n = x.shape[0] * x.shape[1]   # no sum is longer
    return dx, dx_b, terms[0].sum((0, 1)), (32 + n) * STEP * terms[1].sum((0, 1))


# ------------------------------------------------------------------ choice of experts

def scores(logits, softmax):
    l = logits.double()
    return torch.softmax(l, 1) if softmax else torch.sigmoid(l)


def select(logits, bias, rule):
    """(idx, w) in 64 bits.  Without a bias the experts go by their logits, whose
    order is the scores'."""
    T, E = logits.shape
    s = scores(logits, rule.score == 0)
    v = s if bias is None else s + bias.double()
    order = logits.double() if bias is None else v
    per = E // rule.n_groups
    if rule.groups_kept < rule.n_groups:
        of = (v if rule.group_top == 2 or bias is not None else order).view(T, rule.n_groups, per)
        value = of.sort(dim=2, descending=True)[0][..., :rule.group_top].sum(2)
        best = value.sort(dim=1, descending=True, stable=True)[1][:, :rule.groups_kept]
        keep = torch.zeros(T, rule.n_groups, dtype=torch.bool, device=logits.device)
        keep.scatter_(1, best, True)
        order = order.masked_fill(~keep.repeat_interleave(per, 1), -math.inf)
    idx = order.sort(dim=1, descending=True, stable=True)[1][:, :rule.top_k]
    return idx, weights(s, idx, rule)


def told_apart(logits, bias, rule):
    """Rows [T] whose kept and dropped groups 64 bits tell apart: two groups can have
    the same real value in other sums (s1 + b1) + (s2 + b2) = (s1 + b2) + (s2 + b1),
    whose roundings, four of 2^-53 at most, then decide."""
    T, E = logits.shape
    if rule.groups_kept == rule.n_groups or rule.group_top == 1:
        return torch.ones(T, dtype=torch.bool, device=logits.device)
    v = scores(logits, rule.score == 0) + (0 if bias is None else bias.double())
    value = v.view(T, rule.n_groups, -1).sort(dim=2, descending=True)[0][..., :2].sum(2)
    value = value.sort(dim=1, descending=True)[0]
    gap = value[:, rule.groups_kept - 1] - value[:, rule.groups_kept]
    return (gap == 0) & (bias is None or not bool(bias.any())) | (gap > 2.0 ** -50)


def weights(s, idx, rule):
    w = s.gather(1, idx)
    if rule.renorm:
        w = w / w.sum(1, keepdim=True)
    return w * rule.scale


def select_backward(logits, idx, dw, rule):
    """(dlogits, what the roundings are relative to), by autograd in 64 bits."""
    leaf = logits.double().clone().requires_grad_()
    s = scores(leaf, rule.score == 0)
    (g,) = torch.autograd.grad((weights(s, idx, rule) * dw.double()).sum(), leaf)
    s = s.detach()
    w = s.gather(1, idx)
    gd = dw.double().abs() * abs(rule.scale)
    if rule.renorm:
        n = w / w.sum(1, keepdim=True)
        part = n * (gd + (gd * n).sum(1, keepdim=True))
        # the other experts' score cancels; autograd leaves the rounding of 64 bits there
        g = torch.zeros_like(g).scatter_(1, idx, g.gather(1, idx))
        return g, torch.zeros_like(s).scatter_(1, idx, part)
    if rule.score == 0:
        got = torch.zeros_like(s).scatter_(1, idx, gd)
        return g, s * (got + (gd * w).sum(1, keepdim=True))
    return g, torch.zeros_like(s).scatter_(1, idx, gd * w)


# ------------------------------------------------------------------ embedding

def embedding_backward(ids, dout, V, scale):
    """(dtable, sum of the terms' magnitudes, the longest sum)."""
    got = torch.zeros(V, dout.shape[1], dtype=torch.float64, device=dout.device)
    mag, ok = got.clone(), (ids >= 0) & (ids < V)
    at = ids.long()[ok]
    got.index_add_(0, at, dout.double()[ok])
    mag.index_add_(0, at, dout.double()[ok].abs())
    most = int(torch.bincount(at, minlength=1).max()) if at.numel() else 0
    return got * scale, mag * abs(scale), most


# ------------------------------------------------------------------ distillation

def distill(z, ids, teacher, weight, tau, scale):
    """{loss, lse, dz} -> (value, bound without the output's own rounding).

    fp32 in base 2: an exponent x = z log2(e) / tau is off by 3 steps of |x|, a
    fast exponential by 4 steps and the sum by a step an element and a thread;
    so lse, and with it each log q, by err below, and a probability by as much
    relative to itself."""
    T, V = z.shape
    f, there = z.double() / tau, (ids >= 0) & (ids < V)
    y = torch.where(there, teacher.double() / tau, -math.inf)
    w = torch.ones(T, dtype=torch.float64, device=z.device) if weight is None else weight.double()
    live = (w != 0) & (y > -math.inf).any(1)
    f = torch.where(live[:, None], f, torch.zeros_like(f))
    y = torch.where(live[:, None], y, torch.zeros_like(y))
    w = torch.where(live, w, 0.0)
    lse = torch.logsumexp(f, 1)
    logp = torch.log_softmax(y, 1)
    p = torch.where(live[:, None], logp.exp(), 0.0)
    at = ids.long().clamp(0, V - 1)
    logq = f.gather(1, at) - lse[:, None]
    gap = torch.where(p > 0, logp - logq, 0.0)
    big = f.abs().masked_fill(f.abs() == math.inf, 0).amax(1)
    ybig = y.abs().masked_fill(y.abs() == math.inf, 0).amax(1)
    err = STEP * (8 * big + 4 * lse.abs() + V / 32 + 32)
    perr = STEP * (8 * ybig + ids.shape[1] + 32)
    loss = w * scale * tau * tau * (p * gap).sum(1)
    terms = (p * torch.where(p > 0, logp.abs() + logq.abs(), 0.0)).sum(1)
    loss_b = w.abs() * scale * tau * tau * (2 * err + 2 * perr + (perr + 32 * STEP) * terms)
    q = (f - lse[:, None]).exp() * live[:, None]
    fac = (w * scale * tau)[:, None]
    psum = torch.zeros_like(q).scatter_add_(1, at, torch.where(there & live[:, None], p, 0.0))
    dz = fac * (q - psum)
    dz_b = fac.abs() * (q * (2 * err + 8 * STEP)[:, None] + psum * (2 * perr + 8 * STEP)[:, None])
    return {"loss": (loss, loss_b), "lse": (torch.where(live, lse, 0.0), err), "dz": (dz, dz_b)}
