"""Plain 64-bit implementations of the training block's operators, with the
elementwise bounds that the kernels' roundings allow.

U is the largest relative error of one rounding to bf16 (8 significant bits,
to nearest).  EPS bounds what fp32 arithmetic adds: sums of up to a few
thousand terms and the fast exponential, relative to the sum of magnitudes.
"""
import math

import torch

U = 2.0 ** -8
EPS = 2.0 ** -16


def within(name, got, want, bound):
    """|got - want| <= bound, elementwise, with a report of the worst."""
    got, want = got.double(), want.double()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    assert bool(torch.isfinite(got).all()), f"{name}: non-finite values"
    over = (got - want).abs() - bound
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 0, f"{name}: {int((over > 0).sum())} of {over.numel()} past their bound, by {worst:.3g}"


# ------------------------------------------------------------------ norm

def norm_forward(b, r, gate, w_post, w_pre, alpha, beta, eps):
    r = r.double()
    y = alpha * r
    rb = None
    if b is not None:
        b = b.double()
        rb = torch.rsqrt((b * b).mean(1) + eps)
        g = 1.0 if gate is None else gate.double()
        y = y + beta * g * (b * rb[:, None] * w_post.double())
    if w_pre is None:
        return y, None, rb, None
    ry = torch.rsqrt((y * y).mean(1) + eps)
    return y, y * ry[:, None] * w_pre.double(), rb, ry


def norm_backward(dn, dy, b, r, gate, w_post, w_pre, alpha, beta, eps):
    """Gradients by autograd in 64 bits, as a dict."""
    leaf = lambda t: None if t is None else t.double().detach().requires_grad_()  # noqa: E731
    b, r, gate, w_post, w_pre = map(leaf, (b, r, gate, w_post, w_pre))
    y, n, _, _ = norm_forward(b, r, gate, w_post, w_pre, alpha, beta, eps)
    loss = 0.0
    if n is not None:
        loss = loss + (n * dn.double()).sum()
    if dy is not None:
        loss = loss + (y * dy.double()).sum()
    names = {"db": b, "dr": r, "dgate": gate, "dw_post": w_post, "dw_pre": w_pre}
    names = {k: t for k, t in names.items() if t is not None}
    got = torch.autograd.grad(loss, list(names.values()), allow_unused=True)
    return dict(zip(names, got))


# ------------------------------------------------------------------ rotary

def rotary_angles(rows, rot, base=10000.0, scaling="none", factor=1.0, orig_len=0.0,
                  beta_fast=32.0, beta_slow=1.0):
    i = torch.arange(rot // 2, dtype=torch.float64)
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2 * i / rot)
    if scaling == "linear":
        f = f / factor
    if scaling == "by_parts":
        turns = orig_len * f / (2 * math.pi)
        keep = ((turns - beta_slow) / (beta_fast - beta_slow)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
    return torch.arange(rows, dtype=torch.float64)[:, None] * f


def rotary(x, table, pos, rot, interleaved, inverse):
    x = x.double().clone()
    c, s = (table.double()[pos.long()][:, None, :, e] for e in (0, 1))
    if inverse:
        s = -s
    if interleaved:
        a, b = x[..., 0:rot:2].clone(), x[..., 1:rot:2].clone()
        x[..., 0:rot:2], x[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        h = rot // 2
        a, b = x[..., :h].clone(), x[..., h:rot].clone()
        x[..., :h], x[..., h:rot] = a * c - b * s, b * c + a * s
    return x


# ------------------------------------------------------------------ attention

def attention(q, k, v, lens, scale, first=0, dout=None):
    """Outputs and, with dout, gradients, each with its bound: a dict name ->
    (value, bound).  Sequences of lens tokens from token ``first`` on."""
    T, hq, D = q.shape
    hk = k.shape[1]
    q, k, v = q.double(), k.double(), v.double()
    z = lambda h: torch.zeros(T, h, D, dtype=torch.float64, device=q.device)  # noqa: E731
    out, out_b = z(hq), z(hq)
    lse = torch.full((hq, T), -math.inf, dtype=torch.float64, device=q.device)
    g = {n: (z(h), z(h)) for n, h in (("dq", hq), ("dk", hk), ("dv", hk))}
    do = None if dout is None else dout.double()
    at = first
    for n in lens:
        sl = slice(at, at + n)
        at += n
        if not n:
            continue
        keep = torch.ones(n, n, dtype=torch.bool, device=q.device).tril()
        for h in range(hq):
            kv = h // (hq // hk)
            qh, kh, vh = q[sl, h], k[sl, kv], v[sl, kv]
            s = (qh @ kh.T * scale).masked_fill(~keep, -math.inf)
            lse[h, sl] = torch.logsumexp(s, 1)
            p = torch.exp(s - lse[h, sl][:, None])
            o = p @ vh
            out[sl, h] = o
            out_b[sl, h] = (U + EPS) * (p @ vh.abs()) + U * o.abs()
            if do is None:
                continue
            d = do[sl, h]
            dp = d @ vh.T
            ds = p * (dp - (d * o).sum(1, keepdim=True))
            # D from out in two bf16 parts, dP in fp32, P as in out
            slack = p * EPS * ((d.abs() * o.abs()).sum(1, keepdim=True) + d.abs() @ vh.abs().T)
            wide = (U + EPS) * ds.abs() + (1 + U) * slack
            g["dq"][0][sl, h] += scale * ds @ kh
            g["dq"][1][sl, h] += scale * wide @ kh.abs()
            g["dk"][0][sl, kv] += scale * ds.T @ qh
            g["dk"][1][sl, kv] += scale * wide.T @ qh.abs()
            g["dv"][0][sl, kv] += p.T @ d
            g["dv"][1][sl, kv] += (U + EPS) * (p.T @ d.abs())
    res = {"out": (out, out_b), "lse": (lse, None)}
    if do is not None:
        res.update({n: (x, b * (1 + U) + U * x.abs()) for n, (x, b) in g.items()})
    return res
