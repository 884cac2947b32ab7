"""Plain 64-bit implementations of the gated linear recurrence, the norms between blocks
and the gated feed-forward projections (formulas, token by token), with what rounding
errors scale with: every ``*_size`` is the same expression over the absolute values of
its terms.  Gradients come from automatic differentiation of the 64-bit formulas.
Sequences are given by ``cu``, a list of packed offsets.
"""
from __future__ import annotations

import torch


def d(t, grad=False):
    return None if t is None else t.detach().double().cpu().requires_grad_(grad)


def silu(x):
    return x / (1 + torch.exp(-x))


def silu_slope(x):
    s = 1 / (1 + torch.exp(-x))
    return s * (1 + x * (1 - s))


# ---------------------------------------------------------------- recurrence
def decays(f, decay, unit):
    """log a, a, m, sigmoid(f), -dm / d(log a)."""
    sf = 1 / (1 + torch.exp(-f))
    la = -torch.log1p(torch.exp(-f)) if decay is None else decay.clamp(max=0) * sf
    a = torch.exp(la)
    room = -torch.expm1(la)
    m = torch.sqrt(room * (2 - room)) if unit else room
    k = torch.where(m > 0, a * a / m.clamp(min=1e-300), 0.0) if unit else a
    return la, a, m, sf, k


def walk(a, b, init, cu):
    """h_t = a_t h_{t-1} + b_t per sequence: the states and the last ones."""
    hs, last = [], []
    for s in range(len(cu) - 1):
        h = init[s]
        for t in range(cu[s], cu[s + 1]):
            h = a[t] * h + b[t]
            hs.append(h)
        last.append(h)
    return (torch.stack(hs) if hs else a[:0]), torch.stack(last)


def recur(x, f, decay, i, z, unit, init, cu):
    """y, final (differentiable)."""
    _, a, m, _, _ = decays(f, decay, unit)
    b = m * x if i is None else m * x / (1 + torch.exp(-i))
    h, last = walk(a, b, init, cu)
    return (h if z is None else h * silu(z)), last


def recur_all(x, f, decay, i, z, unit, init, cu, dy=None, d_final=None):
    """dict of (value, size) of y, final and, with dy, of the gradients."""
    D, B = x.shape[1], len(cu) - 1
    zero = torch.zeros(B, D).double()
    grad = dy is not None
    x, f, decay, i, z, init = (d(t, grad) for t in (x, f, decay, i, z, init))
    dy, d_final = d(dy), d(d_final)
    y, last = recur(x, f, decay, i, z, unit, zero if init is None else init, cu)
    with torch.no_grad():
        la, a, m, sf, k = decays(f, decay, unit)
        si = torch.ones_like(x) if i is None else 1 / (1 + torch.exp(-i))
        hb, lastb = walk(a, m * si * x.abs(), zero if init is None else init.abs(), cu)
        gate = torch.ones_like(x) if z is None else silu(z).abs()
        out = dict(y=(y.detach(), hb * gate), final=(last.detach(), lastb))
        a_max = float(a.max()) if a.numel() else 0.0
        longest = max([q - p for p, q in zip(cu, cu[1:])] + [1])
        out["memory"] = min(longest, 1 / max(1e-9, 1 - a_max))
    if not grad:
        return out
    loss = (y * dy).sum() + (0 if d_final is None else (last * d_final).sum())
    loss.backward()
    with torch.no_grad():
        # e from the end, with absolute values
        e = torch.zeros_like(x)
        before = torch.zeros_like(x)
        d0 = zero.clone()
        for s in range(B):
            cur = zero[s] if d_final is None else d_final[s].abs()
            for t in reversed(range(cu[s], cu[s + 1])):
                e[t] = dy[t].abs() * gate[t] + cur
                cur = a[t] * e[t]
                before[t] = hb[t - 1] if t > cu[s] else (0 if init is None else init[s].abs())
            d0[s] = cur
        sx = si * x.abs()
        c = a * before + k * sx
        w = (1 - sf) * (la.abs() if decay is not None else 1.0)
        g = lambda t: None if t is None else t.grad  # noqa: E731
        out["dx"] = (g(x), e * m * si)
        out["df"] = (g(f), e * c * w)
        out["di"] = None if i is None else (g(i), e * m * sx * (1 - si))
        out["dz"] = None if z is None else (g(z), dy.abs() * hb * (1 + z.abs()) / (1 + torch.exp(-z)))
        out["d_decay"] = None if decay is None else (g(decay), (e * c * sf).sum(0))
        out["d_init"] = (g(init) if init is not None else None, d0)
    return out


# ---------------------------------------------------------------- norms
def norm(x, layer, eps):
    if layer:
        x = x - x.mean(-1, keepdim=True)
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)


def block_norm(res, y, z, pw, pb, scale, w, b, layer, eps):
    s = res
    if y is not None:
        p = y if pw is None else norm(y, layer, eps) * pw + (0 if pb is None else pb)
        p = p if z is None else p * silu(z)
        s = res + (p if scale is None else p * scale)
    u = None if w is None else norm(s, layer, eps) * w + (0 if b is None else b)
    return s, u


def _norm_size(x, xb, layer, eps):
    """r, |norm(x)|, and the size of its terms where x's is xb (an error of xb's size in
    every element moves the mean by its mean and r by r^2 mean(|x| xb))."""
    c = x - x.mean(-1, keepdim=True) if layer else x
    cb = xb + xb.mean(-1, keepdim=True) if layer else xb
    r = 1 / torch.sqrt((c * c).mean(-1, keepdim=True) + eps)
    n = (c * r).abs()
    return r, n, cb * r + n * (n * cb * r).mean(-1, keepdim=True) + n


def _back_size(dn, n, r, layer):
    out = dn + n * (dn * n).mean(-1, keepdim=True)
    return r * (out + (dn.mean(-1, keepdim=True) if layer else 0))


def block_norm_all(res, y, z, pw, pb, scale, w, b, layer, eps, du=None, ds=None):
    grad = du is not None or ds is not None
    res, y, z, pw, pb, scale, w, b = (d(t, grad) for t in (res, y, z, pw, pb, scale, w, b))
    du, ds = d(du), d(ds)
    s, u = block_norm(res, y, z, pw, pb, scale, w, b, layer, eps)
    one = torch.ones(res.shape[-1]).double()
    with torch.no_grad():
        sb = res.abs()
        if y is not None:
            pb_ = y.abs()
            if pw is not None:
                ry, ny, nyb = _norm_size(y, y.abs(), layer, eps)
                pb_ = nyb * pw.abs() + (0 if pb is None else pb.abs())
            gate = torch.ones_like(y) if z is None else silu(z).abs()
            slope = None if z is None else (1 + z.abs()) / (1 + torch.exp(-z))
            k = one if scale is None else scale.abs()
            sb = sb + k * pb_ * gate
        out = dict(s=(s.detach(), sb))
        if w is not None:
            rs, ns, nsb = _norm_size(s, sb, layer, eps)
            out["u"] = (u.detach(), nsb * w.abs() + (0 if b is None else b.abs()))
    if not grad:
        return out
    loss = 0
    if du is not None:
        loss = loss + (u * du).sum()
    if ds is not None:
        loss = loss + (s * ds).sum()
    loss.backward()
    g = lambda t: None if t is None else t.grad  # noqa: E731
    with torch.no_grad():
        db = torch.zeros_like(res) if ds is None else ds.abs()
        if du is not None:
            db = db + _back_size(du.abs() * w.abs(), nsb, rs, layer)
            out["dw"] = (g(w), (du.abs() * nsb).sum(0))
            out["db"] = None if b is None else (g(b), du.abs().sum(0))
        out["d_res"] = (g(res), db)
        if y is not None:
            out["d_scale"] = None if scale is None else (g(scale), (db * pb_ * gate).sum(0))
            db = db * k
            out["dz"] = None if z is None else (g(z), db * pb_ * slope)
            db = db * gate
            if pw is not None:
                out["d_post_weight"] = (g(pw), (db * nyb).sum(0))
                out["d_post_bias"] = None if pb is None else (g(pb), db.sum(0))
                db = _back_size(db * pw.abs(), nyb, ry, layer)
            out["dy"] = (g(y), db)
    return out


# ---------------------------------------------------------------- feed-forward
def glu_all(x, wg, wu, dh=None):
    """dict of (value, tolerance) of h, dx, dwg, dwu.

    g and u are sums of D products in fp32: each of the D / 16 accumulating steps
    rounds (or cuts off) by at most 2^-23 of what has been summed, and so do a few additions
    inside a step: (D / 16 + 4) 2^-22 of the absolute sum covers them.  Sigmoid and products: 2^-20.
    dg and du are rounded to bf16: 2^-8."""
    x, wg, wu, dh = d(x), d(wg), d(wu), d(dh)
    step = lambda n: (n / 16 + 4) * 2.0 ** -22  # noqa: E731
    g, u = x @ wg.t(), x @ wu.t()
    gb, ub = (x.abs() @ w.abs().t() * step(x.shape[1]) for w in (wg, wu))
    sg = silu(g)
    out = dict(h=(sg * u, 1.1 * gb * u.abs() + (sg.abs() + 1.1 * gb) * ub + 2.0 ** -20 * (sg * u).abs()))
    if dh is None:
        return out
    slope = silu_slope(g)
    dg, du = dh * u * slope, dh * sg
    # silu'' is at most 1/2
    dgb = dh.abs() * (0.5 * gb * (u.abs() + ub) + ub * 1.1) + 2.0 ** -20 * (dh * u).abs() * (1 + g.abs())
    dub = dh.abs() * 1.1 * gb + 2.0 ** -20 * du.abs()
    dgb, dub = dgb + (dg.abs() + dgb) * 2.0 ** -8, dub + (du.abs() + dub) * 2.0 ** -8
    R, F = dh.shape
    ga, ua = dg.abs() + dgb, du.abs() + dub
    out["dx"] = (dg @ wg + du @ wu, dgb @ wg.abs() + dub @ wu.abs() +
                 step(2 * F) * (ga @ wg.abs() + ua @ wu.abs()))
    out["dwg"] = (dg.t() @ x, dgb.t() @ x.abs() + step(R) * (ga.t() @ x.abs()))
    out["dwu"] = (du.t() @ x, dub.t() @ x.abs() + step(R) * (ua.t() @ x.abs()))
    return out
