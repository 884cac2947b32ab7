"""Plain 64-bit implementations of the causal convolution and the selective scan
with their gradients (formulas, token by token), for the tests.

``absolute=True`` evaluates the same sums over the absolute values of their
terms (decays and step sizes as they are): what rounding errors scale with.
Sequences are given by ``cu``, a list of packed offsets.
"""
from __future__ import annotations

import torch


def d(t):
    return None if t is None else t.detach().double().cpu()


def sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def silu(x):
    return x * sigmoid(x)


def silu_grad(x):
    s = sigmoid(x)
    return s * (1 + x * (1 - s))


def conv(x, w, bias, init, cu, act, dy=None, d_final=None, absolute=False):
    """x [R, D], w [D, W], init [B, W-1, D]; dict of y, final and, with dy, the gradients."""
    x, w, bias, init, dy, d_final = map(d, (x, w, bias, init, dy, d_final))
    R, D = x.shape
    W = w.shape[1]
    K, B = W - 1, len(cu) - 1
    ab = torch.abs if absolute else (lambda t: t)
    out = dict(y=torch.zeros(R, D).double(), final=torch.zeros(B, K, D).double(),
               dx=torch.zeros(R, D).double(), dw=torch.zeros(D, W).double(),
               db=torch.zeros(D).double(), d_init=torch.zeros(B, K, D).double())
    for s in range(B):
        lo, hi = cu[s], cu[s + 1]
        front = init[s] if init is not None else torch.zeros(K, D).double()
        seq = torch.cat([front, x[lo:hi]])
        T = hi - lo
        out["final"][s] = seq[T:]
        p = torch.zeros(T, D).double() if bias is None else bias.expand(T, D).clone()
        pa = p.abs()
        for k in range(W):
            p = p + w[:, k] * seq[k:k + T]
            pa = pa + (w[:, k] * seq[k:k + T]).abs()
        out["y"][lo:hi] = (pa if absolute else silu(p) if act else p)
        if dy is None:
            continue
        # a sum's rounding moves silu' by at most half of its own size
        dp = dy[lo:hi] * (silu_grad(p) if act else 1.0)
        if absolute:
            dp = dy[lo:hi].abs() * ((silu_grad(p).abs() + pa) if act else 1.0)
        g = torch.zeros(K + T, D).double()
        for k in range(W):
            g[k:k + T] += ab(w[:, k]) * dp
            out["dw"][:, k] += (dp * ab(seq[k:k + T])).sum(0)
        out["db"] += dp.sum(0)
        if d_final is not None:
            g[T:] += ab(d_final[s])
        out["d_init"][s], out["dx"][lo:hi] = g[:K], g[K:]
    return out


def scan(u, dt, a, b, c, skip, z, bias, softplus, init, cu, dy=None, d_final=None, absolute=False):
    """u, dt, z [R, D], a [D, N], b, c [R, N], init [B, D, N]; dict of y, final and the gradients."""
    u, dt, a, b, c, skip, z, bias, init, dy, d_final = map(
        d, (u, dt, a, b, c, skip, z, bias, init, dy, d_final))
    R, D = u.shape
    N, B = a.shape[1], len(cu) - 1
    x = dt if bias is None else dt + bias
    delta = torch.where(x > 30, x, torch.log1p(torch.exp(x.clamp(max=30)))) if softplus else x
    slope = sigmoid(x) if softplus else torch.ones_like(x)
    decay = torch.exp(delta[..., None] * a)
    zero = torch.zeros(B, D, N).double()
    h0 = init if init is not None else zero
    gate, dgate = (silu(z), silu_grad(z)) if z is not None else (None, None)
    if absolute:
        u, a, b, c, h0 = u.abs(), a.abs(), b.abs(), c.abs(), h0.abs()
        skip = None if skip is None else skip.abs()
        dy = None if dy is None else dy.abs()
        d_final = None if d_final is None else d_final.abs()
        if z is not None:
            gate, dgate = gate.abs(), sigmoid(z) * (1 + z.abs())
        drive = delta.abs()
    else:
        drive = delta
    h = torch.zeros(R, D, N).double()
    before = torch.zeros(R, D, N).double()
    final = zero.clone()
    for s in range(B):
        cur = h0[s]
        for t in range(cu[s], cu[s + 1]):
            before[t] = cur
            cur = decay[t] * cur + (drive[t] * u[t])[:, None] * b[t]
            h[t] = cur
        final[s] = cur
    y = (h * c[:, None]).sum(-1)
    if skip is not None:
        y = y + skip * u
    out = dict(y=y * gate if z is not None else y, final=final)
    if dy is None:
        return out
    g = dy * gate if z is not None else dy
    e = torch.zeros(R, D, N).double()
    d_init = zero.clone()
    for s in range(B):
        cur = d_final[s] if d_final is not None else zero[s]
        for t in reversed(range(cu[s], cu[s + 1])):
            e[t] = g[t][:, None] * c[t] + cur
            cur = decay[t] * e[t]
        d_init[s] = cur
    eb = (e * b[:, None]).sum(-1)
    w = e * decay * before
    ddelta = (w * a).sum(-1) + u * eb
    ddt = ddelta * slope
    out.update(du=drive * eb + (skip * g if skip is not None else 0), ddt=ddt,
               da=(w * drive[..., None]).sum(0), db=(e * (drive * u)[..., None]).sum(1),
               dc=(h * g[..., None]).sum(1), dskip=(g * u).sum(0) if skip is not None else None,
               dz=dy * y * dgate if z is not None else None,
               dbias=ddt.sum(0) if bias is not None else None, d_init=d_init)
    return out
