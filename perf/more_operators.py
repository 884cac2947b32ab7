"""Cases, plain forms and exact values of the operators that complete a recurrent block:
a gated linear recurrence with one state per channel, the norms and the residual
sum between two blocks, and the gated feed-forward projections.

    recur:  log a = decay sigmoid(f), or log sigmoid(f) without decay;  m = sqrt(1 - a^2) or 1 - a
            h_t = a_t h_{t-1} + m_t sigmoid(i_t) x_t,   y_t = h_t silu(z_t)
    norm:   p = norm(y) post_weight + post_bias;  s = res + scale p silu(z);  u = norm(s) weight + bias
    glu:    h = silu(x Wg^T) * (x Wu^T)

With ``own`` false ``run`` computes them from elementary torch operations in
fp32; with ``own`` true it calls the library.
"""
import math
import random

import torch

own = False

BF16, F32 = "bf16", "fp32"
EPS = 1e-5


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a dense prompt batch at the sizes of the prefill benchmark (4 x 2048 tokens, 16 x 128 channels):
        # learned decays, both gates and an output gate from one projection (strided rows)
        dict(name="recur_prompt", kind="recur", rows=8192, nseq=4, packed=False, dim=2048, io=BF16, decay=True, unit=True,
             i=True, z=True, init=True),
        # few long ragged prompts: too few channels to fill the GPU without splitting the token axis
        dict(name="recur_long", kind="recur", rows=20001, nseq=3, packed=True, dim=2048, io=BF16, decay=True, unit=True,
             i=True, z=False, init=True),
        # every gradient of the recurrence in a training step
        dict(name="recur_train", kind="recur_bwd", rows=8192, nseq=4, packed=False, dim=2048, io=BF16, decay=True, unit=True,
             i=True, z=True, init=False),
        # a small ragged fp32 fine-tuning batch, odd sizes, the gate itself as decay
        dict(name="recur_train_odd", kind="recur_bwd", rows=777, nseq=5, packed=True, dim=520, io=F32, decay=False,
             unit=False, i=False, z=True, init=True),
        # one token of 64 concurrent sequences over a pool of pages: latency
        dict(name="recur_token", kind="recur_step", nseq=64, dim=2048, io=BF16, decay=True, unit=True, i=True, z=True),
        # between two blocks of a prompt batch: norm of the block's output, its gate, the residual sum in
        # fp32, the next block's norm
        dict(name="norm_prompt", kind="norm", rows=16384, dim=2048, io=BF16, y=True, res32=True, layer=False, post=True,
             z=True, scale=True),
        # the same for one token of a few sequences: latency
        dict(name="norm_token", kind="norm", rows=16, dim=2048, io=BF16, y=True, res32=False, layer=False, post=False,
             z=False, scale=False),
        # every gradient of it in a training step
        dict(name="norm_train", kind="norm_bwd", rows=8192, dim=2048, io=BF16, y=True, res32=False, layer=True, post=True,
             z=True, scale=True),
        # the feed-forward projections of a prompt batch (inner size 8192)
        dict(name="glu_prompt", kind="glu", rows=8192, dim=2048, inner=8192),
        # one token of eight sequences: the weights stream through once
        dict(name="glu_token", kind="glu", rows=8, dim=2048, inner=8192),
        # every gradient in a training step
        dict(name="glu_train", kind="glu_bwd", rows=4096, dim=2048, inner=8192),
        # a small odd batch: partial tiles in every direction
        dict(name="glu_train_odd", kind="glu_bwd", rows=777, dim=520, inner=1352),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["recur", "recur", "recur_bwd", "recur_bwd", "recur_step", "norm", "norm", "norm_bwd", "norm_bwd", "glu",
                       "glu", "glu_bwd"])
    flip = lambda: rng.random() < 0.5  # noqa: E731
    if kind.startswith("glu"):
        dim, inner = 8 * _log(rng, 8, 512), 8 * _log(rng, 16, 1536)
        most = 8192 * 2048 * 8192 // (dim * inner) // (1 if kind == "glu" else 3)
        return dict(kind=kind, rows=_log(rng, 1, min(16384, most)), dim=dim, inner=inner)
    io = rng.choice([BF16, BF16, F32])
    dim = 8 * _log(rng, 8, 512)
    if kind.startswith("norm"):
        most = (16384 if kind == "norm" else 8192) * 2048 // dim // (2 if io == F32 else 1)
        y = rng.random() < 0.85
        return dict(kind=kind, rows=_log(rng, 1, min(65536, most)), dim=dim, io=io, y=y, res32=io == F32 or flip(),
                    layer=flip(), post=y and flip(), z=y and flip(), scale=y and flip())
    gates = dict(decay=flip(), unit=flip(), i=flip(), z=flip())
    if kind == "recur_step":
        return dict(kind=kind, nseq=_log(rng, 1, 1280), dim=dim, io=io, **gates)
    most = (20001 if kind == "recur" else 8192) * 2048 // dim // (2 if io == F32 else 1)
    nseq = _log(rng, 1, 16)
    packed = flip()
    rows = _log(rng, 1, min(65536, most))
    rows = rows if packed else nseq * max(1, rows // nseq)
    if rows > most:
        nseq, rows = 1, most
    return dict(kind=kind, rows=rows, nseq=nseq, packed=packed, dim=dim, io=io, init=flip(), **gates)


def _lengths(case):
    """Lengths of the packed sequences, the same for every seed; an empty one among five or more."""
    if not case["packed"]:
        return [case["rows"] // case["nseq"]] * case["nseq"]
    r = random.Random(case["rows"] * 1009 + case["nseq"])
    cuts = sorted(r.randint(0, case["rows"]) for _ in range(case["nseq"] - 1))
    if len(cuts) >= 4:
        cuts[1] = cuts[2]
    cuts = [0] + cuts + [case["rows"]]
    return [b - a for a, b in zip(cuts, cuts[1:])]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev, kind = "cuda", case["kind"]
    dt_io = torch.float32 if case.get("io") == F32 else torch.bfloat16
    D = case["dim"]

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return torch.empty(*shape, dtype=torch.float32, device=dev).normal_(mean, std, generator=g).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0, dtype=torch.float32):
        return torch.empty(*shape, dtype=torch.float32, device=dev).uniform_(lo, hi, generator=g).to(dtype)

    s = {"case": case}
    if kind.startswith("glu"):
        R, F = case["rows"], case["inner"]
        s["x"] = normal(R, D, dtype=dt_io)                             # a norm's output
        s["wg"], s["wu"] = (uniform(F, D, lo=-(3 / D) ** 0.5, hi=(3 / D) ** 0.5, dtype=dt_io) for _ in range(2))
        if kind == "glu_bwd":
            s["d_out"] = normal(R, F, std=0.1, dtype=dt_io)
        return s
    if kind.startswith("norm"):
        R = case["rows"]
        rt = torch.float32 if case["res32"] else dt_io
        s["res"] = normal(R, D, std=2.0, dtype=rt)
        s["w"] = 1.0 + normal(D, std=0.1)
        s["b"] = normal(D, std=0.1) if case["layer"] else None
        s["y"] = normal(R, D, std=0.7, mean=0.1, dtype=dt_io) if case["y"] else None
        s["pw"] = 1.0 + normal(D, std=0.1) if case["post"] else None
        s["pb"] = normal(D, std=0.1) if case["post"] and case["layer"] else None
        s["z"] = normal(R, 2 * D, dtype=dt_io)[:, D:] if case["z"] else None  # half of the input projection's output
        s["scale"] = normal(D, mean=0.5, std=0.1) if case["scale"] else None
        if kind == "norm_bwd":
            s["du"], s["ds"] = normal(R, D, dtype=dt_io), normal(R, D, std=0.5, dtype=rt)
        return s
    # f, i, x and z are columns of one projection's output
    wide = 1 + 1 + case["i"] + case["z"]
    # the decay of an open gate is u^8 with u between 0.9 and 0.999
    s["decay"] = 8.0 * torch.log(uniform(D, lo=0.9, hi=0.999)) if case["decay"] else None
    mean = 0.0 if case["decay"] else 3.0                               # the gate itself as decay: mostly open
    if kind == "recur_step":
        n = case["nseq"]
        lead = (n,)
        order = torch.randperm(2 * n, generator=g, device=dev).to(torch.int32)
        s["slots"], s["out_slots"] = order[:n].contiguous(), order[n:].contiguous()
        s["pool"] = normal(2 * n, D, std=0.5)
    else:
        cu = [0]
        for x in _lengths(case):
            cu.append(cu[-1] + x)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        s["longest"] = max(_lengths(case))
        lead = (case["rows"],) if case["packed"] else (case["nseq"], case["rows"] // case["nseq"])
        s["init"] = normal(case["nseq"], D, std=0.5) if case["init"] else None
        if kind == "recur_bwd":
            s["d_out"] = normal(*lead, D, dtype=dt_io)
            s["d_final"] = normal(case["nseq"], D) if case["init"] else None
    s["shape"] = (*lead, D)
    s["proj"] = normal(*lead, wide * D, dtype=dt_io)
    if mean:
        s["proj"][..., D:2 * D] += mean
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    kind = s["case"]["kind"]
    if kind.startswith("recur"):
        return _recur(s)
    if kind.startswith("norm"):
        return _norm(s)
    return _glu(s)


def _streams(s):
    """x, f, i, z: columns of the projection's output (i and z where the case has them)."""
    case, D, p = s["case"], s["case"]["dim"], s["proj"]
    i = p[..., 2 * D:3 * D] if case["i"] else None
    return p[..., :D], p[..., D:2 * D], i, p[..., -D:] if case["z"] else None


def _recur(s):
    case, kind = s["case"], s["case"]["kind"]
    x, f, i, z = _streams(s)
    if own:
        import gated_linear_attention_gla_gb300 as gla
        kw = dict(decay=s["decay"], i=i, z=z, unit_variance=case["unit"])
        if kind == "recur_step":
            y = gla.recur_step(x, f, s["pool"], slots=s["slots"], out_slots=s["out_slots"], **kw)
            return {"y": y, "pool": s["pool"]}
        kw.update(init_state=s["init"], cu_seqlens=s["cu"] if case["packed"] else None)
        if kind == "recur":
            y, final = gla.recur_fwd(x, f, **kw)
            return {"y": y, "final": final}
        g = gla.recur_bwd(x, f, s["d_out"], d_final_state=s["d_final"], **kw)
        return dict(zip(("dx", "df", "ddecay", "di", "dz", "d_init"), g))
    if kind == "recur_step":
        a, m, _, _ = _decays(f.float(), s["decay"], case["unit"])
        h = a * s["pool"][s["slots"].long()] + _drive(m, i, x)
        s["pool"][s["out_slots"].long()] = h
        return {"y": _gated(h, z).to(x.dtype), "pool": s["pool"]}
    return _recur_plain(s, x, f, i, z)


def _silu(x):
    return x * torch.sigmoid(x)


def _decays(f, decay, unit):
    """a, m, log a and the forget gate's sigmoid; 1 - a and 1 - a^2 without cancellation."""
    sig = torch.sigmoid(f)
    log_a = decay * sig if decay is not None else -torch.clamp(-f, min=0) - torch.log1p(torch.exp(-torch.abs(f)))
    m = torch.sqrt(-torch.expm1(2 * log_a)) if unit else -torch.expm1(log_a)
    return torch.exp(log_a), m, log_a, sig


def _drive(m, i, x):
    return m * x.float() if i is None else m * torch.sigmoid(i.float()) * x.float()


def _gated(h, z):
    return h if z is None else h * _silu(z.float())


def _doubling(a, x, longest):
    """h_t = a_t h_{t-1} + x_t over the first axis, h_{-1} = 0, in log2(longest) passes."""
    step = 1
    while step < longest:
        x = torch.cat([x[:step], x[step:] + a[step:] * x[:-step]])
        if 2 * step < longest:
            a = torch.cat([a[:step], a[step:] * a[:-step]])
        step *= 2
    return x


def _recur_plain(s, x, f, i, z):
    case = s["case"]
    R, D, B = case["rows"], case["dim"], case["nseq"]
    flat = lambda t: None if t is None else t.reshape(R, D).float()  # noqa: E731
    back = lambda t: t.to(s["proj"].dtype).reshape(s["shape"])  # noqa: E731
    x, f, i, z = map(flat, (x, f, i, z))
    cu = s["cu"].long()
    some = (cu[1:] > cu[:-1])[:, None]
    first, last = cu[:-1].clamp(max=R - 1), (cu[1:] - 1).clamp(min=0)  # rows of the sequences that have any
    r = torch.arange(R, device=x.device)
    inside = (r > cu[torch.searchsorted(s["cu"][1:], r.to(torch.int32), right=True)])[:, None]
    a, m, log_a, sig = _decays(f, s["decay"], case["unit"])
    carry = a * inside
    init = s["init"] if s["init"] is not None else torch.zeros(B, D, device=x.device)
    h = _doubling(carry, _drive(m, i, x).index_add(0, first, torch.where(some, a[first] * init, 0.0)), s["longest"])
    if case["kind"] == "recur":
        return {"y": back(_gated(h, z)), "final": torch.where(some, h[last], init)}
    dy = flat(s["d_out"])
    sz = torch.sigmoid(z) if z is not None else None
    dh = dy * z * sz if z is not None else dy
    d_final = s["d_final"] if s["d_final"] is not None else torch.zeros_like(init)
    # e_t = dL/dh_t = dh_t + a_{t+1} e_{t+1}: the same recurrence from the end
    dh = dh.index_add(0, last, torch.where(some, d_final, 0.0))
    after = torch.cat([carry[1:], torch.zeros_like(carry[:1])])
    e = _doubling(after.flip(0), dh.flip(0), s["longest"]).flip(0)
    before = (torch.cat([torch.zeros_like(h[:1]), h[:-1]]) * inside).index_add(0, first, torch.where(some, init, 0.0))
    si = torch.sigmoid(i) if i is not None else torch.ones_like(x)
    dm = torch.where(m > 0, a * a / m, 0.0) if case["unit"] else a       # -dm / dlog a
    d_log_a = e * (a * before - dm * si * x)
    df = d_log_a * (log_a if s["decay"] is not None else 1.0) * torch.sigmoid(-f)
    return {"dx": back(e * m * si), "df": back(df), "ddecay": (d_log_a * sig).sum(0) if s["decay"] is not None else None,
            "di": back(e * m * x * si * (1 - si)) if i is not None else None,
            "dz": back(dy * h * (sz * (1 + z * (1 - sz)))) if z is not None else None,
            "d_init": torch.where(some, a[first] * e[first], d_final)}


def _normed(x, layer):
    """The normalised rows and 1 / their deviation."""
    if layer:
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * r, r


def _norm_grad(d, n, r, layer):
    """Gradient of the rows from that of the normalised rows."""
    d = d - n * (d * n).mean(-1, keepdim=True)
    if layer:
        d = d - d.mean(-1, keepdim=True)
    return d * r


def _norm(s):
    case = s["case"]
    bwd, layer = case["kind"] == "norm_bwd", case["layer"]
    res, y, z = s["res"], s["y"], s["z"]
    if own:
        import gated_linear_attention_gla_gb300 as gla
        kw = dict(y=y, z=z, post_weight=s["pw"], post_bias=s["pb"], scale=s["scale"], weight=s["w"], bias=s["b"],
                  kind="layer" if layer else "rms", eps=EPS)
        if not bwd:
            return dict(zip(("res", "u"), gla.block_norm_fwd(res, **kw, out_dtype=_io(case))))
        g = gla.block_norm_bwd(res, s["du"], d_res_out=s["ds"], **kw)
        return dict(zip(("d_res", "dy", "dz", "d_post_weight", "d_post_bias", "d_scale", "dw", "db"), g))
    total = res.float()
    if y is not None:
        p, rp = _normed(y.float(), layer) if s["pw"] is not None else (y.float(), None)
        q = p if s["pw"] is None else p * s["pw"]
        if s["pb"] is not None:
            q = q + s["pb"]
        k = _gated(q, z)
        total = total + (k if s["scale"] is None else k * s["scale"])
    n, r = _normed(total, layer)
    if not bwd:
        u = n * s["w"] if s["b"] is None else n * s["w"] + s["b"]
        return {"res": total.to(res.dtype) if y is not None else None, "u": u.to(_io(case))}
    du = s["du"].float()
    d = s["ds"].float() + _norm_grad(du * s["w"], n, r, layer)
    out = {"d_res": d.to(res.dtype), "dy": None, "dz": None, "d_post_weight": None, "d_post_bias": None, "d_scale": None,
           "dw": (du * n).sum(0), "db": du.sum(0) if s["b"] is not None else None}
    if y is None:
        return out
    if s["scale"] is not None:
        out["d_scale"] = (d * k).sum(0)
        d = d * s["scale"]
    if z is not None:
        zf = z.float()
        sig = torch.sigmoid(zf)
        out["dz"] = (d * q * (sig * (1 + zf * (1 - sig)))).to(z.dtype)
        d = d * zf * sig
    if s["pw"] is not None:
        out["d_post_weight"] = (d * p).sum(0)
        out["d_post_bias"] = d.sum(0) if s["pb"] is not None else None
        d = _norm_grad(d * s["pw"], p, rp, layer)
    out["dy"] = d.to(y.dtype)
    return out


def _io(case):
    return torch.float32 if case["io"] == F32 else torch.bfloat16


def _glu(s):
    x, wg, wu = s["x"], s["wg"], s["wu"]
    if own:
        import gated_linear_attention_gla_gb300 as gla
        if s["case"]["kind"] == "glu":
            return {"h": gla.glu_fwd(x, wg, wu)}
        return dict(zip(("dx", "dwg", "dwu"), gla.glu_bwd(x, wg, wu, s["d_out"])))
    dtype = x.dtype
    x, wg, wu = x.float(), wg.float(), wu.float()
    g, u = x @ wg.t(), x @ wu.t()
    sig = torch.sigmoid(g)
    if s["case"]["kind"] == "glu":
        return {"h": (g * sig * u).to(dtype)}
    dh = s["d_out"].float()
    dg, du = dh * u * (sig * (1 + g * (1 - sig))), dh * g * sig
    return {"dx": (dg @ wg + du @ wu).to(dtype), "dwg": (dg.t() @ x).to(dtype), "dwu": (du.t() @ x).to(dtype)}


# ---------------------------------------------------------------------------
# What a pass has to read, write and compute
# ---------------------------------------------------------------------------
def work(case):
    kind, D = case["kind"], case["dim"]
    if kind.startswith("glu"):
        R, F = case["rows"], case["inner"]
        if kind == "glu":
            return {"bytes": 2 * (R * D + 2 * F * D + R * F), "flops": 4 * R * D * F}
        return {"bytes": 2 * (2 * R * D + 4 * F * D + R * F), "flops": 12 * R * D * F}
    e = 4 if case["io"] == F32 else 2
    if kind.startswith("norm"):
        R, t = case["rows"], 4 if case["res32"] else 2
        vectors = 4 * D * (1 + case["layer"] + case["post"] * (1 + case["layer"]) + case["scale"])
        if kind == "norm":
            return {"bytes": R * D * (t * (1 + case["y"]) + e * (1 + case["y"] + case["z"])) + vectors, "flops": 15 * R * D}
        return {"bytes": R * D * (3 * t + e * (1 + 2 * case["y"] + 2 * case["z"])) + 2 * vectors, "flops": 40 * R * D}
    B = case["nseq"]
    ins, par = 2 + case["i"] + case["z"], 4 * D * case["decay"]
    if kind == "recur_step":
        return {"bytes": B * D * (8 + e * (ins + 1)) + par + 8 * B, "flops": 20 * B * D}
    R, state = case["rows"], 4 * B * D
    if kind == "recur":
        return {"bytes": R * D * e * (ins + 1) + par + state * (1 + case["init"]), "flops": 20 * R * D}
    return {"bytes": R * D * e * (2 * ins + 1) + 2 * par + state * (1 + 2 * case["init"]), "flops": 50 * R * D}


# ---------------------------------------------------------------------------
# The definitions in 64 bits: token by token, gradients by reverse mode
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind.startswith("glu"):
        return _exact_glu(s)
    if kind.startswith("norm"):
        return _exact_norm(s)
    return _exact_recur_step(s) if kind == "recur_step" else _exact_recur(s)


def _leaf(t):
    return None if t is None else t.detach().double().requires_grad_(True)


def _grad(t):
    return None if t is None else t.grad


def _silu64(x):
    return x / (1 + torch.exp(-x))


def _gates64(f, i, decay, unit):
    """log a, and the factor of x."""
    gate = 1 / (1 + torch.exp(-f))
    log_a = gate.log() if decay is None else gate * decay
    room = -torch.expm1(log_a)                                         # 1 - a
    if unit:
        room = (room * (2 - room)).sqrt()
    return log_a, room if i is None else room / (1 + torch.exp(-i))


def _exact_recur_step(s):
    case = s["case"]
    d = lambda t: None if t is None else t.double()  # noqa: E731
    x, f, i, z = map(d, _streams(s))
    pool = s["pool"].double()
    log_a, w = _gates64(f, i, d(s["decay"]), case["unit"])
    h = pool[s["slots"].long()] * log_a.exp() + w * x
    pool[s["out_slots"].long()] = h
    return {"y": h if z is None else h * _silu64(z), "pool": pool}


class _Walk(torch.autograd.Function):
    """h_t = a_t h_{t-1} + b_t for one sequence [T, D] from h_{-1}, one token after another."""

    @staticmethod
    def forward(ctx, a, b, h):
        front, states = h, []
        for x, y in zip(a.unbind(0), b.unbind(0)):
            h = x * h + y
            states.append(h)
        states = torch.stack(states)
        ctx.save_for_backward(a, states, front)
        return states

    @staticmethod
    def backward(ctx, d):
        a, states, front = ctx.saved_tensors
        e, es = torch.zeros_like(front), []
        for x, y in zip(reversed(a.unbind(0)), reversed(d.unbind(0))):
            e = e + y
            es.append(e)
            e = e * x
        es = torch.stack(es[::-1])
        return es * torch.cat([front[None], states[:-1]]), es, e


def _exact_recur(s):
    case = s["case"]
    R, D, B = case["rows"], case["dim"], case["nseq"]
    bwd = case["kind"] == "recur_bwd"
    keep = _leaf if bwd else (lambda t: None if t is None else t.double())
    x, f, i, z = (keep(None if t is None else t.reshape(R, D)) for t in _streams(s))
    decay = keep(s["decay"])
    init = keep(s["init"] if s["init"] is not None else torch.zeros(B, D, device=s["proj"].device))
    log_a, w = _gates64(f, i, decay, case["unit"])
    a, b = log_a.exp(), w * x
    cu = s["cu"].tolist()
    hs, finals = [], []
    for k, (lo, hi) in enumerate(zip(cu, cu[1:])):
        if hi > lo:
            hs.append(_Walk.apply(a[lo:hi], b[lo:hi], init[k]))
        finals.append(hs[-1][-1] if hi > lo else init[k])
    h, finals = torch.cat(hs), torch.stack(finals)
    y = h if z is None else h * _silu64(z)
    if not bwd:
        return {"y": y.reshape(s["shape"]), "final": finals}
    loss = (y * s["d_out"].reshape(R, D).double()).sum()
    if s["d_final"] is not None:
        loss = loss + (finals * s["d_final"].double()).sum()
    loss.backward()
    shaped = lambda t: None if t is None else t.grad.reshape(s["shape"])  # noqa: E731
    return {"dx": shaped(x), "df": shaped(f), "ddecay": _grad(decay), "di": shaped(i), "dz": shaped(z), "d_init": init.grad}


def _exact_norm(s):
    case = s["case"]
    bwd = case["kind"] == "norm_bwd"
    keep = _leaf if bwd else (lambda t: None if t is None else t.double())
    res, y, z, pw, pb, scale, w, b = (keep(s[k]) for k in ("res", "y", "z", "pw", "pb", "scale", "w", "b"))

    def norm(x, weight, bias):
        if case["layer"]:
            x = x - x.sum(1, keepdim=True) / case["dim"]
        x = x / (x.square().sum(1, keepdim=True) / case["dim"] + EPS).sqrt() * weight
        return x if bias is None else x + bias

    total = res
    if y is not None:
        p = y if pw is None else norm(y, pw, pb)
        p = p if z is None else p * _silu64(z)
        total = res + (p if scale is None else p * scale)
    u = norm(total, w, b)
    if not bwd:
        return {"res": None if y is None else total, "u": u}
    ((u * s["du"].double()).sum() + (total * s["ds"].double()).sum()).backward()
    return {"d_res": res.grad, "dy": _grad(y), "dz": _grad(z), "d_post_weight": _grad(pw), "d_post_bias": _grad(pb),
            "d_scale": _grad(scale), "dw": w.grad, "db": _grad(b)}


def _exact_glu(s):
    if s["case"]["kind"] == "glu":
        x, wg, wu = (s[k].double() for k in ("x", "wg", "wu"))
        return {"h": _silu64(x @ wg.t()) * (x @ wu.t())}
    x, wg, wu = (_leaf(s[k]) for k in ("x", "wg", "wu"))
    (_silu64(x @ wg.t()) * (x @ wu.t()) * s["d_out"].double()).sum().backward()
    return {"dx": x.grad, "dwg": wg.grad, "dwu": wu.grad}
