"""Cases, plain forms and exact values of the selective-scan operators and of the
page operators of a state pool.

A selective-scan layer runs, per token and channel, a short causal convolution
(``conv_*``), a state space scan whose decay depends on the token (``scan_*``),
and keeps both states in pools of pages, one page per sequence, which a server
forks and compacts (``fork_pages``, ``compact_pages``, ``free_pages``).

    conv:  p_t[d] = bias[d] + sum_j weight[d][W-1-j] x_{t-j}[d],   y = silu(p) or p
    scan:  delta = softplus(dt + dt_bias),  h_t[d][n] = exp(delta a[d][n]) h_{t-1}[d][n] + delta u b_t[n],
           y_t[d] = (sum_n c_t[n] h_t[d][n] + skip[d] u) * silu(z)

With ``own`` false ``run`` computes them from elementary torch operations in
fp32; with ``own`` true it calls the library.
"""
import math
import random

import torch

own = False

BF16, F32 = "bf16", "fp32"


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # prompts of sixteen requests packed into one call in front of the scan: x is
        # half of the input projection's output (strided rows); about 1.1 GB of tensors
        dict(name="conv_prompt", kind="conv", rows=65536, nseq=16, packed=True, dim=2048, width=4, io=BF16, silu=True,
             bias=True, init=True),
        # the convolution's gradients in a training step
        dict(name="conv_train", kind="conv_bwd", rows=8192, nseq=4, packed=False, dim=2048, width=4, io=BF16, silu=True,
             bias=True, init=False),
        # one token of 64 concurrent sequences: latency
        dict(name="conv_token", kind="conv_step", nseq=64, dim=2048, width=4, io=BF16, silu=True, bias=True),
        # a dense prompt batch at the sizes of the prefill benchmark (4 x 2048 tokens, 16 x 128 channels)
        dict(name="scan_prompt", kind="scan", rows=8192, nseq=4, packed=False, dim=2048, n=16, io=BF16, z=True, skip=True,
             init=True),
        # few long ragged prompts: too few channels to fill the GPU without splitting the token axis
        dict(name="scan_long", kind="scan", rows=20001, nseq=3, packed=True, dim=2048, n=16, io=BF16, z=True, skip=True,
             init=True),
        # every gradient of the scan in a training step
        dict(name="scan_train", kind="scan_bwd", rows=8192, nseq=4, packed=False, dim=2048, n=16, io=BF16, z=True,
             skip=True, init=False),
        # a small ragged fp32 fine-tuning batch, odd sizes, no gate
        dict(name="scan_train_odd", kind="scan_bwd", rows=777, nseq=5, packed=True, dim=520, n=8, io=F32, z=False,
             skip=True, init=True),
        # one token of one sequence: latency
        dict(name="scan_token_one", kind="scan_step", nseq=1, dim=2048, n=16, io=BF16, z=True, skip=True),
        # one token of 1280 concurrent sequences, the decode benchmark's batch
        dict(name="scan_token_many", kind="scan_step", nseq=1280, dim=2048, n=16, io=BF16, z=True, skip=True),
        # four samples forked from running requests in a small pool: latency
        dict(name="fork_few", kind="fork", slots=64, live=24, forks=4, fresh=0, layers=1, state=2048 * 16, tail=3 * 2048),
        # a beam step over a large batch: 256 forks and some new requests in four layers' pools
        dict(name="fork_many", kind="fork", slots=1280, live=900, forks=240, fresh=16, layers=4, state=2048 * 16,
             tail=3 * 2048),
        # half of a pool of linear-attention states (16 heads of 128 x 128) has finished: free, then compact
        dict(name="compact_half", kind="compact", slots=1024, live=800, done=288, layers=1, state=16 * 128 * 128, tail=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["conv", "conv_bwd", "conv_step", "scan", "scan", "scan_bwd", "scan_bwd", "scan_step", "fork", "compact"])
    io = rng.choice([BF16, BF16, F32])
    dim = 8 * _log(rng, 8, 512)
    flip = lambda: rng.random() < 0.5  # noqa: E731
    if kind in ("conv", "conv_bwd"):
        most = (65536 if kind == "conv" else 8192) * 2048 // dim // (2 if io == F32 else 1)
        nseq = _log(rng, 1, 16)
        packed = flip()
        rows = _log(rng, 1, min(65536, most))
        rows = rows if packed else nseq * max(1, rows // nseq)
        if rows > most:
            nseq, rows = 1, most
        return dict(kind=kind, rows=rows, nseq=nseq, packed=packed, dim=dim, width=rng.randint(2, 4), io=io, silu=flip(),
                    bias=flip(), init=flip())
    if kind == "conv_step":
        return dict(kind=kind, nseq=_log(rng, 1, 1280), dim=dim, width=rng.randint(2, 4), io=io, silu=flip(), bias=flip())
    if kind in ("scan", "scan_bwd"):
        n = rng.choice([8, 16, 16, 32, 64])
        most = (17000 if kind == "scan" else 8192) * 2048 * 16 // (dim * n) // (2 if io == F32 else 1)
        nseq = _log(rng, 1, 16)
        packed = flip()
        rows = _log(rng, 1, min(20001, most))
        rows = rows if packed else nseq * max(1, rows // nseq)
        if rows > most:
            nseq, rows = 1, most
        return dict(kind=kind, rows=rows, nseq=nseq, packed=packed, dim=dim, n=n, io=io, z=flip(), skip=flip(), init=flip())
    if kind == "scan_step":
        n = rng.choice([8, 16, 16, 32, 64])
        return dict(kind=kind, nseq=_log(rng, 1, max(1, 1280 * 2048 * 16 // max(dim * n, 2048 * 16))), dim=dim, n=n, io=io,
                    z=flip(), skip=flip())
    slots = _log(rng, 8, 1024)
    live = rng.randint(1, slots)
    layers = rng.randint(1, 4)
    state = 4 * _log(rng, 256, min(65536, 131072 * 768 // (4 * slots * layers)))
    tail = rng.choice([0, 8 * _log(rng, 64, min(1536, state // 8))])
    if kind == "fork":
        forks = rng.randint(0, slots - live)
        return dict(kind=kind, slots=slots, live=live, forks=forks, fresh=rng.randint(0, min(16, slots - live - forks)),
                    layers=layers, state=state, tail=tail)
    return dict(kind=kind, slots=slots, live=live, done=rng.randint(0, live), layers=layers, state=state, tail=tail)


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


def _dtype(case):
    return torch.bfloat16 if case["io"] == BF16 else torch.float32


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = "cuda"

    def normal(*shape, std=1.0, dtype=torch.float32):
        return torch.empty(*shape, dtype=torch.float32, device=dev).normal_(0.0, std, generator=g).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.empty(*shape, dtype=torch.float32, device=dev).uniform_(lo, hi, generator=g)

    kind, s = case["kind"], {"case": case}
    if kind in ("fork", "compact"):
        S, L = case["slots"], case["live"]
        order = torch.randperm(S, generator=g, device=dev).to(torch.int32)
        used = torch.zeros(S, dtype=torch.int32, device=dev)
        used[order[:L].long()] = 1
        s["used"] = used
        s["pools"] = [normal(S, case["state"]) for _ in range(case["layers"])]
        if case["tail"]:
            s["pools"] += [normal(S, case["tail"], dtype=torch.bfloat16) for _ in range(case["layers"])]
        if kind == "fork":
            pick = torch.randint(0, L, (case["forks"],), generator=g, device=dev)
            s["parents"] = torch.cat([order[:L][pick], torch.full((case["fresh"],), -2, dtype=torch.int32, device=dev)])
        else:
            s["done"] = order[:case["done"]].contiguous()
            s["slots"] = order[case["done"]:L].contiguous()
        return s

    dim, dt_io = case["dim"], _dtype(case)
    if kind in ("conv", "conv_bwd", "conv_step"):
        W = case["width"]
        s["weight"] = uniform(dim, W, lo=-W ** -0.5, hi=W ** -0.5)
        s["bias"] = uniform(dim, lo=-W ** -0.5, hi=W ** -0.5) if case["bias"] else None
    else:
        N = case["n"]
        s["a"] = -torch.arange(1, N + 1, device=dev, dtype=torch.float32) * torch.exp(normal(dim, N, std=0.1))
        delta = torch.exp(uniform(dim, lo=math.log(1e-3), hi=math.log(1e-1)))
        s["dt_bias"] = delta + torch.log(-torch.expm1(-delta))  # softplus(dt_bias) = delta
        s["skip"] = 1.0 + normal(dim, std=0.1) if case["skip"] else None
    if kind in ("conv_step", "scan_step"):
        n = case["nseq"]
        order = torch.randperm(2 * n, generator=g, device=dev).to(torch.int32)
        s["slots"], s["out_slots"] = order[:n].contiguous(), order[n:].contiguous()
        if kind == "conv_step":
            s["xz"] = normal(n, 2 * dim, dtype=dt_io)  # the input projection's output: x and the gate's half
            s["pool"] = normal(2 * n, W - 1, dim, dtype=dt_io)
        else:
            s["u"] = normal(n, dim, dtype=dt_io)
            s["dt"] = normal(n, dim, std=0.5, dtype=dt_io)
            s["xz"] = normal(n, 2 * dim, dtype=dt_io) if case["z"] else None
            s["bc"] = normal(n, 64 + 2 * N, dtype=dt_io)  # the projection of dt's rank, b and c
            s["pool"] = normal(2 * n, dim, N, std=0.5)
        return s
    R, lens = case["rows"], _lengths(case)
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    s["longest"] = max(lens)
    s["shape"] = (R, dim) if case["packed"] else (case["nseq"], R // case["nseq"], dim)
    lead = s["shape"][:-1]
    B = case["nseq"]
    if kind in ("conv", "conv_bwd"):
        s["xz"] = normal(*lead, 2 * dim, dtype=dt_io)
        s["init"] = normal(B, W - 1, dim, dtype=dt_io) if case["init"] else None
        if kind == "conv_bwd":
            s["d_out"] = normal(*lead, dim, dtype=dt_io)
            s["d_final"] = normal(B, W - 1, dim) if case["init"] else None
    else:
        s["u"] = normal(*lead, dim, dtype=dt_io)
        s["dt"] = normal(*lead, dim, std=0.5, dtype=dt_io)
        s["xz"] = normal(*lead, 2 * dim, dtype=dt_io) if case["z"] else None
        s["bc"] = normal(*lead, 64 + 2 * N, dtype=dt_io)
        s["init"] = normal(B, dim, N, std=0.5) if case["init"] else None
        if kind == "scan_bwd":
            s["d_out"] = normal(*lead, dim, dtype=dt_io)
            s["d_final"] = normal(B, dim, N) if case["init"] else None
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    kind = s["case"]["kind"]
    if kind in ("fork", "compact"):
        return _pages(s)
    if kind.startswith("conv"):
        return _conv(s)
    return _scan(s)


def _halves(s):
    """x (or u's gate z): the first and second halves of the input projection's output."""
    dim = s["case"]["dim"]
    return s["xz"][..., :dim], s["xz"][..., dim:]


def _bc(s):
    N = s["case"]["n"]
    return s["bc"][..., 64:64 + N], s["bc"][..., 64 + N:]


def _conv(s):
    case, kind = s["case"], s["case"]["kind"]
    x = _halves(s)[0]
    if own:
        import gated_linear_attention_gla_gb300 as gla
        act = "silu" if case["silu"] else None
        cu = s["cu"] if case.get("packed") else None
        if kind == "conv":
            y, final = gla.conv_fwd(x, s["weight"], s["bias"], init_state=s["init"], cu_seqlens=cu, activation=act)
            return {"y": y, "final": final}
        if kind == "conv_bwd":
            dx, dw, db, di = gla.conv_bwd(x, s["weight"], s["d_out"], s["bias"], init_state=s["init"],
                                          d_final_state=s["d_final"], cu_seqlens=cu, activation=act)
            return {"dx": dx, "dw": dw, "db": db, "d_init": di}
        y = gla.conv_step(x, s["weight"], s["pool"], s["bias"], activation=act, slots=s["slots"], out_slots=s["out_slots"])
        return {"y": y, "pool": s["pool"]}
    return _conv_step_plain(s, x) if kind == "conv_step" else _conv_plain(s, x)


def _conv_step_plain(s, x):
    case = s["case"]
    old = s["pool"][s["slots"].long()]
    window = torch.cat([old, x[:, None]], dim=1)                       # [n, W, D]
    p = (window.float() * s["weight"].t()).sum(1)
    if s["bias"] is not None:
        p = p + s["bias"]
    y = p * torch.sigmoid(p) if case["silu"] else p
    s["pool"][s["out_slots"].long()] = window[:, 1:]
    return {"y": y.to(x.dtype), "pool": s["pool"]}


def _rows_of(cu, R):
    """Sequence, position and length of each packed row."""
    r = torch.arange(R, device=cu.device)
    seq = torch.searchsorted(cu[1:], r.to(torch.int32), right=True)
    return r, seq, r - cu[seq], cu[seq + 1] - cu[seq]


def _conv_plain(s, x):
    """Rows with the initial state's in front of them all; each tap is a gather of those rows."""
    case = s["case"]
    W, dim, R, B = case["width"], case["dim"], case["rows"], case["nseq"]
    cu, K = s["cu"].long(), case["width"] - 1
    dev = x.device
    init = s["init"] if s["init"] is not None else torch.zeros(B, K, dim, dtype=x.dtype, device=dev)
    rows = torch.cat([init.reshape(B * K, dim), x.reshape(R, dim)])    # row B*K + r is packed row r
    r, seq, pos, _ = _rows_of(s["cu"], R)
    back = K - torch.arange(W, device=dev)                             # tap w reaches back[w] tokens
    at = pos[:, None] - back
    taps = torch.where(at >= 0, B * K + r[:, None] - back, seq[:, None] * K + K + at)
    window = rows[taps].float()                                        # [R, W, D]
    p = (window * s["weight"].t()).sum(1)
    if s["bias"] is not None:
        p = p + s["bias"]
    i = torch.arange(K, device=dev)
    lens = (cu[1:] - cu[:-1])[:, None]
    end = lens - K + i                                                 # position of the final state's rows
    last = torch.where(end >= 0, B * K + cu[:-1, None] + end, torch.arange(B, device=dev)[:, None] * K + K + end)
    if case["kind"] == "conv":
        y = p * torch.sigmoid(p) if case["silu"] else p
        return {"y": y.to(x.dtype).reshape(s["shape"]), "final": rows[last]}
    d_p = s["d_out"].reshape(R, dim).float()
    if case["silu"]:
        sig = torch.sigmoid(p)
        d_p = d_p * (sig * (1 + p * (1 - sig)))
    d_w = (window * d_p[:, None]).sum(0).t().contiguous()
    # the gradient of every row, the initial state's too: tap W-1-j of the token j later
    seq_q = torch.cat([torch.arange(B, device=dev).repeat_interleave(K, output_size=B * K), seq])
    pos_q = torch.cat([(i - K).repeat(B), pos])
    j = torch.arange(W, device=dev)
    to = pos_q[:, None] + j
    ok = (to >= 0) & (to < lens[seq_q])
    src = torch.where(ok, cu[seq_q, None] + to, 0)
    d_rows = (d_p[src] * ok[..., None] * s["weight"].t().flip(0)).sum(1)
    if s["d_final"] is not None:
        d_rows = d_rows.index_add(0, last.reshape(-1), s["d_final"].reshape(B * K, dim))
    return {"dx": d_rows[B * K:].to(x.dtype).reshape(s["shape"]), "dw": d_w,
            "db": d_p.sum(0) if s["bias"] is not None else None, "d_init": d_rows[:B * K].reshape(B, K, dim)}


def _scan(s):
    case, kind = s["case"], s["case"]["kind"]
    z = _halves(s)[1] if case["z"] else None
    b, c = _bc(s)
    if own:
        import gated_linear_attention_gla_gb300 as gla
        cu = s["cu"] if case.get("packed") else None
        if kind == "scan":
            y, final = gla.scan_fwd(s["u"], s["dt"], s["a"], b, c, skip=s["skip"], z=z, dt_bias=s["dt_bias"],
                                    init_state=s["init"], cu_seqlens=cu)
            return {"y": y, "final": final}
        if kind == "scan_bwd":
            g = gla.scan_bwd(s["u"], s["dt"], s["a"], b, c, s["d_out"], skip=s["skip"], z=z, dt_bias=s["dt_bias"],
                             init_state=s["init"], d_final_state=s["d_final"], cu_seqlens=cu)
            return dict(zip(("du", "ddt", "da", "db", "dc", "dskip", "dz", "ddt_bias", "d_init"), g))
        y = gla.scan_step(s["u"], s["dt"], s["a"], b, c, s["pool"], skip=s["skip"], z=z, dt_bias=s["dt_bias"],
                          slots=s["slots"], out_slots=s["out_slots"])
        return {"y": y, "pool": s["pool"]}
    return _scan_step_plain(s, z, b, c) if kind == "scan_step" else _scan_plain(s, z, b, c)


def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-torch.abs(x)))


def _scan_step_plain(s, z, b, c):
    u = s["u"].float()
    delta = _softplus(s["dt"].float() + s["dt_bias"])
    h = torch.exp(delta[..., None] * s["a"]) * s["pool"][s["slots"].long()] + (delta * u)[..., None] * b.float()[:, None]
    y = (h * c.float()[:, None]).sum(-1)
    if s["skip"] is not None:
        y = y + s["skip"] * u
    if z is not None:
        y = y * (z.float() * torch.sigmoid(z.float()))
    s["pool"][s["out_slots"].long()] = h
    return {"y": y.to(s["u"].dtype), "pool": s["pool"]}


def _doubling(a, x, longest):
    """h_t = a_t h_{t-1} + x_t over the first axis, h_{-1} = 0, in log2(longest) passes."""
    step = 1
    while step < longest:
        x = torch.cat([x[:step], x[step:] + a[step:] * x[:-step]])
        if 2 * step < longest:
            a = torch.cat([a[:step], a[step:] * a[:-step]])
        step *= 2
    return x


def _scan_plain(s, z, b, c):
    case = s["case"]
    R, dim, N = case["rows"], case["dim"], case["n"]
    cu = s["cu"].long()
    some = cu[1:] > cu[:-1]
    first, last = cu[:-1].clamp(max=R - 1), (cu[1:] - 1).clamp(min=0)  # rows of the sequences that have any
    dtype, A = s["u"].dtype, s["a"]
    u = s["u"].reshape(R, dim).float()
    x = s["dt"].reshape(R, dim).float() + s["dt_bias"]
    bm, cm = b.reshape(R, N).float(), c.reshape(R, N).float()
    delta = _softplus(x)
    _, _, pos, lens = _rows_of(s["cu"], R)
    inside = (pos > 0).float()[:, None, None]
    decay = torch.exp(delta[..., None] * A)
    drive = (delta * u)[..., None] * bm[:, None]
    if s["init"] is not None:
        drive.index_add_(0, first, torch.where(some[:, None, None], decay[first] * s["init"], 0.0))
    h = _doubling(decay * inside, drive, s["longest"])
    del drive
    y = (h * cm[:, None]).sum(-1)
    if s["skip"] is not None:
        y = y + s["skip"] * u
    if z is not None:
        zf = z.reshape(R, dim).float()
        sig = torch.sigmoid(zf)
    init = s["init"] if s["init"] is not None else torch.zeros(case["nseq"], dim, N, device=A.device)
    if case["kind"] == "scan":
        out = y * (zf * sig) if z is not None else y
        return {"y": out.to(dtype).reshape(s["shape"]), "final": torch.where(some[:, None, None], h[last], init)}
    g = s["d_out"].reshape(R, dim).float()
    dz = None
    if z is not None:
        dz = (g * y * (sig * (1 + zf * (1 - sig)))).to(dtype).reshape(s["shape"])
        g = g * (zf * sig)
    # e_t = dL/dh_t = c_t g_t + decay_{t+1} e_{t+1}: the same recurrence from the end
    drive = g[..., None] * cm[:, None]
    if s["d_final"] is not None:
        drive.index_add_(0, last, torch.where(some[:, None, None], s["d_final"], 0.0))
    after = torch.cat([decay[1:] * inside[1:], torch.zeros_like(decay[:1])])
    e = _doubling(after.flip(0), drive.flip(0), s["longest"]).flip(0)
    del drive, after
    dc = (h * g[..., None]).sum(1)
    db = (e * (delta * u)[..., None]).sum(1)
    eb = (e * bm[:, None]).sum(-1)
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]]) * inside
    before.index_add_(0, first, torch.where(some[:, None, None], init, 0.0))
    del h
    w = e * decay * before
    del before
    d_delta = (w * A).sum(-1) + u * eb
    du = delta * eb + (s["skip"] * g if s["skip"] is not None else 0.0)
    ddt = d_delta * torch.sigmoid(x)
    zero = s["d_final"] if s["d_final"] is not None else torch.zeros_like(init)
    return {"du": du.to(dtype).reshape(s["shape"]), "ddt": ddt.to(dtype).reshape(s["shape"]),
            "da": (w * delta[..., None]).sum(0), "db": db.to(dtype).reshape(*s["shape"][:-1], N),
            "dc": dc.to(dtype).reshape(*s["shape"][:-1], N), "dskip": (g * u).sum(0) if s["skip"] is not None else None,
            "dz": dz, "ddt_bias": ddt.sum(0), "d_init": torch.where(some[:, None, None], decay[first] * e[first], zero)}


def _pages(s):
    case, pools, used = s["case"], s["pools"], s["used"]
    if own:
        import gated_linear_attention_gla_gb300 as gla
        if case["kind"] == "fork":
            children, left = gla.fork_pages(pools, used, s["parents"], used_out=torch.empty_like(used))
            return {"children": children, "used": left, "pools": pools}
        left = gla.free_pages(used, s["done"], used_out=torch.empty_like(used))
        slots, left, moved = gla.compact_pages(pools, left, s["slots"])
        return {"slots": slots, "used": left, "moved": moved, "pools": pools}
    S = case["slots"]
    page = torch.arange(S, device=used.device)
    if case["kind"] == "fork":
        n = case["forks"] + case["fresh"]
        children = torch.sort(used, stable=True)[1][:n]                # the lowest free pages first
        left = used.index_fill(0, children, 1)
        new = (s["parents"] == -2)[:, None]
        for pool in pools:
            pool[children] = torch.where(new, 0.0, pool[s["parents"].clamp(min=0).long()]).to(pool.dtype)
        return {"children": children.to(torch.int32), "used": left, "pools": pools}
    left = used.index_fill(0, s["done"].long(), 0)
    live = left != 0
    L = live.sum()
    # the k-th live page at or behind L goes to the k-th free page in front of L; the
    # list is padded with the last page onto itself (it is no free page in front of L)
    far, hole = live & (page >= L), ~live & (page < L)
    holes = torch.sort(~hole, stable=True)[1][:S // 2 + 1]
    some = torch.arange(S // 2 + 1, device=used.device) < hole.sum()
    src = torch.where(some, torch.sort(~far, stable=True)[1][:S // 2 + 1], S - 1)
    dst = torch.where(some, holes, S - 1)
    rank = (torch.cumsum(far, 0) - 1).clamp(0, S // 2)
    moved = torch.where(far, holes[rank], torch.where(live, page, -1))
    for pool in pools:
        pool[dst] = pool[src]
    return {"slots": moved[s["slots"].long()].to(torch.int32), "used": (page < L).to(torch.int32),
            "moved": moved.to(torch.int32), "pools": pools}


# ---------------------------------------------------------------------------
# What a pass has to read, write and compute
# ---------------------------------------------------------------------------
def work(case):
    kind = case["kind"]
    if kind in ("fork", "compact"):
        page = case["layers"] * (4 * case["state"] + 2 * case["tail"])
        if kind == "fork":
            moved = case["forks"] * 2 + case["fresh"]                  # read and written, or zeroed
            return {"bytes": moved * page + 8 * case["slots"] + 8 * (case["forks"] + case["fresh"]), "flops": 0}
        L = case["live"] - case["done"]
        return {"bytes": 2 * L * (1 - L / case["slots"]) * page + 16 * case["slots"] + 8 * L, "flops": 0}
    e, D, B = 2 if case["io"] == BF16 else 4, case["dim"], case["nseq"]
    if kind == "conv_step":
        W = case["width"]
        return {"bytes": B * D * e * (2 * W) + D * 4 * (W + case["bias"]), "flops": 2 * B * D * W}
    if kind in ("conv", "conv_bwd"):
        W, R = case["width"], case["rows"]
        par = D * 4 * (W + case["bias"])
        state = B * (W - 1) * D
        if kind == "conv":
            return {"bytes": 2 * R * D * e + par + state * e * (1 + case["init"]), "flops": 2 * R * D * W}
        return {"bytes": 3 * R * D * e + 2 * par + state * (4 + case["init"] * (4 + e)), "flops": 6 * R * D * W}
    N = case["n"]
    par = 4 * D * (N + 1 + case["skip"])
    if kind == "scan_step":
        return {"bytes": B * (2 * 4 * D * N + D * e * (3 + case["z"]) + 2 * N * e) + par, "flops": 7 * B * D * N}
    R = case["rows"]
    state = 4 * B * D * N
    if kind == "scan":
        return {"bytes": R * e * (D * (3 + case["z"]) + 2 * N) + par + state * (1 + case["init"]), "flops": 7 * R * D * N}
    return {"bytes": R * e * (D * (5 + 2 * case["z"]) + 4 * N) + 2 * par + state * (1 + 2 * case["init"]),
            "flops": 25 * R * D * N}


# ---------------------------------------------------------------------------
# The definitions in 64 bits: token by token, gradients by reverse mode
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind in ("fork", "compact"):
        return _exact_pages(s)
    if kind == "conv_step":
        return _exact_conv_step(s)
    if kind == "scan_step":
        return _exact_scan_step(s)
    if kind.startswith("conv"):
        return _exact_conv(s)
    return _exact_scan(s)


def _silu64(x):
    return x / (1 + torch.exp(-x))


def _leaf(t):
    return None if t is None else t.detach().double().requires_grad_(True)


def _exact_conv(s):
    case = s["case"]
    D, W, K = case["dim"], case["width"], case["width"] - 1
    x = _halves(s)[0].reshape(case["rows"], D)
    cu = s["cu"].tolist()
    bwd = case["kind"] == "conv_bwd"
    w, bias = (_leaf(s["weight"]), _leaf(s["bias"])) if bwd else (s["weight"].double(), None if s["bias"] is None else s["bias"].double())
    ys, finals, dxs, dis = [], [], [], []
    for i, (lo, hi) in enumerate(zip(cu, cu[1:])):
        front = s["init"][i].double() if s["init"] is not None else torch.zeros(K, D, dtype=torch.float64, device=x.device)
        seq = torch.cat([front, x[lo:hi].double()])
        if bwd:
            seq.requires_grad_(True)
        T = hi - lo
        p = sum(w[:, k] * seq[k:k + T] for k in range(W))
        if bias is not None:
            p = p + bias
        y = _silu64(p) if case["silu"] else p
        if bwd:
            loss = (y * s["d_out"].reshape(-1, D)[lo:hi].double()).sum()
            if s["d_final"] is not None:
                loss = loss + (seq[T:] * s["d_final"][i].double()).sum()
            loss.backward()
            dxs.append(seq.grad[K:])
            dis.append(seq.grad[:K])
        else:
            ys.append(y)
            finals.append(seq[T:])
    if not bwd:
        return {"y": torch.cat(ys).reshape(s["shape"]), "final": torch.stack(finals)}
    return {"dx": torch.cat(dxs).reshape(s["shape"]), "dw": w.grad, "db": None if bias is None else bias.grad,
            "d_init": torch.stack(dis)}


def _exact_conv_step(s):
    case = s["case"]
    x = _halves(s)[0].double()
    pool = s["pool"].double()
    old = pool[s["slots"].long()]
    w = s["weight"].double()
    p = x * w[:, -1]
    for k in range(case["width"] - 1):
        p = p + old[:, k] * w[:, k]
    if s["bias"] is not None:
        p = p + s["bias"].double()
    pool[s["out_slots"].long(), :-1] = old[:, 1:]
    pool[s["out_slots"].long(), -1] = x
    return {"y": _silu64(p) if case["silu"] else p, "pool": pool}


def _token64(h, delta, u, a, b, c, skip, z):
    """One token of the definition: the new state and the output."""
    h = h * torch.exp(delta[..., None] * a) + delta[..., None] * u[..., None] * b[:, None, :]
    y = torch.einsum("bdn,bn->bd", h, c)
    if skip is not None:
        y = y + skip * u
    return h, y if z is None else y * _silu64(z)


def _delta64(x):
    return torch.where(x > 30, x, torch.log1p(torch.exp(torch.clamp(x, max=30))))


def _exact_scan_step(s):
    case = s["case"]
    d = lambda t: None if t is None else t.double()  # noqa: E731
    z = d(_halves(s)[1]) if case["z"] else None
    b, c = _bc(s)
    pool = s["pool"].double()
    h, y = _token64(pool[s["slots"].long()], _delta64(d(s["dt"]) + d(s["dt_bias"])), d(s["u"]), d(s["a"]), d(b), d(c),
                    d(s["skip"]), z)
    pool[s["out_slots"].long()] = h
    return {"y": y, "pool": pool}


def _exact_scan(s):
    """All sequences token by token together; those that have ended keep their state."""
    case = s["case"]
    R, D, N, B = case["rows"], case["dim"], case["n"], case["nseq"]
    bwd = case["kind"] == "scan_bwd"
    if bwd and s["longest"] * B * D * N * 8 * 8 > 60e9:
        return None  # more than is held of intermediate states
    z = _halves(s)[1].reshape(R, D) if case["z"] else None
    b, c = _bc(s)
    keep = _leaf if bwd else (lambda t: None if t is None else t.double())
    u, dt, bm, cm, zz = (keep(None if t is None else t.reshape(R, -1)) for t in (s["u"], s["dt"], b, c, z))
    a, skip, bias = keep(s["a"]), keep(s["skip"]), keep(s["dt_bias"])
    init = keep(s["init"] if s["init"] is not None else torch.zeros(B, D, N, device=s["a"].device))
    cu = s["cu"].tolist()
    lens = [y - x for x, y in zip(cu, cu[1:])]
    order = sorted(range(B), key=lambda i: -lens[i])                   # the longest first: those alive are a prefix
    delta = _delta64(dt + bias)
    h = init[order]
    ys, at, finals = [], [], []
    alive = B
    for t in range(s["longest"]):
        while alive and lens[order[alive - 1]] <= t:
            finals.append((order[alive - 1], h[alive - 1]))
            alive -= 1
            h = h[:alive]
        rows = [cu[i] + t for i in order[:alive]]
        idx = slice(rows[0], rows[0] + 1) if alive == 1 else torch.tensor(rows, device=u.device)
        h, y = _token64(h, delta[idx], u[idx], a, bm[idx], cm[idx], skip, None if zz is None else zz[idx])
        ys.append(y)
        at += rows
    finals += [(order[i], h[i]) for i in range(alive)]
    finals = torch.stack([f for _, f in sorted(finals, key=lambda p: p[0])])
    y = torch.empty(R, D, dtype=torch.float64, device=u.device)
    y[torch.tensor(at, device=u.device)] = torch.cat(ys).detach()
    if not bwd:
        return {"y": y.reshape(s["shape"]), "final": finals}
    weight = s["d_out"].reshape(R, D).double()[torch.tensor(at, device=u.device)]
    loss = (torch.cat(ys) * weight).sum()
    if s["d_final"] is not None:
        loss = loss + (finals * s["d_final"].double()).sum()
    loss.backward()
    shape, lead = s["shape"], s["shape"][:-1]
    return {"du": u.grad.reshape(shape), "ddt": dt.grad.reshape(shape), "da": a.grad, "db": bm.grad.reshape(*lead, N),
            "dc": cm.grad.reshape(*lead, N), "dskip": None if skip is None else skip.grad,
            "dz": None if zz is None else zz.grad.reshape(shape), "ddt_bias": bias.grad, "d_init": init.grad}


def _exact_pages(s):
    """The tables page by page on the host; the pools' values where those say."""
    case, S = s["case"], s["case"]["slots"]
    used = s["used"].tolist()
    pairs = []                                                         # (to, from or None)
    if case["kind"] == "fork":
        free = [p for p in range(S) if not used[p]]
        pairs = [(free[i], None if q == -2 else q) for i, q in enumerate(s["parents"].tolist())]
    else:
        for p in s["done"].tolist():
            used[p] = 0
        L = sum(used)
        pairs = list(zip([p for p in range(L) if not used[p]], [p for p in range(L, S) if used[p]]))
    pools = []
    for pool in s["pools"]:
        out = pool.double()
        for to, frm in pairs:
            out[to] = 0 if frm is None else pool[frm].double()
        pools.append(out)
    return {k: None for k in (("children", "used") if case["kind"] == "fork" else ("slots", "used", "moved"))} | {"pools": pools}
