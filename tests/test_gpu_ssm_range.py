"""The selective scan and the causal convolution over the rest of their documented range,
against the plain 64-bit implementations: decays above 1, long sequences and many rows,
infinities and NaN, tensors of more than 2^31 elements, malformed offsets, very many
channels.

Tolerances as in test_gpu_ssm, per element, as parts of the same sum over the
absolute values of its terms (its decays as they are, so that growth is in it).
"""
import threading

import pytest
import torch

import ssm_ref
from parity import check_bf16_rounding
from test_gpu_ssm import DT, cu_of, gla, gpu, lead, near, rnd, scan_factor, scan_inputs, strided  # noqa: F401

pytestmark = pytest.mark.gpu

ORDER = ("u", "dt", "a", "b", "c", "skip", "z", "bias")
GRADS = ("du", "ddt", "da", "db", "dc", "dskip", "dz", "dbias", "d_init")


# ---------------------------------------------------------------------------
# Decays above 1: without softplus the step size has any sign, and a has any.
# ---------------------------------------------------------------------------
def signed_inputs(lens, D, N, io, seed, softplus):
    """Exponents delta a from -3 to 3, many of them small ones on both sides of zero."""
    g = torch.Generator().manual_seed(seed)
    cu, R, B = cu_of(lens), sum(lens), len(lens)
    ty = DT[io]
    dt = 1.5 * (2 * torch.rand(R, D, generator=g) - 1)
    if max(lens) > 64:  # few large steps, so that states stay far inside fp32's range
        large = torch.rand(R, 1, generator=g) < 1 / 16
        dt = torch.where(large, dt, dt * 0.1)
    a = 2 * (2 * torch.rand(D, N, generator=g) - 1)
    a[0], a[-1] = 2.0, -2.0
    return dict(u=rnd(g, R, D, dtype=ty), dt=(dt - 1 if softplus else dt).to(ty), a=a,
                b=rnd(g, R, N, dtype=ty), c=rnd(g, R, N, dtype=ty), skip=rnd(g, D),
                z=rnd(g, R, D, dtype=ty), bias=rnd(g, D, std=0.01), init=rnd(g, B, D, N),
                dy=rnd(g, R, D, dtype=ty), df=rnd(g, B, D, N)), cu


def signed_factor(x, cu, softplus):
    """Nothing is forgotten: every step of a sequence counts.  A step: |delta a| < 3.1 costs three
    roundings of the exponent (9.3 * 2^-24), the exponential 2^-22, the product and the sum 2^-23:
    below 2^-20.  With softplus |delta a| < 2, and delta is off by up to 2^-22 (8 * 2^-24 of the
    exponent): below 2^-19.  A chunk's decay is the exponential of a sum of step sizes, off by
    2^-24 of every partial sum, each at most twice the largest from the start on."""
    d = x["dt"].double() + x["bias"].double()
    d = torch.log1p(torch.exp(d)) if softplus else d
    steps = max(q - p for p, q in zip(cu, cu[1:]))
    walk = max([float(d[p:q].cumsum(0).abs().amax(0).mul(x["a"].double().abs().amax(1)).max())
                for p, q in zip(cu, cu[1:]) if q > p])
    return steps * (2 ** -19 if softplus else 2 ** -20) + steps * 2 * walk * 2 ** -24 + 2 ** -17


@pytest.mark.parametrize("softplus", [False, True])
@pytest.mark.parametrize("lens,packed", [([20, 1, 0, 17], True), ([12, 12], False), ([400], False)])
@pytest.mark.parametrize("io,D,N", [("fp32", 40, 8), ("fp32", 136, 16), ("fp32", 24, 64), ("bf16", 72, 16),
                                    ("bf16", 40, 32)])
def test_scan_with_decays_above_one(gla, io, D, N, lens, packed, softplus):  # noqa: F811
    """Whole sequences, and (400 tokens) sequences in chunks; softplus has a > 0 only for short ones."""
    x, cu = signed_inputs(lens, D, N, io, 31, softplus)
    if softplus and max(lens) > 64:
        x["a"] = torch.where(x["a"] > 0, x["a"] * 0.05, x["a"])  # steps of one sign add up
    more = (softplus, x["init"], cu, x["dy"], x["df"])
    ref = ssm_ref.scan(*[x[k] for k in ORDER], *more)
    size = ssm_ref.scan(*[x[k] for k in ORDER], *more, absolute=True)
    L = lambda t: strided(lead(t, lens, packed))  # noqa: E731
    args = (L(x["u"]), L(x["dt"]), gpu(x["a"]), L(x["b"]), L(x["c"]))
    kw = dict(skip=gpu(x["skip"]), z=L(x["z"]), dt_bias=gpu(x["bias"]), softplus=softplus,
              init_state=gpu(x["init"]),
              cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda() if packed else None)
    f = signed_factor(x, cu, softplus)
    y, fin = gla.scan_fwd(*args, **kw, out_dtype=torch.float32)
    near(y.reshape(ref["y"].shape), ref["y"], size["y"], f, "y")
    near(fin, ref["final"], size["final"], f, "final")
    got = gla.scan_bwd(*args, gpu(lead(x["dy"], lens, packed)), **kw, d_final_state=gpu(x["df"]),
                       grad_dtype=torch.float32)
    f = 2 * f + sum(lens) * 2 ** -24
    for k, v in zip(GRADS, got):
        near(v.reshape(ref[k].shape), ref[k], size[k], f, k)
    gla.status_sync()


@pytest.mark.parametrize("softplus", [False, True])
@pytest.mark.parametrize("io,R,D,N", [("fp32", 7, 72, 8), ("fp32", 5, 136, 16), ("fp32", 6, 24, 64),
                                      ("bf16", 5, 40, 32)])
def test_scan_step_with_decays_above_one(gla, io, R, D, N, softplus):  # noqa: F811
    x, cu = signed_inputs([1] * R, D, N, io, 32, softplus)
    ref = ssm_ref.scan(*[x[k] for k in ORDER], softplus, x["init"], cu)
    size = ssm_ref.scan(*[x[k] for k in ORDER], softplus, x["init"], cu, absolute=True)
    state = gpu(x["init"]).clone()
    y = gla.scan_step(gpu(x["u"]), gpu(x["dt"]), gpu(x["a"]), gpu(x["b"]), gpu(x["c"]), state,
                      skip=gpu(x["skip"]), z=gpu(x["z"]), dt_bias=gpu(x["bias"]), softplus=softplus,
                      out_dtype=torch.float32)
    f = signed_factor(x, cu, softplus)
    near(y, ref["y"], size["y"], f, "y")
    near(state, ref["final"], size["final"], f, "state")


def test_decays_around_one_in_fp32_rows(gla):  # noqa: F811
    """One step of a state of 1 without drive is the decay itself, over exponents of both signs, 2^-26 ..
    8: below 2^-22 for the exponential and 2^-24 for each of three roundings of its argument."""
    N = 8
    e = torch.cat([s * 2.0 ** torch.linspace(-26, 3, 1024).double() for s in (1, -1)]).float()
    D = e.numel() // N
    state = torch.ones(1, D, N, device="cuda")
    one, zero = torch.ones(1, D, device="cuda"), torch.zeros(1, N, device="cuda")
    gla.scan_step(one, one, gpu(e.reshape(D, N)), zero, zero, state, softplus=False)
    want = torch.exp(e.double())
    err = (state.double().cpu().flatten() - want).abs() / want
    assert bool((err <= 2 ** -22 + 2 ** -24 + 3 * 2 ** -24 * e.double().abs()).all()), float(err.max())


# ---------------------------------------------------------------------------
# Long sequences, long chunks, many rows: every stage of the pipelines is passed.
# ---------------------------------------------------------------------------
def some(x, sel):
    """The inputs of the channels ``sel``, which are independent of the others."""
    by_row = ("u", "dt", "z", "dy")
    return {k: None if v is None else v[:, sel] if k in by_row + ("init", "df") else
            v[sel] if k in ("a", "skip", "bias") else v for k, v in x.items()}


# chunks of 224 tokens; of 80 and of 336 (no multiples of a tile's 64 tokens); packed, of 128;
# whole sequences of many tiles; 33 and 47 chunks of 64, the last one partial
@pytest.mark.parametrize("io,D,N,lens,packed", [
    ("bf16", 2048, 16, [2048], False), ("bf16", 512, 64, [700], False), ("fp32", 1024, 64, [1500], False),
    ("bf16", 2048, 16, [1100, 0, 1300], True), ("fp32", 2048, 16, [600] * 4, False),
    ("bf16", 264, 8, [2100], False), ("fp32", 40, 32, [5, 3000, 64], True)])
def test_scan_long(gla, io, D, N, lens, packed):  # noqa: F811
    x, cu = scan_inputs(lens, D, N, io, 33)
    sel = torch.cat([torch.arange(0, D, max(1, D // 12)), torch.arange(D - 4, D)]).unique()
    part = some(x, sel)
    ref = ssm_ref.scan(*[part[k] for k in ORDER], True, part["init"], cu)
    size = ssm_ref.scan(*[part[k] for k in ORDER], True, part["init"], cu, absolute=True)
    L = lambda t: strided(lead(t, lens, packed))  # noqa: E731
    args = (L(x["u"]), L(x["dt"]), gpu(x["a"]), L(x["b"]), L(x["c"]))
    kw = dict(skip=gpu(x["skip"]), z=L(x["z"]), dt_bias=gpu(x["bias"]), init_state=gpu(x["init"]),
              cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda() if packed else None)
    f = scan_factor(x, cu, True)
    y, fin = gla.scan_fwd(*args, **kw, out_dtype=torch.float32)
    near(y.reshape(-1, D)[:, sel], ref["y"], size["y"], f, "y")
    near(fin[:, sel], ref["final"], size["final"], f, "final")
    if io == "bf16":
        y16, fin16 = gla.scan_fwd(*args, **kw)
        check_bf16_rounding(y16, y)
        assert torch.equal(fin16, fin)
    gla.status_sync()


# 33 chunks; 18 and 47 chunks beside an empty sequence; every channel, since db and dc sum over them
@pytest.mark.parametrize("io,D,N,lens,packed", [
    ("fp32", 40, 8, [2100], False), ("bf16", 72, 16, [1100, 0, 3000, 1], True), ("bf16", 24, 64, [1200, 1200], False),
    ("fp32", 136, 32, [1500], False)])
def test_scan_gradients_long(gla, io, D, N, lens, packed):  # noqa: F811
    x, cu = scan_inputs(lens, D, N, io, 34)
    more = (True, x["init"], cu, x["dy"], x["df"])
    ref = ssm_ref.scan(*[x[k] for k in ORDER], *more)
    size = ssm_ref.scan(*[x[k] for k in ORDER], *more, absolute=True)
    L = lambda t: strided(lead(t, lens, packed))  # noqa: E731
    got = gla.scan_bwd(L(x["u"]), L(x["dt"]), gpu(x["a"]), L(x["b"]), L(x["c"]),
                       gpu(lead(x["dy"], lens, packed)), skip=gpu(x["skip"]), z=L(x["z"]),
                       dt_bias=gpu(x["bias"]), init_state=gpu(x["init"]), d_final_state=gpu(x["df"]),
                       cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda() if packed else None,
                       grad_dtype=torch.float32)
    f = scan_factor(x, cu, True, gradients=True) + sum(lens) * 2 ** -24
    for k, v in zip(GRADS, got):
        near(v.reshape(ref[k].shape), ref[k], size[k], f, k)
    gla.status_sync()


def step_check(gla, x, R, io, slots, outs, pool):  # noqa: F811
    """One scan step over a pool against the formula in 64 bits, on the GPU (some inputs are large)."""
    before = pool.clone()
    out = torch.full((R, x["u"].shape[1]), 7.0, device="cuda")
    gla.scan_step(x["u"], x["dt"], x["a"], x["b"], x["c"], pool, skip=x["skip"], z=x["z"],
                  dt_bias=x["bias"], slots=slots, out_slots=outs, out=out)
    gla.status_sync()
    live = (slots >= 0) & (outs >= 0)
    assert bool((out[~live] == 7.0).all())
    untouched = torch.ones(pool.shape[0], dtype=torch.bool, device="cuda")
    untouched[outs[live].long()] = False
    assert torch.equal(pool[untouched], before[untouched])
    D64 = {k: v.double() for k, v in x.items()}
    delta = torch.nn.functional.softplus(D64["dt"] + D64["bias"], threshold=60)[live]
    u, z = D64["u"][live], D64["z"][live]
    old, b, c = before[slots[live].long()].double(), D64["b"][live][:, None], D64["c"][live][:, None]
    del before
    kept, drive = torch.exp(delta[..., None] * D64["a"]) * old, (delta * u)[..., None] * b
    gate = z * torch.sigmoid(z)
    h, h_size = kept + drive, kept.abs() + drive.abs()
    y = ((h * c).sum(-1) + D64["skip"] * u) * gate
    y_size = ((h_size * c.abs()).sum(-1) + (D64["skip"] * u).abs()) * gate.abs()
    f = 2 ** -20 + 2 ** -17
    assert bool(((pool[outs[live].long()].double() - h).abs() <= f * h_size + 1e-30).all())
    assert bool(((out[live].double() - y).abs() <= f * y_size + 1e-30).all())


@pytest.mark.parametrize("io,R,D,N", [
    ("bf16", 573, 2048, 8), ("fp32", 291, 2048, 16), ("bf16", 71, 2432, 64), ("fp32", 67, 2424, 64),
    ("bf16", 1001, 1032, 32)])
def test_scan_step_of_many_rows(gla, io, R, D, N):  # noqa: F811
    """Blocks that walk five groups of rows and more, the last one partial, rows without a page among them."""
    x, _ = scan_inputs([1] * R, D, N, io, 35)
    x = {k: gpu(v) for k, v in x.items() if k not in ("init", "dy", "df")}
    g = torch.Generator().manual_seed(36)
    order = torch.randperm(2 * R + 1, generator=g).to(torch.int32)
    slots, outs = gpu(order[:R].clone()), gpu(order[R:2 * R].clone())
    slots[[0, 5, R // 2, R - 1]] = -1
    outs[[6, R // 3]] = -1
    pool = torch.randn(2 * R + 1, D, N, generator=torch.Generator(device="cuda").manual_seed(37), device="cuda")
    step_check(gla, x, R, io, slots, outs, pool)


def test_scan_step_of_more_rows_than_tables_hold(gla):  # noqa: F811
    """More blocks than two waves, because a block's table of pages holds 1024 rows."""
    R, D, N = 940_003, 8, 8
    x, _ = scan_inputs([1] * R, D, N, "bf16", 38)
    x = {k: gpu(v) for k, v in x.items() if k not in ("init", "dy", "df")}
    slots = torch.arange(R, dtype=torch.int32, device="cuda")
    slots[::1000] = -1
    pool = torch.randn(R, D, N, generator=torch.Generator(device="cuda").manual_seed(39), device="cuda")
    step_check(gla, x, R, "bf16", slots, slots.clone(), pool)


def test_conv_step_of_many_rows(gla):  # noqa: F811
    """More rows than one grid dimension is given, some without a page, against the formula in 64 bits."""
    R, D, W = 100_003, 16, 3
    g = torch.Generator(device="cuda").manual_seed(54)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, w, bias, pool = r(R, D), r(D, W), r(D), r(2 * R, W - 1, D)
    order = torch.randperm(2 * R, generator=g, device="cuda").to(torch.int32)
    slots, outs = order[:R].clone(), order[R:].clone()
    slots[::777] = -1
    outs[5::1000] = -1
    before, out = pool.clone(), torch.full((R, D), 7.0, device="cuda")
    gla.conv_step(x, w, pool, bias, slots=slots, out_slots=outs, out=out)
    gla.status_sync()
    live = (slots >= 0) & (outs >= 0)
    window = torch.cat([before[slots[live].long()], x[live][:, None]], 1)
    terms = window.double() * w.double().t()
    size = terms.abs().sum(1) + bias.abs()
    assert bool(((out[live].double() - terms.sum(1) - bias).abs() <= 2 ** -18 * size).all())
    assert bool((out[~live] == 7.0).all())
    want = before
    want[outs[live].long()] = window[:, 1:]
    assert torch.equal(pool, want)


# ---------------------------------------------------------------------------
# Infinities and NaN stay in their sequence, rows and channels.
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_other_sequences_of_a_poisoned_one(gla, io, bad):  # noqa: F811
    """A packed sequence full of ``bad`` changes no bit of its neighbours' results."""
    lens, D, N, W = [37, 0, 70, 1, 129, 33], 136, 16, 4
    x, cu = scan_inputs(lens, D, N, io, 40)
    x = {k: gpu(v) for k, v in x.items()}
    w, wb = torch.randn(D, W, device="cuda"), torch.randn(D, device="cuda")
    ci = torch.randn(len(lens), W - 1, D, device="cuda").to(DT[io])
    cu_gpu = torch.tensor(cu, dtype=torch.int32).cuda()

    def everything():
        y, f = gla.conv_fwd(x["u"], w, wb, init_state=ci, cu_seqlens=cu_gpu, activation="silu")
        dx, _, _, di = gla.conv_bwd(x["u"], w, x["dy"], wb, init_state=ci, d_final_state=ci.float(),
                                    cu_seqlens=cu_gpu, activation="silu")
        args = (x["u"], x["dt"], x["a"], x["b"], x["c"])
        kw = dict(skip=x["skip"], z=x["z"], dt_bias=x["bias"], init_state=x["init"], cu_seqlens=cu_gpu)
        o, h = gla.scan_fwd(*args, **kw)
        du, ddt, _, db, dc, _, dz, _, dh = gla.scan_bwd(*args, x["dy"], **kw, d_final_state=x["df"])
        return [y, dx, o, du, ddt, db, dc, dz], [f, di, h, dh]

    rows, states = everything()
    s = 2
    for k in ("u", "dt", "b", "c", "z", "dy"):
        x[k][cu[s]:cu[s + 1]] = bad
    x["init"][s], x["df"][s], ci[s] = bad, bad, bad
    rows2, states2 = everything()
    gla.status_sync()
    keep = torch.ones(cu[-1], dtype=torch.bool)
    keep[cu[s]:cu[s + 1]] = False
    others = [i for i in range(len(lens)) if i != s]
    for p, q in zip(rows, rows2):
        assert torch.equal(p[keep.cuda()], q[keep.cuda()])
    for p, q in zip(states, states2):
        assert torch.equal(p[others], q[others])


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_other_rows_of_a_poisoned_one_in_steps(gla, io):  # noqa: F811
    R, D, N, W = 9, 136, 16, 4
    x, _ = scan_inputs([1] * R, D, N, io, 41)
    x = {k: gpu(v) for k, v in x.items()}
    w, cs = torch.randn(D, W, device="cuda"), torch.randn(R, W - 1, D, device="cuda").to(DT[io])

    def everything():
        h, c = x["init"].clone(), cs.clone()
        y = gla.scan_step(x["u"], x["dt"], x["a"], x["b"], x["c"], h, skip=x["skip"], z=x["z"], dt_bias=x["bias"])
        return [y, h, gla.conv_step(x["u"], w, c, activation="silu"), c]

    first = everything()
    for k in ("u", "dt", "b", "c", "z"):
        x[k][3] = float("nan")
    others = [i for i in range(R) if i != 3]
    assert all(torch.equal(p[others], q[others]) for p, q in zip(first, everything()))


# ---------------------------------------------------------------------------
# More than 2^31 elements
# ---------------------------------------------------------------------------
def test_prompts_of_more_than_31_bits(gla):  # noqa: F811
    """Packed bf16 rows of 2^31 and some elements: the last sequences, which start behind
    element 2^31, are those of a call on them alone (convolution: bit for bit) and the
    definition's (scan: some channels)."""
    D, N, W, tail = 2048, 16, 4, [70, 0, 1, 33]
    head = 2 ** 31 // D + 7
    g = torch.Generator(device="cuda").manual_seed(42)
    lens = [head] + tail
    R, B, T = sum(lens), len(lens), sum(tail)
    cu = torch.tensor(cu_of(lens), dtype=torch.int32, device="cuda")
    cu_tail = torch.tensor(cu_of([0] + tail), dtype=torch.int32, device="cuda")
    x = torch.empty(R, D, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    w = torch.randn(D, W, generator=g, device="cuda")
    init = torch.randn(B, W - 1, D, generator=g, device="cuda").to(torch.bfloat16)
    y, f = gla.conv_fwd(x, w, init_state=init, cu_seqlens=cu, activation="silu")
    y2, f2 = gla.conv_fwd(x[head:], w, init_state=init, cu_seqlens=cu_tail, activation="silu")
    assert torch.equal(y[head:], y2) and torch.equal(f[1:], f2[1:])
    dx, _, _, di = gla.conv_bwd(x, w, y, init_state=init, cu_seqlens=cu, activation="silu")
    dx2, _, _, di2 = gla.conv_bwd(x[head:], w, y2, init_state=init, cu_seqlens=cu_tail, activation="silu")
    assert torch.equal(dx[head:], dx2) and torch.equal(di[1:], di2[1:])
    gla.status_sync()
    del dx
    a = -torch.arange(1, N + 1, device="cuda").float() * torch.rand(D, 1, generator=g, device="cuda").add(0.5)
    dt = torch.empty(R, D, dtype=torch.bfloat16, device="cuda").normal_(-3, 0.5, generator=g)
    bc = torch.randn(R, 2 * N, generator=g, device="cuda").to(torch.bfloat16)
    b, c = bc[:, :N], bc[:, N:]
    o, h = gla.scan_fwd(y, dt, a, b, c, z=x, cu_seqlens=cu, out_dtype=torch.float32)
    sel = torch.tensor([0, 1, 1000, 2047], device="cuda")
    cl = cu_of([0] + tail)
    ins = (y[head:][:, sel], dt[head:][:, sel], a[sel], b[head:], c[head:], None, x[head:][:, sel], None, True, None, cl)
    names = dict(zip(ORDER, ins))
    factor = scan_factor({k: None if v is None else v.cpu() for k, v in names.items()}, cl, True)
    ref, size = ssm_ref.scan(*ins), ssm_ref.scan(*ins, absolute=True)
    near(o[head:][:, sel], ref["y"], size["y"], factor, "y")
    near(h[1:, sel], ref["final"][1:], size["final"][1:], factor, "final")
    gla.status_sync()
    del o
    dy = x
    got = gla.scan_bwd(y, dt, a, b, c, dy, z=x, cu_seqlens=cu)
    alone = gla.scan_bwd(y[head:], dt[head:], a, b[head:], c[head:], dy[head:], z=x[head:], cu_seqlens=cu_tail)
    for k, p, q in zip(GRADS, got, alone):
        if p is not None and p.shape[0] == R:
            assert torch.equal(p[head:], q) and q.shape[0] == T, k
    assert torch.equal(got[8][1:], alone[8][1:])
    gla.status_sync()


def test_pools_of_more_than_31_bits(gla):  # noqa: F811
    """Pages behind element 2^31 of a pool step as pages of a small one."""
    D, N, W, R = 2048, 16, 4, 3
    P = 2 ** 31 // (D * N) + 9
    x, _ = scan_inputs([1] * R, D, N, "bf16", 43)
    x = {k: gpu(v) for k, v in x.items()}
    slots = torch.tensor([P - 1, P - 3, 5], dtype=torch.int32, device="cuda")
    outs = torch.tensor([P - 1, P - 2, P - 5], dtype=torch.int32, device="cuda")
    pool = torch.zeros(P, D, N, device="cuda")
    pool[slots.long()] = x["init"]
    state = x["init"].clone()
    args = (x["u"], x["dt"], x["a"], x["b"], x["c"])
    y = gla.scan_step(*args, pool, dt_bias=x["bias"], slots=slots, out_slots=outs)
    assert torch.equal(y, gla.scan_step(*args, state, dt_bias=x["bias"]))
    assert torch.equal(pool[outs.long()], state)
    del pool
    P = 2 ** 31 // (D * (W - 1)) + 9
    w, cs = torch.randn(D, W, device="cuda"), torch.randn(R, W - 1, D, device="cuda").to(torch.bfloat16)
    pool = torch.zeros(P, W - 1, D, dtype=torch.bfloat16, device="cuda")
    slots, outs = slots.clone(), outs.clone()
    slots[:2], outs[:] = torch.tensor([P - 1, P - 3]), torch.tensor([P - 1, P - 2, P - 5])
    pool[slots.long()] = cs
    y = gla.conv_step(x["u"], w, pool, slots=slots, out_slots=outs)
    assert torch.equal(y, gla.conv_step(x["u"], w, cs))
    assert torch.equal(pool[outs.long()], cs)
    gla.status_sync()


# ---------------------------------------------------------------------------
# Malformed offsets are reported whatever else is asked for.
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("D", [8, 64, 2048])
@pytest.mark.parametrize("states", [False, True])
def test_malformed_offsets_of_convolutions(gla, D, states):  # noqa: F811
    """A start before or behind the first row, an end outside, decreasing ones next to a run's border
    and far down a long table; also without the outputs that belong to sequences, which
    have blocks of their own."""
    R = 64
    x = torch.randn(R, D, device="cuda").to(torch.bfloat16)
    w = torch.ones(D, 4, device="cuda")
    many = [min(i // 4, R) for i in range(301)]     # 300 sequences, most of one row or none
    many[-1] = R
    calls = (lambda c: gla.conv_fwd(x, w, cu_seqlens=c, output_final_state=states),
             lambda c: gla.conv_bwd(x, w, x, cu_seqlens=c, need_d_init=states))
    bad = [[0, 70, 64], [3, 20, 64], [0, 20, 60], [0, 40, 20, 64], [0, -5, 64], [0, -5, 70], [-1, 64], [-3, 0, 64],
           [0, 33, 32, 64], [0, 0, -1, 0, 64], [0, 2 ** 31 - 1, 64], [0, -2 ** 31, 64],
           many[:250] + [many[250] - 2] + many[251:], many[:-2] + [R + 1, R], [-1] + many[1:]]
    for cu in bad:
        c = torch.tensor(cu, dtype=torch.int32, device="cuda")
        for call in calls:
            call(c)
            with pytest.raises(gla.GlaError) as e:
                gla.status_sync()
            assert e.value.status == 1, cu
    for cu in ([0, 64], [0, 0, 64, 64], many):
        for call in calls:
            call(torch.tensor(cu, dtype=torch.int32, device="cuda"))
    gla.status_sync()


# ---------------------------------------------------------------------------
# Very many channels
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("io,D", [("bf16", 65535 * 128 + 8), ("bf16", 2 ** 24), ("fp32", 2 ** 24)])
def test_conv_of_very_many_channels(gla, io, D):  # noqa: F811
    """Up to the documented 2^24, forwards and backwards: more tiles of channels than a grid
    dimension holds.  All channels against the formula in 64 bits, on the GPU."""
    T, W = 3, 2
    g = torch.Generator(device="cuda").manual_seed(44)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, dy, w, bias = r(1, T, D).to(DT[io]), r(1, T, D).to(DT[io]), r(D, W), r(D)
    y, fin = gla.conv_fwd(x, w, bias, out_dtype=torch.float32)
    dx, dw, db, di = gla.conv_bwd(x, w, dy, bias, grad_dtype=torch.float32)
    gla.status_sync()
    x, dy, w = x[0].double(), dy[0].double(), w.double()
    back = torch.cat([torch.zeros_like(x[:1]), x[:-1]])
    after = torch.cat([dy[1:], torch.zeros_like(dy[:1])])
    zero = torch.zeros_like(x[0])

    def same(got, terms):
        """W + 1 products and sums at most: below 2^-18 of their absolute values."""
        size = sum(t.abs() for t in terms)
        assert bool(((got.double() - sum(terms)).abs() <= 2 ** -18 * size).all())

    same(y[0], [w[:, 1] * x, w[:, 0] * back, bias.double().expand_as(x)])
    assert torch.equal(fin[0, 0].double(), x[-1])
    same(dx[0], [w[:, 1] * dy, w[:, 0] * after])
    same(di[0, 0], [w[:, 0] * dy[0], zero])
    same(dw[:, 1], list(dy * x))
    same(dw[:, 0], list(dy * back))
    same(db, list(dy))


def test_scan_of_very_many_channels(gla):  # noqa: F811
    """2^24 channels of two tokens, prompt, gradients and step, against the formula in 64 bits on the GPU."""
    D, N = 2 ** 24, 8
    g = torch.Generator(device="cuda").manual_seed(45)
    r = lambda *s, std=1.0: torch.randn(*s, generator=g, device="cuda") * std  # noqa: E731
    u, dt, dy = (r(1, 2, D, std=s).to(torch.bfloat16) for s in (1.0, 0.5, 1.0))
    b, c = r(1, 2, N).to(torch.bfloat16), r(1, 2, N).to(torch.bfloat16)
    a = -torch.rand(D, N, generator=g, device="cuda") - 0.1
    init = r(1, D, N)
    y, fin = gla.scan_fwd(u, dt, a, b, c, init_state=init, out_dtype=torch.float32)
    got = gla.scan_bwd(u, dt, a, b, c, dy, init_state=init, grad_dtype=torch.float32)
    state = init.clone()
    y0 = gla.scan_step(u[:, 0], dt[:, 0], a, b[:, 0], c[:, 0], state, out_dtype=torch.float32)
    gla.status_sync()
    for lo in range(0, D, 2 ** 22):                             # (64-bit states of 2^22 channels are 256 MB)
        at = slice(lo, lo + 2 ** 22)
        U, X, G, A, H = u[0, :, at].double(), dt[0, :, at].double(), dy[0, :, at].double(), a[at].double(), \
            init[0, at].double()
        B, C = b[0].double(), c[0].double()
        delta = torch.nn.functional.softplus(X, threshold=60)
        decay = torch.exp(delta[..., None] * A)
        h = [H]
        size = H.abs()
        sizes = []
        for t in range(2):
            drive = (delta[t] * U[t])[:, None] * B[t]
            h.append(decay[t] * h[-1] + drive)
            size = decay[t] * size + drive.abs()
            sizes.append(size)
        f = 2 ** -17 + 2 * 2 ** -20
        ok = lambda p, q, s, f=f: bool(((p.double() - q).abs() <= f * s + 1e-30).all())  # noqa: E731
        for t in range(2):
            assert ok(y[0, t, at], (h[t + 1] * C[t]).sum(-1), (sizes[t] * C[t].abs()).sum(-1))
        assert ok(fin[0, at], h[2], sizes[1])
        assert ok(state[0, at], h[1], sizes[0]) and ok(y0[0, at], (h[1] * C[0]).sum(-1), (sizes[0] * C[0].abs()).sum(-1))
        e1 = G[1][:, None] * C[1]
        e0 = G[0][:, None] * C[0] + decay[1] * e1
        e0s = (G[0][:, None] * C[0]).abs() + decay[1] * e1.abs()
        du, ddt, da, _, _, _, _, _, di = got
        assert ok(di[0, at], decay[0] * e0, decay[0] * e0s, 2 * f)
        for t, (e, es) in enumerate(((e0, e0s), (e1, e1.abs()))):
            s1, s1s = (e * B[t]).sum(-1), (es * B[t].abs()).sum(-1)
            before, bs = (h[t], H.abs() if t == 0 else sizes[0])
            w, ws = e * decay[t] * before, es * decay[t] * bs
            slope = torch.sigmoid(X[t])
            assert ok(du[0, t, at], delta[t] * s1, delta[t] * s1s, 2 * f)
            assert ok(ddt[0, t, at], ((w * A).sum(-1) + U[t] * s1) * slope,
                      ((ws * A.abs()).sum(-1) + U[t].abs() * s1s) * slope, 2 * f)
            part, part_s = (w * delta[t][:, None], ws * delta[t][:, None]) if t == 0 else \
                (part + w * delta[t][:, None], part_s + ws * delta[t][:, None])
        assert ok(da[at], part, part_s, 2 * f)


# ---------------------------------------------------------------------------
# Every built variant of the convolutions over hundreds of ends of sequences, again and again
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("io,out", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")])
def test_convolution_variants_at_sequence_ends(gla, io, out, act, W):  # noqa: F811
    """A build of an earlier kernel, right by its source, let the address of the next sequence's offset into
    the registers of a sequence's last row before they were stored, in some blocks of some
    runs.  So every variant runs over many ends with the GPU full, six times, to the same
    bits, and all rows are compared with the formula in fp32 (each side within 2^-18 of the
    terms, gradients 2^-17, as in test_gpu_ssm; then one rounding of the result)."""
    D, K = 2048, W - 1
    g = torch.Generator(device="cuda").manual_seed(46)
    lens = torch.randint(0, 120, (300,), generator=torch.Generator().manual_seed(47)).tolist()
    cu, R, B = cu_of(lens), sum(lens), len(lens)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, dy = r(R, D).to(DT[io]), r(R, D).to(DT[io])
    w, bias, init = r(D, W) * 0.5, r(D), r(B, K, D).to(DT[io])
    df = r(B, K, D)
    cu_gpu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    kw = dict(init_state=init, cu_seqlens=cu_gpu, activation=act)

    def everything():
        y, fin = gla.conv_fwd(x, w, bias, **kw, out_dtype=DT[out])
        return [y, fin, *gla.conv_bwd(x, w, dy, bias, **kw, d_final_state=df, grad_dtype=DT[out])]

    first = everything()
    for _ in range(5):
        assert all(torch.equal(p, q) for p, q in zip(first, everything()))
    gla.status_sync()
    # rows of the initial states in front of them all; row i of a window lies K - i rows back
    rows = torch.cat([init.reshape(B * K, D), x]).float()
    seq = torch.arange(B, device="cuda").repeat_interleave(torch.tensor(lens, device="cuda"))
    at = torch.arange(R, device="cuda")
    start = cu_gpu.long()
    pos, left = at - start[seq], start[seq + 1] - at

    def back(j):
        return torch.where(pos >= j, B * K + at - j, seq * K + K + pos - j)

    p, size = bias.expand(R, D).clone(), bias.abs().expand(R, D).clone()
    for j in range(W):
        t = rows[back(j)] * w[:, K - j]
        p += t
        size += t.abs()
    s = torch.sigmoid(p)
    y = p * s if act else p
    half = torch.finfo(DT[out]).eps / 2
    err = (first[0].float() - y).abs()
    assert bool((err <= 2 * 2 ** -18 * size + half * y.abs()).all())
    dp = dy.float() * (s * (1 + p * (1 - s)) if act else 1)
    # silu' moves with p by at most a half
    dp_size = dy.float().abs() * (((s * (1 + p * (1 - s))).abs() + size) if act else 1)
    del p, s, y, err, size
    dx, dx_size = torch.zeros(R, D, device="cuda"), torch.zeros(R, D, device="cuda")
    for j in range(W):
        ok = (left > j)[:, None]
        src = torch.where(left > j, at + j, at)
        dx += torch.where(ok, dp[src] * w[:, K - j], 0.0)
        dx_size += torch.where(ok, dp_size[src] * w[:, K - j].abs(), 0.0)
    last = left <= K
    extra = torch.where(last[:, None], df[seq, (K - left).clamp(min=0)], 0.0)
    dx += extra
    dx_size += extra.abs()
    assert bool(((first[2].float() - dx).abs() <= 2 * 2 ** -17 * dx_size + half * dx.abs()).all())


# ---------------------------------------------------------------------------
# Nothing to do, and as many sequences as can be counted
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("packed", [False, True])
def test_sequences_without_tokens(gla, io, packed):  # noqa: F811
    """Three sequences of no tokens: final states are the initial ones (or zero), the initial states'
    gradients the final ones', parameters' gradients zero, in place and onto used memory."""
    D, N, W, B = 136, 16, 4, 3
    ty = DT[io]
    g = torch.Generator(device="cuda").manual_seed(48)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    none = lambda n: torch.empty(*((0, n) if packed else (B, 0, n)), dtype=ty, device="cuda")  # noqa: E731
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda") if packed else None
    w, bias, ci, df = r(D, W), r(D), r(B, W - 1, D).to(ty), r(B, W - 1, D)
    a, h, dh, p = -r(D, N).abs(), r(B, D, N), r(B, D, N), r(D)
    for init in (ci, None):
        y, f = gla.conv_fwd(none(D), w, bias, init_state=init, cu_seqlens=cu)
        assert y.numel() == 0 and torch.equal(f, ci if init is not None else torch.zeros_like(ci))
    state = ci.clone()
    gla.conv_fwd(none(D), w, bias, init_state=state, final_state=state, cu_seqlens=cu)
    assert torch.equal(state, ci)
    dx, dw, db, di = gla.conv_bwd(none(D), w, none(D), bias, init_state=ci, d_final_state=df, cu_seqlens=cu)
    assert torch.equal(di, df) and not dw.any() and not db.any() and dx.shape == none(D).shape
    args = (none(D), none(D), a, none(N), none(N))
    for init in (h, None):
        y, f = gla.scan_fwd(*args, init_state=init, cu_seqlens=cu)
        assert y.numel() == 0 and torch.equal(f, h if init is not None else torch.zeros_like(h))
    got = dict(zip(GRADS, gla.scan_bwd(*args, none(D), skip=p, z=none(D), dt_bias=p, init_state=h,
                                       d_final_state=dh, cu_seqlens=cu)))
    assert torch.equal(got["d_init"], dh) and not got["da"].any() and not got["dskip"].any() and \
        not got["dbias"].any() and got["db"].numel() == 0
    if not packed:  # and no sequences at all
        x = torch.empty(0, 5, D, dtype=ty, device="cuda")
        bc = torch.empty(0, 5, N, dtype=ty, device="cuda")
        assert gla.conv_fwd(x, w)[0].shape == x.shape and gla.scan_fwd(x, x, a, bc, bc)[1].shape == (0, D, N)
        assert not gla.conv_bwd(x, w, x)[1].any() and not gla.scan_bwd(x, x, a, bc, bc, x)[2].any()
    gla.status_sync()


def test_most_sequences(gla):  # noqa: F811
    """2^31 - 2 sequences, all empty but the last, which has one token: a block each, and one for the row."""
    B, D = 2 ** 31 - 2, 8
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    cu[B] = 1
    x = torch.arange(D, device="cuda").to(torch.bfloat16)[None] + 1
    final = torch.full((B, 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
    y, _ = gla.conv_fwd(x, torch.ones(D, 2, device="cuda"), cu_seqlens=cu, final_state=final)
    gla.status_sync()
    assert torch.equal(y, x) and torch.equal(final[B - 1], x)
    for lo in range(0, B - 1, 2 ** 28):
        assert not final[lo:min(lo + 2 ** 28, B - 1)].any()


# ---------------------------------------------------------------------------
# Chains of launches captured, and calls at the same time
# ---------------------------------------------------------------------------
def chain_inputs(seed, R=3001, D=1032, N=16, W=4, n=5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std)  # noqa: E731
    bf = torch.bfloat16
    cut = sorted(torch.randint(0, R, (n - 1,), generator=torch.Generator().manual_seed(seed)).tolist())
    return dict(x=r(R, D).to(bf), dt=(r(R, D, std=0.5) - 3).to(bf), bc=r(R, 2 * N).to(bf), z=r(R, D).to(bf),
                dy=r(R, D).to(bf), a=-r(D, N).abs() - 0.1, h=r(n, D, N), w=r(D, W), ci=r(n, W - 1, D).to(bf),
                skip=r(D), cu=torch.tensor([0] + cut + [R], dtype=torch.int32, device="cuda"),
                parents=torch.randint(0, 8, (n,), generator=g, device="cuda").to(torch.int32),
                used=(torch.arange(24, device="cuda") < 8).to(torch.int32), pool=r(24, D, N), tail=r(24, W - 1, D).to(bf))


def chain(gla, t, stream=None):  # noqa: F811
    """Every operator that takes more than one launch, the pools' pages and the steps on them."""
    N, kw = t["a"].shape[1], dict(cu_seqlens=t["cu"], stream=stream)
    u, cf = gla.conv_fwd(t["x"], t["w"], init_state=t["ci"], activation="silu", **kw)
    args = (u, t["dt"], t["a"], t["bc"][:, :N], t["bc"][:, N:])
    y, h = gla.scan_fwd(*args, skip=t["skip"], z=t["z"], init_state=t["h"], **kw)
    g = gla.scan_bwd(*args, t["dy"], skip=t["skip"], z=t["z"], init_state=t["h"], d_final_state=t["h"], **kw)
    dx = gla.conv_bwd(t["x"], t["w"], g[0], init_state=t["ci"], activation="silu", **kw)
    pools = [t["pool"], t["tail"]]
    kids, used = gla.fork_pages(pools, t["used"], t["parents"], used_out=torch.empty_like(t["used"]), stream=stream)
    n = kids.shape[0]
    v = gla.conv_step(t["x"][:n], t["w"], t["tail"], activation="silu", slots=kids, stream=stream)
    o = gla.scan_step(v, *(q[:n] for q in args[1:2]), t["a"], args[3][:n], args[4][:n], t["pool"], slots=kids, stream=stream)
    slots, left, moved = gla.compact_pages(pools, used, kids, used_out=torch.empty_like(used), stream=stream)
    return [p for p in (u, cf, y, h, *g, *dx, kids, used, v, o, slots, left, moved) if p is not None]


def test_chains_captured_and_replayed(gla):  # noqa: F811
    """Chunked scans, gradients, forks, steps and compaction as one graph, replayed on new inputs (the pools
    go back to what they were between runs)."""
    t, other = chain_inputs(49), chain_inputs(50)
    keep = {k: t[k].clone() for k in ("pool", "tail")}
    warm = chain(gla, t)
    torch.cuda.synchronize()
    for k, v in keep.items():
        t[k].copy_(v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = chain(gla, t)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(warm, held))
    for k in t:
        t[k].copy_(other[k])
    graph.replay()
    fresh = chain(gla, other)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(held, fresh))
    assert torch.equal(t["pool"], other["pool"]) and torch.equal(t["tail"], other["tail"])
    gla.status_sync()


def test_calls_at_the_same_time(gla):  # noqa: F811
    """The same chains from three threads on three streams, over and over, against each alone."""
    inputs = [chain_inputs(s) for s in (51, 52, 53)]
    saved = [{k: t[k].clone() for k in ("pool", "tail")} for t in inputs]
    alone = [chain(gla, t) for t in inputs]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            stream, t = torch.cuda.Stream(), inputs[i]
            with torch.cuda.stream(stream):
                for _ in range(8):
                    for k, v in saved[i].items():
                        t[k].copy_(v)
                    got = chain(gla, t, stream if i else None)
                    if not all(torch.equal(p, q) for p, q in zip(got, alone[i])):
                        wrong.append(i)
        except Exception as e:  # noqa: BLE001
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    gla.status_sync()
    assert not wrong
