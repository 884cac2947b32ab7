"""The gated linear recurrence, the norms between blocks and the projections on the GPU over the
ends of their ranges, against the plain 64-bit implementations (tests/block_ref.py).

Tolerances as in test_gpu_block.py; what a test adds to them is derived in it.
"""
import pytest
import torch

import block_ref
import test_gpu_block as base
from parity import check_bf16_rounding
from test_gpu_block import DT, F32, gla, gpu, near, recur_inputs, rnd  # noqa: F401

pytestmark = pytest.mark.gpu

INF = float("inf")


def bf16_values(lo, hi):
    """Every bf16 number of [lo, hi]."""
    v = torch.arange(-(1 << 15), 1 << 15, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    v = v[(v.float() >= lo) & (v.float() <= hi)].float().sort().values
    return v[torch.cat([torch.ones(1, dtype=torch.bool), v[1:] != v[:-1]])]


def room_for(gigabytes):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < (gigabytes + 8) << 30:
        pytest.skip(f"needs {gigabytes} GB of free GPU memory")


# ---------------------------------------------------------------- recurrence
def gates_over(values, T, io, i, z, decay, seed):
    """Inputs [T, D] whose gates run through the values, every channel through others."""
    g = torch.Generator().manual_seed(seed)
    D = (len(values) + 7) // 8 * 8
    at = torch.arange(D) % len(values)
    roll = lambda k: torch.stack([values[(at + (7 * t + k) % len(values)) % len(values)]  # noqa: E731
                                  for t in range(T)]).to(DT[io])
    return dict(x=rnd(g, T, D, dtype=DT[io]), f=roll(0), decay=-torch.rand(D, generator=g) if decay else None,
                i=roll(3) if i else None, z=roll(5) if z else None, init=rnd(g, 1, D),
                dy=rnd(g, T, D, dtype=DT[io]), df=rnd(g, 1, D))


def gate_gradients(x, unit):
    """df and di with their sizes from the formulas e (a h - k s(i) x) times the slope of log a, and
    e m x s(i) s(-i): automatic differentiation forms 1 - a and 1 - s by subtractions that leave 0 of
    a gate beyond 37."""
    v = {n: None if t is None else t.double() for n, t in x.items()}
    la, a, m, _, k = block_ref.decays(v["f"], v["decay"], unit)
    s = lambda t: 1 / (1 + torch.exp(-t))  # noqa: E731
    one = torch.ones_like(a)
    si, ni = (one, one) if v["i"] is None else (s(v["i"]), s(-v["i"]))
    gate = one if v["z"] is None else block_ref.silu(v["z"])
    w = s(-v["f"]) * (1 if v["decay"] is None else la)

    def both(sign):  # the values, or with absolute values of all terms the sizes
        sx, dy, g, wt = si * sign(v["x"]), sign(v["dy"]), sign(gate), sign(w)
        h, e, before = sign(v["init"][0]), sign(v["df"][0]), []
        df, di = torch.empty_like(a), torch.empty_like(a)
        for t in range(len(a)):
            before.append(h)
            h = a[t] * h + m[t] * sx[t]
        for t in reversed(range(len(a))):
            e = dy[t] * g[t] + e
            kx = k[t] * sx[t]
            df[t] = e * (a[t] * before[t] + (kx if sign is torch.abs else -kx)) * wt[t]
            di[t] = e * m[t] * sx[t] * ni[t]
            e = a[t] * e
        return df, di

    (df, di), (dfs, dis) = both(lambda t: t), both(torch.abs)
    return dict(df=(df, dfs), di=(di, dis))


def check_gates(gla, x, unit, io):
    """Prompt, gradients and single tokens.  A gate of size v adds the rounding of its exponential's
    argument, |v| 2^-24, to a sigmoid's error (bf16 rows): at most 100 2^-24 < 2^-17, in
    each of the sigmoids of a product: of f twice (a and 1 - a, or log a and 1 - s(f)), of i and z."""
    T, D = x["x"].shape
    ref = block_ref.recur_all(x["x"], x["f"], x["decay"], x["i"], x["z"], unit, x["init"], [0, T],
                              x["dy"], x["df"])
    for n, pair in gate_gradients(x, unit).items():
        ref[n] = ref[n] and pair
    tol = 2 * (ref["memory"] * 2 ** -22 + 2 ** -18) + (4 * 2 ** -17 if io == "bf16" else 0)
    rows = [None if x[n] is None else x[n][None].cuda() for n in ("x", "f", "i", "z")]
    kw = dict(decay=gpu(x["decay"]), i=rows[2], z=rows[3], unit_variance=unit)
    y, fin = gla.recur_fwd(*rows[:2], init_state=gpu(x["init"]), out_dtype=F32, **kw)
    near(y, ref["y"], tol, "y")
    near(fin, ref["final"], tol, "final")
    if io == "bf16":
        check_bf16_rounding(gla.recur_fwd(*rows[:2], init_state=gpu(x["init"]), **kw)[0], y)
    out = gla.recur_bwd(*rows[:2], x["dy"][None].cuda(), init_state=gpu(x["init"]),
                        d_final_state=gpu(x["df"]), grad_dtype=F32, **kw)
    for n, t in zip(("dx", "df", "d_decay", "di", "dz", "d_init"), out):
        assert (t is None) == (ref[n] is None), n
        if t is not None:
            near(t, ref[n], 3 * tol + (T * 2 ** -24 if n == "d_decay" else 0), n)
    state = gpu(x["init"]).clone()
    for t in range(T):
        one = [None if r is None else r[:, t] for r in rows]
        yt = gla.recur_step(one[0], one[1], state, kw["decay"], one[2], one[3], unit, out_dtype=F32)
        near(yt, (ref["y"][0][t:t + 1], ref["y"][1][t:t + 1]), tol, f"step {t}")
    near(state, ref["final"], tol, "steps' state")
    gla.status_sync()


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("unit", [True, False])
@pytest.mark.parametrize("i,z", [(False, False), (True, False), (False, True), (True, True)])
def test_recur_gates_far_below_zero(gla, io, unit, i, z):
    """The gate itself as decay, over every bf16 number from -100 to -80, where exponentials pass the largest
    number and reciprocals the smallest: a is 0 and the drive whole."""
    check_gates(gla, gates_over(bf16_values(-100, -80), 4, io, i, z, False, 70), unit, io)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("unit", [True, False])
@pytest.mark.parametrize("decay,i,z", [(False, True, True), (True, True, True)])
def test_recur_gates_of_every_size(gla, io, unit, decay, i, z):
    """Every bf16 gate of size 2^-6 to 60, either sign."""
    v = bf16_values(-60, 60)
    check_gates(gla, gates_over(v[v.abs() >= 2 ** -6], 4, io, i, z, decay, 71), unit, io)


@pytest.mark.parametrize("unit", [True, False])
def test_recur_gates_at_the_infinities(gla, unit):
    """bf16 rows, the gate itself as decay: shut it passes the drive alone, open the state alone; with
    infinities and the largest numbers."""
    T, D = 12, 64
    g = torch.Generator().manual_seed(72)
    x, dy = (rnd(g, 1, T, D, dtype=torch.bfloat16).cuda() for _ in range(2))
    init = rnd(g, 1, D).cuda()
    for v in (-INF, -3.3895e38, -1e30, -200.0, -89.0):
        f = torch.full_like(x, v)
        y, fin = gla.recur_fwd(x, f, unit_variance=unit, init_state=init)
        assert torch.equal(y, x) and torch.equal(fin, x[:, -1].float())
        dx, df, _, _, _, d0 = gla.recur_bwd(x, f, dy, unit_variance=unit, init_state=init)
        assert torch.equal(dx, dy) and not df.any() and not d0.any()
        state = init.clone()
        assert torch.equal(gla.recur_step(x[:, 0], f[:, 0], state, unit_variance=unit), x[:, 0])
    for v in (INF, 3.3895e38, 200.0):
        f = torch.full_like(x, v)
        y, fin = gla.recur_fwd(x, f, unit_variance=unit, init_state=init, out_dtype=F32)
        assert torch.equal(fin, init) and torch.equal(y, init[:, None].expand_as(y))
        dx, df, _, _, _, d0 = gla.recur_bwd(x, f, dy, unit_variance=unit, init_state=init)
        assert not dx.any() and not df.any()
        torch.testing.assert_close(d0[0], dy[0].float().sum(0), rtol=1e-5, atol=1e-5)
    gla.status_sync()


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_recur_factor_of_nearly_open_gates(gla, io):
    """m = sqrt(1 - a^2) of decays next to 1: right down to 1 - a^2 = 2^-126 (although a is 1 from 2^-25 on), 0 below,
    the same in the prompt, the gradients and the step.  From f = -84 and decay = -exp(v): 1 - a^2 =
    2 exp(v - 84) to 2^-80 of it; with x = 1 and d_out = 1 both out and dx are m.  Errors: f's
    sigmoid 2^-21 and 84 2^-24, u's polynomial and products 2^-20, the root 2^-22, half of them in m: 2^-17."""
    v = torch.linspace(-5.0, 6.0, 4096)
    D = len(v)
    decay = -torch.exp(v)
    one = torch.ones(1, 1, D, dtype=DT[io]).cuda()
    f = torch.full_like(one, -84.0)
    room = -2 * decay.double() / (1 + torch.exp(torch.tensor(84.0, dtype=torch.float64)))
    kw = dict(decay=gpu(decay))
    y = gla.recur_fwd(one, f, out_dtype=F32, **kw)[0][0, 0]
    dx = gla.recur_bwd(one, f, one, grad_dtype=F32, **kw)[0][0, 0]
    state = torch.zeros(1, D, device="cuda")
    step = gla.recur_step(one[0], f[0], state, out_dtype=F32, **kw)[0]
    assert torch.equal(y, step) and torch.equal(y == 0, dx == 0)
    for m in (y, dx):
        m, want = m.double().cpu(), room.sqrt()
        below, above = room < 2.0 ** -126 * (1 - 2 ** -16), room > 2.0 ** -126 * (1 + 2 ** -16)
        assert below.sum() > 100 and above.sum() > 1000
        assert not m[below].any() and (((m - want).abs() <= 2 ** -17 * want) | ~above).all()
    gla.status_sync()


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("lens,packed", [([5, 0, 9, 33, 1, 130], True), ([300], False)])
def test_recur_decays_above_zero(gla, io, lens, packed):
    """They act as 0, whatever their value: their gradient is 0, the channels beside them and all other
    gradients are those of a decay of 0 (where the formula's own slope, with 1 - a, is e (h - x))."""
    x = recur_inputs(lens, 72, io, True, True, True, True, 79)
    x["decay"][::3] = 0.0
    base.recur_check(gla, x, lens, packed, False, io)
    above = dict(x, decay=x["decay"].clone())
    above["decay"][::3] = torch.rand(24, generator=torch.Generator().manual_seed(80)) + 0.01
    cu = torch.tensor(base.cu_of(lens), dtype=torch.int32).cuda() if packed else None

    def run(x, unit):
        rows = [base.lead(x[n], lens, packed).cuda() for n in ("x", "f", "dy", "i", "z")]
        kw = dict(decay=gpu(x["decay"]), i=rows[3], z=rows[4], unit_variance=unit, init_state=gpu(x["init"]), cu_seqlens=cu)
        return [*gla.recur_fwd(*rows[:2], **kw), *gla.recur_bwd(*rows[:3], d_final_state=gpu(x["df"]), **kw)]

    for unit in (False, True):
        for n, a, b in zip(("y", "final", "dx", "df", "d_decay", "di", "dz", "d_init"), run(x, unit), run(above, unit)):
            if n == "d_decay":
                assert not b[::3].any() and a[::3].all()
                a[::3] = 0
            assert torch.equal(a, b), n
    gla.status_sync()


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("decay,unit", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("lens,packed", [([5, 0, 9, 33, 1, 130], True), ([37, 37], False), ([260], False)])
def test_recur_every_combination(gla, io, decay, unit, lens, packed):
    """Input gate, output gate and initial states, each there and not."""
    for k in range(8):
        i, z, init = bool(k & 1), bool(k & 2), bool(k & 4)
        base.recur_check(gla, recur_inputs(lens, 72, io, decay, i, z, init, 76 + k), lens, packed, unit, io)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("unit", [True, False])
@pytest.mark.parametrize("most", [1.3, 1.5, 6.0])
@pytest.mark.parametrize("lens,packed", [([5, 0, 90, 33, 1], True), ([300], False)])
def test_recur_strong_decays(gla, io, unit, most, lens, packed):
    """Decays on both sides of 2 ln 2, from where a warp takes the exponential of all arguments; down to
    -6, where log a is off by 6 2^-20 < 2^-17 of a, twice the tolerance's 2^-18, which it doubles."""
    x = recur_inputs(lens, 136, io, True, True, True, True, 77)
    x["decay"] = x["decay"] * (most / 0.8)
    base.recur_check(gla, x, lens, packed, unit, io)


@pytest.mark.parametrize("T,D", [(9000, 64), (3000, 264)])
def test_recur_long_sequence_of_few_channels(gla, T, D):
    x = recur_inputs([T], D, "bf16", True, True, True, True, 78)
    x["decay"] = x["decay"] * 0.02
    base.recur_check(gla, x, [T], False, True, "bf16")


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("decay,i,z", [(True, False, True), (False, True, False)])
@pytest.mark.parametrize("B,T,D", [(90, 20, 264), (400, 1, 200), (161, 127, 72)])
def test_recur_shared_groups(gla, io, decay, i, z, B, T, D):
    """Dense sequences that share a group, in either type."""
    x = recur_inputs([T] * B, D, io, decay, i, z, True, 83)
    base.recur_check(gla, x, [T] * B, False, decay, io)


def test_recur_of_the_most_rows(gla):
    """2^31 - 1 rows of eight channels, packed as one sequence and as single tokens: the first and the last
    rows (between them x is 0, and the state is 0 after some hundred rows)."""
    R, D, n = 2 ** 31 - 1, 8, 1000
    room_for(172)
    g = torch.Generator().manual_seed(84)
    bf = torch.bfloat16
    ends = rnd(g, 2 * n, D, dtype=bf)
    x = torch.zeros(R, D, dtype=bf, device="cuda")
    x[:n], x[-n:] = ends[:n].cuda(), ends[n:].cuda()
    f = torch.zeros(R, D, dtype=bf, device="cuda")
    out = torch.empty(R, D, dtype=bf, device="cuda")
    cu = torch.tensor([0, R], dtype=torch.int32).cuda()
    y, fin = gla.recur_fwd(x, f, cu_seqlens=cu, out=out)
    gla.status_sync()
    ref = block_ref.recur_all(ends, torch.zeros(2 * n, D), None, None, None, True, None, [0, n, 2 * n])
    value, size = ref["y"]
    tol = 2 * (ref["memory"] * 2 ** -22 + 2 ** -18)
    near(torch.cat([y[:n], y[-n:]]), (value, tol * size + 2 ** -8 * value.abs()), 1.001, "y")
    near(fin, (ref["final"][0][1:], ref["final"][1][1:]), tol, "final")
    assert not y[R // 2:R // 2 + n].any()
    state = torch.zeros(R, D, device="cuda")
    gla.recur_step(x, f, state, out=out)
    gla.status_sync()
    want = 0.75 ** 0.5 * ends.double()  # a = 1/2
    near(torch.cat([state[:n], state[-n:]]), (want, want.abs()), tol, "state")
    assert torch.equal(out[-n:], state[-n:].to(bf)) and not state[R // 2:R // 2 + n].any()
    del x, f, out, y, state
    torch.cuda.empty_cache()


# ---------------------------------------------------------------- norms
def norm_check(gla, R, D, io, res32, layer, post, pbias, z, scale, weight, bias, y, means=None, seed=73):
    """block_norm_fwd and block_norm_bwd with these parts; `means`: row k's mean is added to
    res and y of the rows k, k + len, ..."""
    g = torch.Generator().manual_seed(seed)
    dt, rt = DT[io], F32 if res32 else DT[io]
    add = 0.0 if means is None else torch.tensor(means)[torch.arange(R) % len(means)][:, None]
    vec = lambda on, mean=0.0: rnd(g, D, std=0.3, mean=mean) if on else None  # noqa: E731
    res = (rnd(g, R, D, std=2.0) + 2 * add).to(rt)
    yy = (rnd(g, R, D) + add).to(dt) if y else None
    zz = rnd(g, R, D, dtype=dt) if z else None
    pw, pb, sc, w, b = vec(post, 1.0), vec(pbias), vec(scale, 0.5), vec(weight, 1.0), vec(bias)
    du, ds = rnd(g, R, D, dtype=dt) if weight else None, rnd(g, R, D, dtype=rt)
    eps = 1e-5
    ref = block_ref.block_norm_all(res, yy, zz, pw, pb, sc, w, b, layer, eps, du, ds)
    kw = dict(y=base.strided(yy), z=base.strided(zz), post_weight=gpu(pw), post_bias=gpu(pb),
              scale=gpu(sc), weight=gpu(w), bias=gpu(b), kind="layer" if layer else "rms", eps=eps)
    tol = 2 ** -17
    s, u = gla.block_norm_fwd(gpu(res), **kw, out_dtype=F32)
    if y:  # bf16: rounded once where it is stored
        value, size = ref["s"]
        near(s, (value, tol * size + (2 ** -8 * value.abs() if rt is not F32 else 0)), 1.001, "s")
    if weight:
        near(u, ref["u"], tol, "u")
        u2 = gla.block_norm_fwd(gpu(res), **kw, out_dtype=dt)[1]
        assert torch.equal(u2, u.to(dt))
    got = gla.block_norm_bwd(gpu(res), gpu(du), gpu(ds), **kw, grad_dtype=F32)
    for n, t in zip(("d_res", "dy", "dz", "d_post_weight", "d_post_bias", "d_scale", "dw", "db"), got):
        assert (t is None) == (ref.get(n) is None), n
        if t is not None:
            near(t, ref[n], 2 * tol + (R * 2 ** -24 if t.dim() == 1 else 0), n)
    gla.status_sync()


# io, res fp32, layer, post weight, post bias, z, scale, weight, bias, y
PARTS = [("bf16", True, False, True, False, True, True, True, False, True),
         ("bf16", False, True, True, True, True, True, True, True, True),
         ("fp32", True, False, True, True, True, False, True, True, True),
         ("bf16", False, True, True, False, False, True, True, False, True),
         ("fp32", True, True, False, False, True, True, True, True, True),
         ("bf16", True, False, True, True, False, False, False, False, True),
         ("fp32", True, True, False, False, False, False, True, True, False),
         ("bf16", False, False, False, False, False, False, True, True, False)]


@pytest.mark.parametrize("R,D", [(7301, 72), (2001, 2048), (3001, 520), (1001, 4104), (701, 8192)])
@pytest.mark.parametrize("parts", PARTS)
def test_block_norm_of_many_rows(gla, R, D, parts):
    """More rows than the groups of one wave own, an odd number: rows two at a time, rows on their way
    over several turns, sums over them; one and two vectors a thread."""
    norm_check(gla, R, D, *parts)


@pytest.mark.parametrize("D", [8, 72, 264, 1000, 2048, 4088, 4104])
@pytest.mark.parametrize("layer", [True, False])
@pytest.mark.parametrize("post,pbias,z,scale,bias", [(True, False, False, False, False), (True, True, False, True, True),
                                                     (True, False, False, True, True), (True, True, True, False, False),
                                                     (False, False, False, True, True)])
def test_block_norm_parts(gla, D, layer, post, pbias, z, scale, bias):
    """Every part with and without its neighbours, where the last threads of a row have no columns."""
    norm_check(gla, 21, D, "fp32", True, layer, post, pbias, z, scale, True, bias, True)


@pytest.mark.parametrize("io,res32", [("bf16", False), ("bf16", True), ("fp32", True)])
@pytest.mark.parametrize("layer", [True, False])
@pytest.mark.parametrize("D", [72, 4104])
def test_block_norm_every_combination(gla, io, res32, layer, D):
    """Every part there and not."""
    for post, pbias in ((False, False), (True, False), (True, True)):
        for weight, bias in ((False, False), (True, False), (True, True)):
            for z in (False, True):
                for scale in (False, True):
                    norm_check(gla, 9, D, io, res32, layer, post, pbias, z, scale, weight, bias, True)
    for bias in (False, True):
        norm_check(gla, 9, D, io, res32, layer, False, False, False, False, True, bias, False)


@pytest.mark.parametrize("R,D", [(33, 264), (1501, 2048), (401, 5120)])
@pytest.mark.parametrize("parts", [p for p in PARTS if p[2]] + [PARTS[2]])
def test_block_norm_of_far_and_near_means(gla, R, D, parts):
    """Rows whose means are 0 to 1000 deviations, side by side."""
    norm_check(gla, R, D, *parts, means=(0.0, 0.3, 0.49, 0.51, 1000.0, 1.0, -2.0, 0.0, 3.9, 4.1, -30.0))


def test_layer_norm_keeps_the_variance(gla):
    """The factor 1 / deviation of rows whose mean is up to four deviations, from the projection of the results on
    the exact ones (which a wrong mean, and the rounding of 2048 elements, leave out): in units of
    2^-24 the sum of the squares is off by 13 (four in a thread, one of a pair, five in a warp, three of
    warps), 1.25 times that and 6.5 more where the mean, up to half a deviation, is
    taken out of it, one for the difference; half of it in the root, four for the root, one for the product: 17."""
    D, means = 2048, (0.0, 0.2, 0.45, 0.6, 1.0, 2.0, 3.0, 3.9)
    R = 300 * len(means)
    g = torch.Generator().manual_seed(74)
    x = rnd(g, R, D) + torch.tensor(means)[torch.arange(R) % len(means)][:, None]
    du = rnd(g, R, D)
    one = torch.ones(D)
    ref = block_ref.block_norm_all(x, None, None, None, None, None, one, None, True, 1e-12, du)
    u = gla.block_norm_fwd(gpu(x), weight=gpu(one), kind="layer", eps=1e-12)[1]
    d = gla.block_norm_bwd(gpu(x), gpu(du), weight=gpu(one), kind="layer", eps=1e-12)[0]
    for n, t in (("u", u), ("d_res", d)):
        want = ref[n][0]
        off = ((t.double().cpu() * want).sum(-1) / (want * want).sum(-1) - 1).abs()
        assert float(off.max()) <= 17 * 2 ** -24, (n, float(off.max()))


def test_block_norm_of_the_most_rows(gla):
    """2^31 - 1 rows of eight channels: the first and the last rows, forward and gradient."""
    R, D, n = 2 ** 31 - 1, 8, 1000
    room_for(136)
    g = torch.Generator().manual_seed(75)
    ends = rnd(g, 2 * n, D, dtype=torch.bfloat16)
    du, ds = (rnd(g, 2 * n, D, dtype=torch.bfloat16) for _ in range(2))
    w = rnd(g, D, mean=1.0)
    eps = 1e-6
    ref = block_ref.block_norm_all(ends, None, None, None, None, None, w, None, False, eps, du, ds)

    def long(t):
        x = torch.zeros(R, D, dtype=torch.bfloat16, device="cuda")
        x[:n], x[-n:] = t[:n].cuda(), t[n:].cuda()
        return x

    res = long(ends)
    u = gla.block_norm_fwd(res, weight=gpu(w), eps=eps)[1]
    got = torch.cat([u[:n], u[-n:]])
    near(got, (ref["u"][0], 2 ** -17 * ref["u"][1] + 2 ** -8 * ref["u"][0].abs()), 1.001, "u")
    assert not u[n:2 * n].any() and not u[R // 2:R // 2 + n].any()
    del u
    d = gla.block_norm_bwd(res, long(du), long(ds), weight=gpu(w), eps=eps)
    got = torch.cat([d[0][:n], d[0][-n:]])
    near(got, (ref["d_res"][0], 2 ** -16 * ref["d_res"][1] + 2 ** -8 * ref["d_res"][0].abs()), 1.001, "d_res")
    # (of the rows between nothing is added)
    near(d[6], ref["dw"], 2 ** -16 + 2 * n * 2 ** -24, "dw")
    gla.status_sync()
    del res, d
    torch.cuda.empty_cache()


# ---------------------------------------------------------------- feed-forward
@pytest.mark.parametrize("backward", [False, True])
def test_glu_gives_up_again_and_again(gla, backward):
    """Waits that run out, many times over: each call ends with GLA_ERR_TIMEOUT or right, every copy of
    either SM of a pair lands before its block ends, and what runs behind it is right.  (The sums over K
    take a millisecond, so that a wait is open when the limit of a nanosecond has passed.)"""
    g = torch.Generator().manual_seed(80)
    bf = torch.bfloat16
    R, D, F = (1 << 18, 64, 200) if backward else (256, 1 << 18, 128)
    x = rnd(g, R, D, dtype=bf).cuda()
    wg, wu = (rnd(g, F, D, std=D ** -0.5, dtype=bf).cuda() for _ in range(2))
    dh = rnd(g, R, F, dtype=bf).cuda() if backward else None
    run = (lambda: gla.glu_bwd(x, wg, wu, dh)) if backward else (lambda: (gla.glu_fwd(x, wg, wu),))
    want = run()
    gla.status_sync()
    hits = 0
    for _ in range(30):
        gla.set_wait_limit_ns(1)
        try:
            got = run()
        finally:
            gla.set_wait_limit_ns(0)
        behind = run()  # on the same SMs, right behind it
        try:
            gla.status_sync()
            ok = True
        except gla.GlaError as e:
            assert e.status == 5
            hits, ok = hits + 1, False
        for a, b, c in zip(got, behind, want):
            assert torch.equal(b, c) and (not ok or torch.equal(a, c))
    assert hits


def test_glu_gradients_of_the_most_rows(gla):
    """2^26 rows, of numbers whose sums are exact: with w_gate = 0 and w_up the identity dg is
    d_out x / 2 and du is 0, and dw_gate = dg^T x sums halves of whole numbers."""
    R, D = 1 << 26, 8
    g = torch.Generator(device="cuda").manual_seed(81)
    bf = torch.bfloat16
    x = torch.randint(-1, 2, (R, D), generator=g, device="cuda", dtype=torch.int8).to(bf)
    dh = torch.randint(-1, 2, (R, D), generator=g, device="cuda", dtype=torch.int8).to(bf)
    dh[:, 3], x[:, 3] = 1, 1  # one that only grows
    wg, wu = torch.zeros(D, D, dtype=bf, device="cuda"), torch.eye(D, dtype=bf, device="cuda")
    dx, dg, du = gla.glu_bwd(x, wg, wu, dh, grad_dtype=F32)
    gla.status_sync()
    want = torch.zeros(D, D, dtype=torch.float64, device="cuda")
    for k in range(0, R, R // 64):
        xs, hs = x[k:k + R // 64].double(), dh[k:k + R // 64].double()
        want += (hs * xs / 2).t() @ xs
    assert torch.equal(dg.double(), want) and float(want[3, 3]) == R / 2
    assert not du.any() and not dx.any()


def test_glu_of_the_most_rows(gla):
    """2^31 - 1 rows of eight channels and features: the first and the last rows."""
    R, D, n = 2 ** 31 - 1, 8, 1000
    room_for(68)
    g = torch.Generator().manual_seed(82)
    bf = torch.bfloat16
    ends = rnd(g, 2 * n, D, dtype=bf)
    wg, wu = (rnd(g, D, D, std=D ** -0.5, dtype=bf) for _ in range(2))
    x = torch.zeros(R, D, dtype=bf, device="cuda")
    x[:n], x[-n:] = ends[:n].cuda(), ends[n:].cuda()
    h = gla.glu_fwd(x, gpu(wg), gpu(wu))
    gla.status_sync()
    value, tol = block_ref.glu_all(ends, wg, wu)["h"]
    near(torch.cat([h[:n], h[-n:]]), (value, tol + 2 ** -8 * value.abs()), 1.001, "h")
    assert not h[R // 2:R // 2 + n].any()
    del x, h
    torch.cuda.empty_cache()


@pytest.mark.parametrize("R,D,F", [(1, 520, 72), (20, 72, 200), (128, 1032, 136)])
def test_glu_few_rows_are_apart(gla, R, D, F):
    """Infinities and NaN of one row reach no other of the few."""
    g = torch.Generator().manual_seed(85)
    x = rnd(g, R, D, dtype=torch.bfloat16)
    wg, wu = (rnd(g, F, D, std=0.1, dtype=torch.bfloat16).cuda() for _ in range(2))
    a = gla.glu_fwd(gpu(x), wg, wu)
    x[R // 2, 5], x[R - 1, 0] = float("nan"), INF
    b = gla.glu_fwd(gpu(x), wg, wu)
    fine = [r for r in range(R) if r not in (R // 2, R - 1)]
    assert torch.equal(a[fine], b[fine]) and torch.isnan(b[R // 2]).all() and not torch.isfinite(b[R - 1]).all()
    gla.status_sync()


@pytest.mark.parametrize("R,D,F", [(129, 1032, 520), (192, 2048, 264), (255, 72, 1352), (320, 520, 392), (511, 264, 136),
                                   (768, 136, 2056), (128, 520, 1352), (127, 2056, 72), (2, 8192, 136)])
def test_glu_between_few_rows_and_many(gla, R, D, F):
    base.test_glu(gla, R, D, F)
