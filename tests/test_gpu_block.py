"""The gated linear recurrence, the norms between blocks and the gated feed-forward
projections on the GPU against plain 64-bit implementations (tests/block_ref.py).

Tolerances, per element, are multiples of the same sum over the absolute values
of its terms (the sizes in ``block_ref``), which is what fp32 rounding errors scale with:
  recurrence: a sigmoid is off by 2^-21 (hardware exponential and reciprocal 2^-22 each,
      bf16 rows: and its argument's rounding, |f| 2^-24, |f| < 8 here); so log a by
      2^-20 of itself, m by 2^-19 (its square root halves what 1 - a^2 is off by), a by 2^-23
      and its exponent's share, |log a| 2^-20.  A state that remembers N tokens adds N
      roundings of 2^-23 (product and sum), N of a's, and N |log a| 2^-20 <= 2^-19: N 2^-22 +
      2^-18 with the drive's products.  Its map over a run and the maps of
      other runs are the same products in another order: twice that.  Gradients are products of
      such an e, such a state and at most six more factors.
  norms: a sum over a row is off by at most (thread's 16 + 5 + 16) 2^-24 < 2^-18 of its
      absolute sum, and the sizes carry how that moves everything behind it; about ten more
      roundings and a sigmoid: 2^-17 for s and u, twice that for gradients, which go through two
      norms.  Sums over R rows: R 2^-24 more.
  projections: see block_ref.glu_all, which returns tolerances.
bf16 results are required to be the fp32 results rounded once (half a step).
"""
import threading

import pytest
import torch

import block_ref
from parity import check_bf16_rounding

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
F32 = torch.float32


@pytest.fixture(scope="module")
def gla():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_linear_attention_gla_gb300 import build as glabuild
    glabuild.build()
    import gated_linear_attention_gla_gb300 as m
    return m


def rnd(g, *shape, std=1.0, mean=0.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g) * std + mean).to(dtype)


def cu_of(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def gpu(t):
    return None if t is None else t.cuda()


def near(got, pair, factor, what):
    """|got - value| <= factor * size, element by element."""
    ref, size = pair
    err = (got.detach().double().cpu().reshape(ref.shape) - ref).abs()
    bad = ~(err <= factor * size + 1e-30)
    assert not bad.any(), \
        f"{what}: off by {float((err / (size + 1e-30)).max()):.3g} of its terms, allowed {factor:.3g}"


def strided(t):
    """The same rows, as columns of a wider tensor on the GPU."""
    if t is None:
        return None
    wide = torch.full((*t.shape[:-1], t.shape[-1] + 32), 7.0, dtype=t.dtype, device="cuda")
    wide[..., 16:-16] = t.cuda()
    return wide[..., 16:-16]


def lead(t, lens, packed):
    return t if packed or t is None else t.reshape(len(lens), lens[0], *t.shape[1:])


# ---------------------------------------------------------------- recurrence
# (lens, packed): one token, empty sequences, ends inside runs of 4 and 8 and between
# them, dense ones that share a group and that do not (256 tokens and more)
LENS = [([1], True), ([1], False), ([0, 3, 0, 1, 70, 0], True), ([5, 5, 5], False),
        ([31, 1, 8, 2, 255, 4, 257], True), ([64] * 5, False), ([1] * 40, True),
        ([300, 300], False), ([7, 1, 1, 1, 6, 8, 16, 0, 0, 4, 12], True)]
GATES = [("bf16", 264, True, True, True, True, True), ("fp32", 136, True, False, True, False, True),
         ("bf16", 8, False, True, False, False, False), ("fp32", 520, False, False, False, True, True),
         ("bf16", 72, False, True, True, True, True), ("fp32", 64, True, True, False, True, False)]


def recur_inputs(lens, D, io, decay, i, z, init, seed):
    g = torch.Generator().manual_seed(seed)
    R, B, dt = sum(lens), len(lens), DT[io]
    return dict(x=rnd(g, R, D, dtype=dt), f=rnd(g, R, D, mean=0.0 if decay else 2.0, dtype=dt),
                decay=-torch.rand(D, generator=g) * 0.8 if decay else None,
                i=rnd(g, R, D, dtype=dt) if i else None, z=rnd(g, R, D, dtype=dt) if z else None,
                init=rnd(g, B, D) if init else None, dy=rnd(g, R, D, dtype=dt), df=rnd(g, B, D))


def recur_check(gla, x, lens, packed, unit, io, want_in_place=True):
    cu = cu_of(lens)
    init = x["init"]
    ref = block_ref.recur_all(x["x"], x["f"], x["decay"], x["i"], x["z"], unit, init, cu,
                              x["dy"], x["df"])
    tol = 2 * (ref["memory"] * 2 ** -22 + 2 ** -18)
    R = max(1, cu[-1])
    cug = torch.tensor(cu, dtype=torch.int32).cuda() if packed else None
    rows = [strided(lead(x[n], lens, packed)) for n in ("x", "f", "i", "z")]
    kw = dict(decay=gpu(x["decay"]), i=rows[2], z=rows[3], unit_variance=unit, cu_seqlens=cug)
    y, fin = gla.recur_fwd(*rows[:2], init_state=gpu(init), out_dtype=F32, **kw)
    near(y, ref["y"], tol, "y")
    near(fin, ref["final"], tol, "final")
    if io == "bf16":
        y16, fin16 = gla.recur_fwd(*rows[:2], init_state=gpu(init), **kw)
        check_bf16_rounding(y16, y)
        assert torch.equal(fin16, fin)
    if init is not None:  # the state updated in place
        state = gpu(init).clone()
        y2, fin2 = gla.recur_fwd(*rows[:2], init_state=state, final_state=state, out_dtype=F32, **kw)
        assert torch.equal(y2, y) and torch.equal(fin2, fin) and fin2 is state
    dy = gpu(lead(x["dy"], lens, packed))
    grads = {}
    for gd in {DT[io], F32}:
        grads[gd] = gla.recur_bwd(*rows[:2], dy, init_state=gpu(init), d_final_state=gpu(x["df"]),
                                  grad_dtype=gd, **kw)
    names = ("dx", "df", "d_decay", "di", "dz", "d_init")
    got = dict(zip(names, grads[F32]))
    for n in names:
        if got[n] is None:
            assert ref[n] is None
        elif n == "d_decay":
            near(got[n], ref[n], 3 * tol + R * 2 ** -24, n)
        elif ref[n][0] is not None:
            near(got[n], ref[n], 3 * tol, n)
    if io == "bf16":
        for n, p, q in zip(names, grads[DT[io]], grads[F32]):
            if p is None or n in ("d_decay", "d_init"):
                assert p is None or torch.equal(p, q)
            else:
                check_bf16_rounding(p, q)
    gla.status_sync()


@pytest.mark.parametrize("lens,packed", LENS)
@pytest.mark.parametrize("io,D,decay,unit,i,z,init", GATES)
def test_recur(gla, lens, packed, io, D, decay, unit, i, z, init):
    recur_check(gla, recur_inputs(lens, D, io, decay, i, z, init, 7), lens, packed, unit, io)


@pytest.mark.parametrize("lens,packed,D,io", [
    ([2500], False, 64, "bf16"), ([1200, 1200], False, 72, "fp32"), ([700, 0, 1900, 33], True, 136, "bf16")])
def test_recur_long(gla, lens, packed, D, io):
    """Several steps of a cluster's blocks, slow decays."""
    x = recur_inputs(lens, D, io, True, True, True, True, 8)
    x["decay"] = x["decay"] * 0.02
    recur_check(gla, x, lens, packed, True, io)


def test_recur_gradients_against_differences(gla):
    """The directional derivative of the 64-bit formulas, by central differences."""
    lens = [9, 0, 30, 1]
    cu, D = cu_of(lens), 24
    x = recur_inputs(lens, D, "fp32", True, True, True, True, 9)
    g = torch.Generator().manual_seed(10)
    names = ("x", "f", "decay", "i", "z", "init")
    way = {n: rnd(g, *x[n].shape).double() for n in names}

    def loss(t):
        v = {n: x[n].double() + t * way[n] for n in names}
        y, fin = block_ref.recur(v["x"], v["f"], v["decay"], v["i"], v["z"], True, v["init"], cu)
        return float((y * x["dy"].double()).sum() + (fin * x["df"].double()).sum())

    x["decay"] = x["decay"] - 0.2
    h = 1e-5
    slope = (loss(h) - loss(-h)) / (2 * h)
    out = gla.recur_bwd(gpu(x["x"]), gpu(x["f"]), gpu(x["dy"]), gpu(x["decay"]), i=gpu(x["i"]),
                        z=gpu(x["z"]), init_state=gpu(x["init"]), d_final_state=gpu(x["df"]),
                        cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda())
    got = dict(zip(("x", "f", "decay", "i", "z", "init"), out))
    terms = {n: got[n].double().cpu() * way[n] for n in names}
    total = float(sum(t.sum() for t in terms.values()))
    size = float(sum(t.abs().sum() for t in terms.values()))
    # fp32 gradients 2^-16 of their terms; differences: h^2 times a third derivative
    assert abs(total - slope) <= 2 ** -16 * size + 1e-6 * size


@pytest.mark.parametrize("io,D,decay,unit,i,z", [("bf16", 264, True, True, True, True),
                                                 ("fp32", 72, False, False, False, True),
                                                 ("bf16", 2048, True, False, True, False)])
def test_recur_steps_continue_a_prompt(gla, io, D, decay, unit, i, z):
    """Single tokens over a pool of pages, each step writing another page, give the prompt."""
    B, T = 5, 6
    lens = [T] * B
    x = recur_inputs(lens, D, io, decay, i, z, True, 11)
    cu = cu_of(lens)
    ref = block_ref.recur_all(x["x"], x["f"], x["decay"], x["i"], x["z"], unit, x["init"], cu)
    tol = 2 * (ref["memory"] * 2 ** -22 + 2 ** -18)
    pool = torch.full((2 * B + 3, D), 5.0).cuda()
    at = torch.arange(B, dtype=torch.int32)
    pool[:B] = x["init"].cuda()
    seq = {n: None if x[n] is None else x[n].reshape(B, T, D).cuda() for n in ("x", "f", "i", "z")}
    dec = gpu(x["decay"])
    for t in range(T):
        nxt = (at + B) % (2 * B)
        kw = dict(decay=dec, i=None if seq["i"] is None else seq["i"][:, t],
                  z=None if seq["z"] is None else seq["z"][:, t], unit_variance=unit)
        old = pool.clone()
        y = gla.recur_step(seq["x"][:, t], seq["f"][:, t], pool, slots=at.cuda(),
                           out_slots=nxt.cuda(), out_dtype=F32, **kw)
        rows = torch.arange(B) * T + t
        near(y, (ref["y"][0][rows], ref["y"][1][rows]), tol, f"y {t}")
        assert torch.equal(pool[at.long()], old[at.long()])  # the pages read stay
        assert torch.equal(pool[2 * B:], old[2 * B:])
        if io == "bf16":
            dense = old[at.long()].clone()
            y16 = gla.recur_step(seq["x"][:, t], seq["f"][:, t], dense, **kw)
            check_bf16_rounding(y16, y)
            assert torch.equal(dense, pool[nxt.long()])
        at = nxt
    near(pool[at.long()], ref["final"], tol, "states")
    gla.status_sync()


def test_recur_step_tables(gla):
    D = 64
    g = torch.Generator().manual_seed(12)
    x, f = rnd(g, 4, D).cuda(), rnd(g, 4, D).cuda()
    pool = rnd(g, 6, D).cuda()
    old = pool.clone()
    out = torch.full((4, D), 9.0).cuda()
    slots = torch.tensor([2, -1, 0, 5], dtype=torch.int32).cuda()
    gla.recur_step(x, f, pool, slots=slots, out=out)
    gla.status_sync()
    assert torch.equal(pool[[1, 3, 4]], old[[1, 3, 4]]) and bool((out[1] == 9).all())
    assert not torch.equal(pool[2], old[2]) and not torch.equal(pool[5], old[5])
    pool.copy_(old)
    out.fill_(9.0)
    slots = torch.tensor([2, 6, 0, 7], dtype=torch.int32).cuda()  # 6 and 7 are no pages
    gla.recur_step(x, f, pool, slots=slots, out=out)
    with pytest.raises(gla.GlaError):
        gla.status_sync()
    assert torch.equal(pool[[1, 3, 4, 5]], old[[1, 3, 4, 5]]) and bool((out[[1, 3]] == 9).all())
    # two rows read one page and write two others
    gla.recur_step(x[:2], f[:2], pool, slots=torch.tensor([3, 3], dtype=torch.int32).cuda(),
                   out_slots=torch.tensor([1, 4], dtype=torch.int32).cuda())
    gla.status_sync()
    assert torch.equal(pool[3], old[3])


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("decay", [True, False])
def test_recur_sequences_are_apart(gla, io, decay):
    """Infinities and NaN of one sequence reach no other, forwards or backwards."""
    lens, D = [37, 20, 0, 1, 90], 72
    x = recur_inputs(lens, D, io, decay, True, True, True, 13)
    cu = cu_of(lens)
    cug = torch.tensor(cu, dtype=torch.int32).cuda()

    def both(x):
        kw = dict(decay=gpu(x["decay"]), i=gpu(x["i"]), z=gpu(x["z"]), init_state=gpu(x["init"]),
                  cu_seqlens=cug)
        y, fin = gla.recur_fwd(gpu(x["x"]), gpu(x["f"]), **kw)
        g = gla.recur_bwd(gpu(x["x"]), gpu(x["f"]), gpu(x["dy"]), d_final_state=gpu(x["df"]), **kw)
        return [y, g[0], g[1], g[3], g[4]], [fin, g[5]]

    rows, states = both(x)
    bad = {k: None if v is None else v.clone() for k, v in x.items()}
    bad["x"][cu[1] - 1, 0] = float("inf")       # the last token of sequence 0
    bad["x"][cu[1] + 3, 1] = float("nan")
    bad["init"][1, 2] = float("inf")
    bad["dy"][cu[4], 3] = float("inf")          # the first token of the last sequence
    bad["df"][1, 4] = float("nan")
    rows2, states2 = both(bad)
    inside = {0: slice(cu[0], cu[1]), 1: slice(cu[1], cu[2]), 3: slice(cu[3], cu[4]), 4: slice(cu[4], cu[5])}
    hit = {0: {0}, 1: {1, 2, 4}, 3: set(), 4: {3}}
    for s, sl in inside.items():
        fine = [c for c in range(D) if c not in hit[s]]
        for p, q in zip(rows, rows2):
            assert torch.equal(p[sl][:, fine], q[sl][:, fine])
        for p, q in zip(states, states2):
            assert torch.equal(p[s][fine], q[s][fine])
    assert torch.isinf(rows2[0][cu[1] - 1, 0]) or torch.isnan(rows2[0][cu[1] - 1, 0])


def test_recur_closed_gates(gla):
    """Gates at the infinities: what is masked leaves the state and its gradient alone."""
    T, D = 40, 64
    g = torch.Generator().manual_seed(14)
    x, dy = rnd(g, 1, T, D).cuda(), rnd(g, 1, T, D).cuda()
    init, dec = rnd(g, 1, D).cuda(), torch.full((D,), -0.5).cuda()
    inf = float("inf")
    for lowest in (-inf, -3.3895e38):
        f = torch.full((1, T, D), lowest).cuda()
        for unit in (True, False):
            y, fin = gla.recur_fwd(x, f, dec, unit_variance=unit, init_state=init)
            assert torch.equal(fin, init) and torch.equal(y, init[:, None].expand_as(y))
            dx, df, dd, _, _, d0 = gla.recur_bwd(x, f, dy, dec, unit_variance=unit, init_state=init)
            assert not dx.any() and not df.any() and not dd.any()
            torch.testing.assert_close(d0[0], dy[0].sum(0), rtol=1e-5, atol=1e-5)
    # a = sigmoid(-inf) = 0: the state is the drive alone; an input gate at -inf shuts it
    f = torch.full((1, T, D), -inf).cuda()
    y, _ = gla.recur_fwd(x, f, unit_variance=False, init_state=init)
    assert torch.equal(y, x)
    i = torch.full((1, T, D), -inf).cuda()
    y, fin = gla.recur_fwd(x, f, i=i, init_state=init)
    assert not y.any() and not fin.any()
    # a decay above zero acts as zero
    y, fin = gla.recur_fwd(x, x, torch.full((D,), 3.0).cuda(), init_state=init)
    assert torch.equal(fin, init)


@pytest.mark.parametrize("T,lens", [(40, None), (4000, None), (78, [17, 1, 60])])
@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_recur_decay_of_nan(gla, io, T, lens):
    """A channel whose decay is NaN is NaN from its first token on, and the other channels
    have the bits they have beside a finite one (below -2 ln 2, so that either way the
    warp's exponential is the one for all decays)."""
    D = 72
    x = recur_inputs(lens or [T], D, io, True, True, True, True, 21)
    kw = dict(i=gpu(x["i"]), z=gpu(x["z"]), init_state=gpu(x["init"]))
    rows = [gpu(x["x"]), gpu(x["f"]), gpu(x["dy"])]
    if lens is None:
        rows = [v[None] for v in rows]
        kw["i"], kw["z"] = kw["i"][None], kw["z"][None]
    else:
        kw["cu_seqlens"] = torch.tensor(cu_of(lens), dtype=torch.int32).cuda()
    decay = gpu(x["decay"]).clone()
    decay[[3, 65]] = -4.0
    bad = decay.clone()
    bad[[3, 65]] = float("nan")
    fine = [c for c in range(D) if c not in (3, 65)]

    def run(d):
        y, fin = gla.recur_fwd(rows[0], rows[1], d, **kw)
        g = gla.recur_bwd(rows[0], rows[1], rows[2], d, d_final_state=gpu(x["df"]), **kw)
        tok = [v.reshape(-1, D)[:1].contiguous() for v in (rows[0], rows[1], kw["i"], kw["z"])]
        state = kw["init_state"][:1].clone()
        out = gla.recur_step(tok[0], tok[1], state, d, tok[2], tok[3])
        return [y, fin, *g, out, state]

    for p, q in zip(run(decay), run(bad)):
        assert torch.equal(p[..., fine], q[..., fine])
        assert not torch.isnan(p).any() and torch.isnan(q[..., [3, 65]]).all()
    gla.status_sync()


@pytest.mark.parametrize("B,T,D", [(100, 20, 264), (3, 127, 72), (3, 128, 72), (400, 1, 200)])
def test_recur_equal_sequences(gla, B, T, D):
    """Dense sequences that share a group (three by three with a last group of one, in many) and
    that do not."""
    x = recur_inputs([T] * B, D, "bf16", True, True, True, True, 22)
    recur_check(gla, x, [T] * B, False, True, "bf16")


def test_recur_malformed_offsets(gla):
    R, D = 64, 64
    g = torch.Generator().manual_seed(15)
    x, f, dy = (rnd(g, R, D).cuda() for _ in range(3))
    for cu in ([0, 70, 64], [0, 40, 30, 64], [1, 20, 64], [0, 20, 60], [-5, 20, 64], [0, 20, -1]):
        c = torch.tensor(cu, dtype=torch.int32).cuda()
        gla.recur_fwd(x, f, cu_seqlens=c)
        with pytest.raises(gla.GlaError):
            gla.status_sync()
        gla.recur_bwd(x, f, dy, cu_seqlens=c)
        with pytest.raises(gla.GlaError):
            gla.status_sync()
    gla.recur_fwd(x, f, cu_seqlens=torch.tensor([0, 64], dtype=torch.int32).cuda())
    gla.status_sync()


def test_recur_empty_calls(gla):
    D = 64
    init, df = torch.randn(3, D).cuda(), torch.randn(3, D).cuda()
    none = torch.zeros(3, 0, D).cuda()
    y, fin = gla.recur_fwd(none, none, init_state=init)
    assert y.shape == none.shape and torch.equal(fin, init)
    dec = -torch.rand(D).cuda()
    g = gla.recur_bwd(none, none, none, dec, init_state=init, d_final_state=df)
    assert torch.equal(g[5], df) and not g[2].any()
    cu = torch.zeros(4, dtype=torch.int32).cuda()
    rows = torch.zeros(0, D).cuda()
    y, fin = gla.recur_fwd(rows, rows, cu_seqlens=cu)
    assert not fin.any()
    g = gla.recur_bwd(rows, rows, rows, dec, d_final_state=df, cu_seqlens=cu)
    assert torch.equal(g[5], df) and not g[2].any()
    gla.status_sync()


# ---------------------------------------------------------------- norms
NORMS = [  # io, res fp32, layer, post, z, scale, weight, y
    ("bf16", False, False, True, True, True, True, True),
    ("bf16", True, True, True, True, True, True, True),
    ("fp32", True, False, True, False, True, True, True),
    ("fp32", True, True, False, True, False, True, True),
    ("bf16", True, False, False, False, False, True, True),
    ("bf16", False, False, True, True, False, False, True),
    ("bf16", False, True, False, False, False, True, False),
    ("fp32", True, False, False, False, False, True, False)]


@pytest.mark.parametrize("R,D", [(1, 8), (3, 264), (37, 512), (17, 520), (70, 1024), (9, 2048),
                                 (5, 2056), (3, 4096), (2, 8192), (700, 72)])
@pytest.mark.parametrize("io,res32,layer,post,z,scale,weight,y", NORMS)
def test_block_norm(gla, R, D, io, res32, layer, post, z, scale, weight, y):
    g = torch.Generator().manual_seed(16)
    dt, rt = DT[io], F32 if res32 else DT[io]
    vec = lambda on, mean=0.0: rnd(g, D, std=0.3, mean=mean) if on else None  # noqa: E731
    res = rnd(g, R, D, std=2.0, dtype=rt)
    yy = rnd(g, R, D, mean=0.3, dtype=dt) if y else None
    zz = rnd(g, R, D, dtype=dt) if z else None
    pw, pb, sc = vec(post, 1.0), vec(post and layer), vec(scale, 0.5)
    w, b = vec(weight, 1.0), vec(weight and layer)
    du = rnd(g, R, D, dtype=dt) if weight else None
    ds = rnd(g, R, D, dtype=rt)
    eps = 1e-5
    ref = block_ref.block_norm_all(res, yy, zz, pw, pb, sc, w, b, layer, eps, du, ds)
    kw = dict(y=strided(yy), z=strided(zz), post_weight=gpu(pw), post_bias=gpu(pb), scale=gpu(sc),
              weight=gpu(w), bias=gpu(b), kind="layer" if layer else "rms", eps=eps)
    tol = 2 ** -17
    s, u = gla.block_norm_fwd(gpu(res), **kw, out_dtype=F32)
    if y and rt is F32:
        near(s, ref["s"], tol, "s")
    elif y:  # rounded once to bf16 where it is stored
        near(s, (ref["s"][0], tol * ref["s"][1] + 2 ** -8 * ref["s"][0].abs()), 1.001, "s")
    else:
        assert s is None
    if weight:
        near(u, ref["u"], tol, "u")
        s2, u2 = gla.block_norm_fwd(gpu(res), **kw, out_dtype=dt)
        assert s2 is None or torch.equal(s2, s)
        assert torch.equal(u2, u.to(dt))
    else:
        assert u is None
    if y:  # the residual stream in place
        inplace = gpu(res).clone()
        s3, _ = gla.block_norm_fwd(inplace, **kw, res_out=inplace)
        assert s3 is inplace and torch.equal(s3, s)
    names = ("d_res", "dy", "dz", "d_post_weight", "d_post_bias", "d_scale", "dw", "db")
    grads = {gd: gla.block_norm_bwd(gpu(res), gpu(du), gpu(ds), **kw, grad_dtype=gd)
             for gd in {dt, F32}}
    for n, t in zip(names, grads[F32]):
        if ref.get(n) is None:
            assert t is None, n
        else:
            near(t, ref[n], 2 * tol + (R * 2 ** -24 if t.dim() == 1 else 0), n)
    if dt is not F32:
        for n, p, q in zip(names, grads[dt], grads[F32]):
            assert p is None or torch.equal(p, q.to(p.dtype)), n
    gla.status_sync()


def test_block_norm_rows_are_apart(gla):
    """A row with infinities or NaN leaves the others' results alone; a row of zeros is fine."""
    R, D = 40, 200
    g = torch.Generator().manual_seed(17)
    res, y = rnd(g, R, D), rnd(g, R, D)
    w = rnd(g, D).cuda()
    kw = dict(post_weight=w, weight=w)
    du, ds = rnd(g, R, D).cuda(), rnd(g, R, D).cuda()
    res[5] = 0
    y[5] = 0
    a = gla.block_norm_fwd(gpu(res), gpu(y), **kw)
    ga = gla.block_norm_bwd(gpu(res), du, ds, gpu(y), **kw)
    assert not a[1][5].any()
    res[7, 3], y[9, 4], y[11, 0] = float("inf"), float("nan"), float("-inf")
    b = gla.block_norm_fwd(gpu(res), gpu(y), **kw)
    gb = gla.block_norm_bwd(gpu(res), du, ds, gpu(y), **kw)
    fine = [r for r in range(R) if r not in (7, 9, 11)]
    for p, q in zip((*a, ga[0], ga[1]), (*b, gb[0], gb[1])):
        assert torch.equal(p[fine], q[fine])
        assert not torch.isfinite(q[9]).all()


def test_block_norm_without_some_gradients(gla):
    """d_out or d_res_out absent are zeros; no rows give zero gradients of the parameters."""
    R, D = 33, 136
    g = torch.Generator().manual_seed(18)
    res, y, du = (rnd(g, R, D).cuda() for _ in range(3))
    w = rnd(g, D).cuda()
    zero = torch.zeros(R, D).cuda()
    kw = dict(y=y, post_weight=w, weight=w)
    for p, q in zip(gla.block_norm_bwd(res, du, None, **kw), gla.block_norm_bwd(res, du, zero, **kw)):
        assert (p is None and q is None) or torch.equal(p, q)
    got = gla.block_norm_bwd(res, None, du, **kw)
    want = gla.block_norm_bwd(res, zero, du, **kw)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and got[6] is None
    none = torch.zeros(0, D).cuda()
    got = gla.block_norm_bwd(none, none, none, y=none, post_weight=w, weight=w)
    assert not got[3].any() and not got[6].any() and got[0].shape == (0, D)
    s, u = gla.block_norm_fwd(none, none, weight=w)
    assert s.shape == u.shape == (0, D)


@pytest.mark.parametrize("D", [264, 2048])
def test_block_norm_far_means(gla, D):
    """Layer norm of rows whose mean is 1000 deviations, or that are constant.  The mean is off by
    2^-24 times the row's size for each of some four roundings, relative to the deviation 1."""
    R = 37
    g = torch.Generator().manual_seed(24)
    x = rnd(g, R, D) + 1000.0
    x[::3] = 500.0
    w = torch.ones(D)
    ref = block_ref.block_norm_all(x, None, None, None, None, None, w, None, True, 1e-5)
    _, u = gla.block_norm_fwd(gpu(x), weight=gpu(w), kind="layer")
    # eps = 1e-6 against 1e-5 in ref matters in no row but the constant ones, which are 0 in both
    assert not u[::3].any()
    other = [r for r in range(R) if r % 3]
    err = (u.double().cpu() - ref["u"][0])[other].abs()
    assert float(err.max()) <= 8 * 2 ** -24 * 1000 + 2 ** -17 * 5


# ---------------------------------------------------------------- feed-forward
GLU = [(1, 8, 8), (3, 64, 128), (8, 2048, 264), (129, 72, 136), (256, 256, 128), (257, 520, 392),
       (300, 64, 1352), (777, 136, 264), (1000, 328, 72), (64, 1352, 520),
       # few rows: tiles of 56 features, two blocks an SM, whole and shared K, 128 and 129 rows
       (5, 64, 8192), (9, 72, 12288), (128, 1032, 136), (16, 4104, 72),
       # more tiles than pairs of SMs, tiles of both kinds dealt out unevenly
       (2600, 72, 1352), (20500, 264, 72), (300, 520, 2600), (600, 520, 2600)]


@pytest.mark.parametrize("R,D,F", GLU)
def test_glu(gla, R, D, F):
    g = torch.Generator().manual_seed(19)
    bf = torch.bfloat16
    x, dh = rnd(g, R, D, dtype=bf), rnd(g, R, F, dtype=bf)
    wg, wu = (rnd(g, F, D, std=D ** -0.5, dtype=bf) for _ in range(2))
    ref = block_ref.glu_all(x, wg, wu, dh)
    args = (strided(x), gpu(wg), gpu(wu))
    h = gla.glu_fwd(*args, out_dtype=F32)
    near(h, ref["h"], 1.0, "h")
    check_bf16_rounding(gla.glu_fwd(*args), h)
    grads = gla.glu_bwd(*args, gpu(dh), grad_dtype=F32)
    for n, t in zip(("dx", "dwg", "dwu"), grads):
        near(t, ref[n], 1.0, n)
    for p, q in zip(gla.glu_bwd(*args, gpu(dh)), grads):
        check_bf16_rounding(p, q)
    gla.status_sync()


def test_glu_whole_numbers(gla):
    """Small whole numbers: every product's sum is exact, so a wrong or missing term shows."""
    R, D, F = 300, 392, 264
    g = torch.Generator().manual_seed(20)
    bf = torch.bfloat16
    x = torch.randint(-2, 3, (R, D), generator=g).to(bf)
    wg = torch.zeros(F, D).to(bf)
    wg[torch.arange(F), torch.randint(0, D, (F,), generator=g)] = 1.0   # g: one entry of x
    wu = torch.randint(-2, 3, (F, D), generator=g).to(bf)
    h = gla.glu_fwd(gpu(x), gpu(wg), gpu(wu), out_dtype=F32).double().cpu()
    gg, u = x.double() @ wg.double().t(), x.double() @ wu.double().t()
    want = block_ref.silu(gg) * u
    assert ((h - want).abs() <= 2 ** -20 * want.abs()).all()


def test_glu_rows_are_apart(gla):
    """A row with infinities or NaN leaves the other rows alone; no rows give zero gradients."""
    R, D, F = 140, 72, 200
    g = torch.Generator().manual_seed(21)
    bf = torch.bfloat16
    x, dh = rnd(g, R, D, dtype=bf), rnd(g, R, F, dtype=bf)
    wg, wu = (rnd(g, F, D, std=0.1, dtype=bf).cuda() for _ in range(2))
    a = (gla.glu_fwd(gpu(x), wg, wu), gla.glu_bwd(gpu(x), wg, wu, gpu(dh))[0])
    x[3, 5], x[130, 0] = float("nan"), float("inf")
    b = (gla.glu_fwd(gpu(x), wg, wu), gla.glu_bwd(gpu(x), wg, wu, gpu(dh))[0])
    fine = [r for r in range(R) if r not in (3, 130)]
    for p, q in zip(a, b):
        assert torch.equal(p[fine], q[fine]) and torch.isnan(q[3]).any()
    none = x[:0].cuda()
    assert gla.glu_fwd(none, wg, wu).shape == (0, F)
    dx, dg, du = gla.glu_bwd(none, wg, wu, dh[:0].cuda())
    assert dx.shape == (0, D) and not dg.any() and not du.any()
    gla.status_sync()


def test_glu_wait_that_runs_out(gla):
    """A wait limit of a nanosecond ends the kernel early with GLA_ERR_TIMEOUT; the next call,
    with the default limit, is right.  A barrier test may hold a warp for a time the hardware
    defines, and only a wait that is open still after two tests runs out: the sum over K is so
    long (a tile takes about a millisecond) that the epilogue's wait for it is."""
    g = torch.Generator().manual_seed(22)
    bf = torch.bfloat16
    D = 1 << 18
    x = rnd(g, 256, D, dtype=bf).cuda()
    wg, wu = (rnd(g, 128, D, std=D ** -0.5, dtype=bf).cuda() for _ in range(2))
    want = gla.glu_fwd(x, wg, wu)
    gla.status_sync()
    gla.set_wait_limit_ns(1)
    try:
        hit = False
        for _ in range(20):
            gla.glu_fwd(x, wg, wu)
            try:
                gla.status_sync()
            except gla.GlaError as e:
                assert e.status == 5
                hit = True
                break
        assert hit
    finally:
        gla.set_wait_limit_ns(0)
    assert torch.equal(gla.glu_fwd(x, wg, wu), want)
    gla.status_sync()


# ---------------------------------------------------------------- all of them
def test_offsets_beyond_32_bits(gla):
    """Column slices of a projection of more than 2^31 elements: the last rows and columns."""
    R, wide, D = 70001, 32768, 136
    big = torch.empty(R, wide, dtype=torch.bfloat16, device="cuda")
    cols = [big[:, wide - (k + 1) * D:wide - k * D] for k in range(4)]
    g = torch.Generator(device="cuda").manual_seed(25)
    for c in cols:
        c.normal_(generator=g)
    tight = [c.contiguous() for c in cols]
    dec = -torch.rand(D, generator=g, device="cuda")
    w = torch.ones(D, device="cuda")
    cu = torch.tensor([0, 3, 60000, R], dtype=torch.int32).cuda()
    wg, wu = (torch.randn(72, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    dh = torch.randn(R, 72, generator=g, device="cuda").bfloat16()

    def every(x, f, i, z):
        kw = dict(decay=dec, i=i, z=z, cu_seqlens=cu)
        return [*gla.recur_fwd(x, f, **kw), *gla.recur_bwd(x, f, tight[0], **kw),
                *gla.block_norm_fwd(tight[1], x, z, post_weight=w, weight=w),
                *gla.block_norm_bwd(tight[1], tight[2], tight[0], x, z, post_weight=w, weight=w),
                gla.glu_fwd(x, wg, wu), *gla.glu_bwd(x, wg, wu, dh)]

    for a, b in zip(every(*cols), every(*tight)):
        assert (a is None and b is None) or torch.equal(a, b)
    n = 300
    slots = torch.arange(n, dtype=torch.int32).cuda()
    pools = [torch.zeros(n, D, device="cuda") for _ in range(2)]
    y = [gla.recur_step(c[0][R - n:], c[1][R - n:], p, dec, i=c[2][R - n:], slots=slots)
         for c, p in zip((cols, tight), pools)]
    assert torch.equal(*y) and torch.equal(*pools)
    gla.status_sync()


def test_given_buffers(gla):
    """Outputs, states and workspaces that the caller keeps."""
    x = rnd(torch.Generator().manual_seed(26), 2, 300, 136, dtype=torch.bfloat16).cuda()
    w = torch.ones(136).cuda()
    wg = rnd(torch.Generator().manual_seed(27), 264, 136, dtype=torch.bfloat16).cuda()
    y, fin = gla.recur_fwd(x, x, i=x)
    out, state = torch.empty_like(y), torch.empty_like(fin)
    got = gla.recur_fwd(x, x, i=x, out=out, final_state=state)
    assert got[0] is out and got[1] is state and torch.equal(out, y) and torch.equal(state, fin)
    assert gla.recur_fwd(x, x, i=x, output_final_state=False)[1] is None
    ws = torch.empty(64 << 20, dtype=torch.uint8).cuda()
    for call in (lambda **k: gla.recur_bwd(x, x, x, i=x, **k),
                 lambda **k: gla.block_norm_bwd(x, x, x, x, post_weight=w, weight=w, **k),
                 lambda **k: gla.glu_bwd(x, wg, wg, torch.ones(2, 300, 264).bfloat16().cuda(), **k)):
        want = call()
        ws.fill_(255)  # NaN: whatever is read has been written before
        for a, b in zip(call(workspace=ws), want):
            assert (a is None and b is None) or torch.equal(a, b)
    h = gla.glu_fwd(x, wg, wg)
    buf = torch.empty_like(h)
    assert gla.glu_fwd(x, wg, wg, out=buf) is buf and torch.equal(buf, h)
    s, u = gla.block_norm_fwd(x, x, weight=w)
    s2, u2 = torch.empty_like(s), torch.empty_like(u)
    gla.block_norm_fwd(x, x, weight=w, res_out=s2, out=u2)
    assert torch.equal(s, s2) and torch.equal(u, u2)
    gla.status_sync()


@pytest.mark.parametrize("B,T,D", [(1, 5000, 64), (2, 1000, 136), (1, 17, 8), (3, 260, 72)])
def test_recur_state_in_place_again(gla, B, T, D):
    """The final state written over the initial one, over several blocks of a cluster, repeated."""
    g = torch.Generator().manual_seed(28)
    x, f = rnd(g, B, T, D).cuda(), rnd(g, B, T, D, mean=3.0).cuda()
    init = rnd(g, B, D, std=5.0).cuda()
    want = gla.recur_fwd(x, f, init_state=init)
    for _ in range(20):
        state = init.clone()
        y, fin = gla.recur_fwd(x, f, init_state=state, final_state=state)
        assert torch.equal(y, want[0]) and torch.equal(fin, want[1])


def test_recur_many_short_sequences(gla):
    """A hundred thousand sequences of one to three tokens, packed, and of one token, dense."""
    g = torch.Generator().manual_seed(29)
    D = 64
    lens = torch.randint(0, 4, (100003,), generator=g)
    cu = torch.cat([torch.zeros(1, dtype=torch.long), lens.cumsum(0)])
    R = int(cu[-1])
    x, f, dy = (rnd(g, R, D).cuda() for _ in range(3))
    init, df = rnd(g, 100003, D).cuda(), rnd(g, 100003, D).cuda()
    cug = cu.to(torch.int32).cuda()
    dec = -torch.rand(D, generator=g).cuda()
    y, fin = gla.recur_fwd(x, f, dec, init_state=init, cu_seqlens=cug)
    gr = gla.recur_bwd(x, f, dy, dec, init_state=init, d_final_state=df, cu_seqlens=cug)
    # token by token, over all sequences at once, in 64 bits
    d64 = lambda t: t.double()  # noqa: E731
    _, a, m, _, _ = block_ref.decays(d64(f), d64(dec), True)
    h, e = d64(init), d64(df)
    start = cu[:-1].cuda()
    ln = lens.cuda()
    for t in range(3):
        on = ln > t
        rows = start[on] + t
        h[on] = a[rows] * h[on] + m[rows] * d64(x[rows])
        near(y[rows], (h[on].cpu(), (h[on].abs() + 1).cpu()), 2 ** -17, f"y {t}")
    near(fin, (h.cpu(), (h.abs() + 1).cpu()), 2 ** -17, "final")
    for t in (2, 1, 0):
        on = ln > t
        rows = start[on] + t
        e[on] = e[on] + d64(dy[rows])
        near(gr[0][rows], ((e[on] * m[rows]).cpu(), (e[on].abs() + 1).cpu()), 2 ** -17, f"dx {t}")
        e[on] = a[rows] * e[on]
    near(gr[5], (e.cpu(), (e.abs() + 1).cpu()), 2 ** -17, "d_init")
    dense = gla.recur_fwd(x[:, None], f[:, None], dec)
    step = torch.zeros(R, D).cuda()
    out = gla.recur_step(x, f, step, dec)
    assert torch.allclose(dense[0][:, 0], out, rtol=2 ** -19, atol=1e-6) and torch.equal(out, step)
    gla.status_sync()


# ---------------------------------------------------------------- together
class Layer:
    """norm -> projections -> convolution -> recurrence -> projection -> gate, norm, residual, norm ->
    gated feed-forward, with its gradients, from the library's calls and plain products."""

    def __init__(self, gla, D=128, F=256, seed=23):
        g = torch.Generator().manual_seed(seed)
        bf = torch.bfloat16
        self.gla, self.D = gla, D
        self.w_in = rnd(g, 4 * D, D, std=D ** -0.5, dtype=bf).cuda()
        self.w_out = rnd(g, D, D, std=D ** -0.5, dtype=bf).cuda()
        self.filter = rnd(g, D, 4, std=0.5).cuda()
        self.decay = -torch.rand(D, generator=g).cuda()
        self.n1, self.n2, self.n3, self.scale = ((1 + rnd(g, D, std=0.1)).cuda() for _ in range(4))
        self.wg, self.wu = (rnd(g, F, D, std=D ** -0.5, dtype=bf).cuda() for _ in range(2))
        self.w_down = rnd(g, D, F, std=F ** -0.5, dtype=bf).cuda()

    def __call__(self, res, cu, conv_state, state):
        gla, D = self.gla, self.D
        _, u = gla.block_norm_fwd(res, weight=self.n1, out_dtype=torch.bfloat16)
        p = u @ self.w_in.t()
        x, c1 = gla.conv_fwd(p[..., :D], self.filter, init_state=conv_state, cu_seqlens=cu, activation="silu")
        y, s1 = gla.recur_fwd(x, p[..., D:2 * D], self.decay, i=p[..., 2 * D:3 * D], z=p[..., 3 * D:],
                              init_state=state, cu_seqlens=cu)
        y = y @ self.w_out.t()
        mid, v = gla.block_norm_fwd(res, y, post_weight=self.n2, scale=self.scale, weight=self.n3)
        h = gla.glu_fwd(v, self.wg, self.wu)
        out, _ = gla.block_norm_fwd(mid, h @ self.w_down.t())
        self.kept = (u, p, x, y, mid, v, h)
        return out, c1, s1

    def backward(self, res, cu, conv_state, state, d):
        gla, D = self.gla, self.D
        u, p, x, y, mid, v, h = self.kept
        d_mid, dh = gla.block_norm_bwd(mid, None, d, y=h @ self.w_down.t())[:2]
        dh = dh @ self.w_down
        dv, dwg, dwu = gla.glu_bwd(v, self.wg, self.wu, dh)
        d_res, dy, _, dn2, _, dsc, dn3, _ = gla.block_norm_bwd(
            res, dv, d_mid, y=y, post_weight=self.n2, scale=self.scale, weight=self.n3)
        dy = dy @ self.w_out
        dx, df, dd, di, dz, _ = gla.recur_bwd(x, p[..., D:2 * D], dy, self.decay, i=p[..., 2 * D:3 * D],
                                              z=p[..., 3 * D:], init_state=state, cu_seqlens=cu)
        dp0, dfil, _, _ = gla.conv_bwd(p[..., :D], self.filter, dx, init_state=conv_state, cu_seqlens=cu,
                                       activation="silu")
        du = torch.cat([dp0, df, di, dz], -1) @ self.w_in
        d_in, *_, dn1, _ = gla.block_norm_bwd(res, du, d_res, weight=self.n1)
        return d_in, dfil, dd, dn1, dn2, dn3, dsc, dwg, dwu


def layer_inputs(seed, lens, D):
    g = torch.Generator().manual_seed(seed)
    R, B = sum(lens), len(lens)
    cu = torch.tensor(cu_of(lens), dtype=torch.int32).cuda()
    return (rnd(g, R, D).cuda(), cu, rnd(g, B, 3, D, dtype=torch.bfloat16).cuda(), rnd(g, B, D).cuda(),
            rnd(g, R, D).cuda())


def test_layer_captured_and_replayed(gla):
    """The whole layer and its gradients in one CUDA graph, replayed on new inputs, give the
    eager calls' bits."""
    layer = Layer(gla)
    lens = [33, 0, 100, 1, 250]
    static = layer_inputs(1, lens, layer.D)

    def step(x):
        out = layer(*x[:4])
        return (*out, *layer.backward(*x))

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(static)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = step(static)
    for seed in (2, 3):
        new = layer_inputs(seed, lens, layer.D)
        for a, b in zip(static, new):
            a.copy_(b)
        graph.replay()
        want = step(new)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    gla.status_sync()


def test_layer_from_three_threads(gla):
    """Three host threads on three streams at once give the bits of one after another."""
    sizes = [[300, 20], [1] * 50, [700]]
    layers = [Layer(gla, seed=30 + k) for k in range(3)]
    ins = [layer_inputs(40 + k, sizes[k], layers[k].D) for k in range(3)]
    want = [(*layers[k](*ins[k][:4]), *layers[k].backward(*ins[k])) for k in range(3)]
    torch.cuda.synchronize()
    bad = []

    def work(k):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(10):
                got = (*layers[k](*ins[k][:4]), *layers[k].backward(*ins[k]))
                stream.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[k])):
                    bad.append(k)

    ts = [threading.Thread(target=work, args=(k,)) for k in range(3)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert not bad
    gla.status_sync()


def test_same_bits_again(gla):
    """Every call gives the same bits each time (no atomics decide a value)."""
    x = recur_inputs([500, 1, 900], 264, "bf16", True, True, True, True, 50)
    cu = torch.tensor([0, 500, 501, 1401], dtype=torch.int32).cuda()
    args = [gpu(x[n]) for n in ("x", "f")]
    kw = dict(decay=gpu(x["decay"]), i=gpu(x["i"]), z=gpu(x["z"]), init_state=gpu(x["init"]), cu_seqlens=cu)
    w = torch.ones(264).cuda()
    wg = gpu(rnd(torch.Generator().manual_seed(51), 392, 264, dtype=torch.bfloat16))
    dh = gpu(rnd(torch.Generator().manual_seed(52), 1401, 392, dtype=torch.bfloat16))
    first = None
    for _ in range(8):
        got = [*gla.recur_fwd(*args, **kw), *gla.recur_bwd(*args, gpu(x["dy"]), **kw),
               *gla.block_norm_bwd(args[0], args[1], args[1], y=args[0], post_weight=w, weight=w),
               *gla.glu_bwd(args[0], wg, wg, dh)]
        first = first or got
        for a, b in zip(first, got):
            assert (a is None and b is None) or torch.equal(a, b)
    gla.status_sync()


def test_streams(gla):
    """A call on a stream given by argument, its results used there."""
    x = rnd(torch.Generator().manual_seed(60), 64, 128, dtype=torch.bfloat16).cuda()
    w = torch.ones(128).cuda()
    wg = rnd(torch.Generator().manual_seed(61), 136, 128, dtype=torch.bfloat16).cuda()
    want = (gla.glu_fwd(x, wg, wg), gla.block_norm_fwd(x, x, weight=w)[1], gla.recur_fwd(x[None], x[None])[0])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = (gla.glu_fwd(x, wg, wg, stream=s), gla.block_norm_fwd(x, x, weight=w, stream=s)[1],
           gla.recur_fwd(x[None], x[None], stream=s)[0])
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("captured", [False, True])
def test_calls_behind_another_stream(gla, captured):
    """A call on what a slow kernel of another stream writes waits for it, right behind a launch
    that lets the next one start early, eagerly and captured."""
    g = torch.Generator().manual_seed(62)
    R, D = 96, 128
    src = rnd(g, R, D, dtype=torch.bfloat16).cuda()
    w, decay = torch.ones(D).cuda(), -torch.rand(D, generator=g).cuda()
    wg, wu = (rnd(g, D, D, std=D ** -0.5, dtype=torch.bfloat16).cuda() for _ in range(2))
    big = rnd(g, 4096, 4096, std=4096 ** -0.5, dtype=torch.bfloat16).cuda()
    state0 = rnd(g, R, D).cuda()
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    inputs = [torch.zeros_like(src) for _ in range(4)]

    def late(x):  # x holds src once the side stream has come that far
        x.zero_()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            t = big
            for _ in range(8):
                t = t @ big
            x.copy_(src)
        main.wait_stream(side)

    def run(wait):
        state = state0.clone()
        f = gla.glu_fwd(src, wg, wu)
        wait(inputs[0])
        y = gla.recur_fwd(inputs[0][None], f[None], decay)[0][0]
        wait(inputs[1])
        s, u = gla.block_norm_fwd(inputs[1], y, weight=w)
        wait(inputs[2])
        h = gla.glu_fwd(inputs[2], wg, wu)
        wait(inputs[3])
        t = gla.recur_step(inputs[3], h, state, decay)
        return y, s, u, h, t, state

    want = run(lambda x: x.copy_(src))
    torch.cuda.synchronize()
    if captured:
        with torch.cuda.stream(main):
            run(late)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=main):
            got = run(late)
        for _ in range(3):
            graph.replay()
    else:
        with torch.cuda.stream(main):
            for _ in range(3):
                got = run(late)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    gla.status_sync()
