"""The causal convolution and the selective scan on the GPU against plain 64-bit
implementations (tests/ssm_ref.py): prompts, gradients, single tokens.

Tolerances, per element, are multiples of the same sum over the absolute values
of its terms (``ssm_ref`` with ``absolute=True``), which is what fp32 rounding
errors scale with:
  convolution: at most W + 1 = 5 products and sums, a sigmoid (hardware
      exponential 2^-22, its argument 2^-24 |p|, division 2^-22; |p| < 16 here)
      and its product: below 5 * 2^-24 + 2^-21 + 16 * 2^-24 + 4 * 2^-24 < 2^-18.
  scan: a decay is off by 2^-22 (hardware exponential) and 2^-24 times its
      exponent (|delta a| < 4 here: below 2^-21 together), each step adds one
      rounding, and the step size is off by a few 2^-24 (bf16 rows:
      and by |dt + bias| 2^-24), also in every exponent: below 2^-20 per step, over
      the steps that a state remembers, at most min(T, 1 / (1 - slowest decay));
      2^-17 covers the products, the sums over n and the gate around them.  Gradients run two such recurrences.
bf16 results are required to be the fp32 results rounded once (half a step).
"""
import pytest
import torch

import ssm_ref
from parity import check_bf16_rounding

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def gla():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_linear_attention_gla_gb300 import build as glabuild
    glabuild.build()
    import gated_linear_attention_gla_gb300 as m
    return m


def rnd(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def cu_of(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def gpu(t):
    return None if t is None else t.cuda()


def near(got, ref, size, factor, what):
    """|got - ref| <= factor * size, element by element."""
    err = (got.detach().double().cpu() - ref).abs()
    bad = err > factor * size + 1e-30
    assert not bad.any() and not torch.isnan(err).any(), \
        f"{what}: off by {float((err / (size + 1e-30)).max()):.3g} of its terms, allowed {factor:.3g}"


# (lens, packed): one token, shorter than the filter, empty sequences, runs that end
# inside tiles of 32 and 256 rows, sequences that start inside them
LENS = [([1], True), ([2], False), ([0, 3, 0, 1, 70, 0], True), ([33, 33], False),
        ([31, 1, 32, 2, 255, 3, 257], True), ([64] * 5, False), ([1] * 40, True)]


def conv_inputs(lens, D, W, io, seed, wide=0):
    g = torch.Generator().manual_seed(seed)
    cu, R, B = cu_of(lens), sum(lens), len(lens)
    dt = DT[io]
    return dict(x=rnd(g, R, D + wide, dtype=dt)[:, wide // 2:wide // 2 + D], w=rnd(g, D, W, std=0.5),
                bias=rnd(g, D), init=rnd(g, B, W - 1, D, dtype=dt), dy=rnd(g, R, D, dtype=dt),
                df=rnd(g, B, W - 1, D)), cu


def lead(t, lens, packed):
    return t if packed else t.reshape(len(lens), lens[0], *t.shape[1:])


def strided(t, device="cuda"):
    """The same rows, as columns of a wider tensor on the GPU."""
    wide = torch.full((*t.shape[:-1], t.shape[-1] + 32), 7.0, dtype=t.dtype, device=device)
    wide[..., 16:-16] = t.to(device)
    return wide[..., 16:-16]


@pytest.mark.parametrize("lens,packed", LENS)
@pytest.mark.parametrize("io,D,W,act,bias,init", [
    ("bf16", 264, 4, "silu", True, True), ("fp32", 136, 4, None, False, True),
    ("bf16", 8, 3, None, True, False), ("fp32", 1032, 2, "silu", True, False),
    ("bf16", 2048, 2, "silu", False, True)])
def test_conv(gla, lens, packed, io, D, W, act, bias, init):
    x, cu = conv_inputs(lens, D, W, io, 5)
    b, st = x["bias"] if bias else None, x["init"] if init else None
    ref = ssm_ref.conv(x["x"], x["w"], b, st, cu, act, x["dy"], x["df"])
    size = ssm_ref.conv(x["x"], x["w"], b, st, cu, act, x["dy"], x["df"], absolute=True)
    cu_gpu = torch.tensor(cu, dtype=torch.int32).cuda() if packed else None
    xs = strided(lead(x["x"], lens, packed))
    args = (xs, gpu(x["w"]), gpu(b))
    kw = dict(init_state=gpu(st), cu_seqlens=cu_gpu, activation=act)
    y, fin = gla.conv_fwd(*args, **kw, out_dtype=torch.float32)
    near(y.reshape(ref["y"].shape), ref["y"], size["y"], 2 ** -18, "y")
    assert torch.equal(fin.double().cpu(), ref["final"])
    if io == "bf16":
        y16, _ = gla.conv_fwd(*args, **kw)
        check_bf16_rounding(y16, y)
    if init:  # the state updated in place
        state = gpu(st).clone()
        y2, fin2 = gla.conv_fwd(*args, **{**kw, "init_state": state}, final_state=state,
                                out_dtype=torch.float32)
        assert torch.equal(y2, y) and torch.equal(fin2, fin) and fin2 is state
    grads = {}
    for gd in {DT[io], torch.float32}:
        grads[gd] = gla.conv_bwd(xs, gpu(x["w"]), gpu(lead(x["dy"], lens, packed)), gpu(b), **kw,
                                 d_final_state=gpu(x["df"]), grad_dtype=gd)
    dx, dw, db, di = grads[torch.float32]
    # dp has the forward's error once more, a product with dy, and W sums
    R = max(1, sum(lens))
    near(dx.reshape(ref["dx"].shape), ref["dx"], size["dx"], 2 ** -17, "dx")
    near(di, ref["d_init"], size["d_init"], 2 ** -17, "d_init")
    near(dw, ref["dw"], size["dw"], 2 ** -17 + R * 2 ** -24, "dw")
    if bias:
        near(db, ref["db"], size["db"], 2 ** -17 + R * 2 ** -24, "db")
    else:
        assert db is None
    if io == "bf16":
        check_bf16_rounding(grads[DT[io]][0], dx)
        assert all(torch.equal(p, q) for p, q in zip(grads[DT[io]][1:], grads[torch.float32][1:])
                   if p is not None)
    gla.status_sync()


@pytest.mark.parametrize("io,W,act", [("bf16", 4, "silu"), ("fp32", 3, None), ("bf16", 2, "silu")])
def test_conv_long_runs(gla, io, W, act):
    """Enough rows that a thread's run is tens of rows and holds whole groups inside
    sequences, their starts and ends at every place of a group, and empty ones."""
    lens = [1, 0, 2, 3, 4, 0, 0, 5, 6, 7, 8, 9, 10, 11, 700, 13, 37, 1, 1, 1, 1500, 2, 0, 41, 1023, 3, 0]
    D = 2048
    x, cu = conv_inputs(lens, D, W, io, 6)
    ref = ssm_ref.conv(x["x"], x["w"], x["bias"], x["init"], cu, act, x["dy"], x["df"])
    size = ssm_ref.conv(x["x"], x["w"], x["bias"], x["init"], cu, act, x["dy"], x["df"], absolute=True)
    args = (strided(x["x"]), gpu(x["w"]))
    kw = dict(init_state=gpu(x["init"]), cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(),
              activation=act)
    y, fin = gla.conv_fwd(*args, gpu(x["bias"]), **kw, out_dtype=torch.float32)
    near(y, ref["y"], size["y"], 2 ** -18, "y")
    assert torch.equal(fin.double().cpu(), ref["final"])
    dx, dw, db, di = gla.conv_bwd(*args, gpu(x["dy"]), gpu(x["bias"]), **kw,
                                  d_final_state=gpu(x["df"]), grad_dtype=torch.float32)
    R = sum(lens)
    near(dx, ref["dx"], size["dx"], 2 ** -17, "dx")
    near(di, ref["d_init"], size["d_init"], 2 ** -17, "d_init")
    near(dw, ref["dw"], size["dw"], 2 ** -17 + R * 2 ** -24, "dw")
    near(db, ref["db"], size["db"], 2 ** -17 + R * 2 ** -24, "db")
    gla.status_sync()


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("N,D,W", [(1, 8, 2), (5, 520, 4), (64, 2048, 3)])
def test_conv_step_continues_the_prompt(gla, io, N, D, W):
    """Steps equal the prompt's last rows, dense and through slots, in place and onto other pages."""
    x, cu = conv_inputs([9] * N, D, W, io, 6)
    ref = ssm_ref.conv(x["x"], x["w"], x["bias"], None, cu, True)
    size = ssm_ref.conv(x["x"], x["w"], x["bias"], None, cu, True, absolute=True)
    rows = x["x"].reshape(N, 9, D)
    w, b = gpu(x["w"]), gpu(x["bias"])
    _, state = gla.conv_fwd(gpu(rows[:, :6].contiguous()), w, b, activation="silu")
    pool = torch.full((2 * N + 1, W - 1, D), 9.0, dtype=DT[io], device="cuda")
    g = torch.Generator().manual_seed(1)
    order = torch.randperm(2 * N + 1, generator=g).to(torch.int32)
    slots, other = gpu(order[:N]).contiguous(), gpu(order[N:2 * N]).contiguous()
    pool[slots.long()] = state
    spare = int(order[2 * N])
    for t in range(6, 9):
        xt = strided(rows[:, t])
        old = pool[slots.long()].clone()
        y2 = gla.conv_step(xt, w, pool, b, activation="silu", slots=slots, out_slots=other,
                           out_dtype=torch.float32)
        assert torch.equal(pool[slots.long()], old)
        y = gla.conv_step(xt, w, state, b, activation="silu", out_dtype=torch.float32)
        slots, other = other, slots
        assert torch.equal(y, y2) and torch.equal(pool[slots.long()], state)
        near(y, ref["y"].reshape(N, 9, D)[:, t], size["y"].reshape(N, 9, D)[:, t], 2 ** -18, f"y{t}")
        if io == "bf16":
            y16 = gla.conv_step(xt, w, pool, b, activation="silu", slots=other, out_slots=slots)
            check_bf16_rounding(y16, y)
    assert torch.equal(state.double().cpu(), ref["final"])
    assert (pool[spare] == 9.0).all()
    gla.status_sync()


def scan_inputs(lens, D, N, io, seed, dt_std=0.5, softplus=True):
    g = torch.Generator().manual_seed(seed)
    cu, R, B = cu_of(lens), sum(lens), len(lens)
    ty = DT[io]
    delta = torch.exp(torch.rand(D, generator=g) * 4.6 - 6.9)   # 1e-3 .. 1e-1
    dt = rnd(g, R, D, std=dt_std, dtype=ty) if softplus else (torch.rand(R, D, generator=g) * 0.1).to(ty)
    return dict(u=rnd(g, R, D, dtype=ty), dt=dt,
                a=-torch.arange(1, N + 1).float() * (0.1 + torch.rand(D, N, generator=g)),
                b=rnd(g, R, N, dtype=ty), c=rnd(g, R, N, dtype=ty), skip=rnd(g, D),
                z=rnd(g, R, D, dtype=ty), bias=delta + torch.log(-torch.expm1(-delta)),
                init=rnd(g, B, D, N), dy=rnd(g, R, D, dtype=ty), df=rnd(g, B, D, N)), cu


def scan_factor(x, cu, softplus, gradients=False):
    """The tolerance of the file's head: 2^-20 per remembered step."""
    T = max(b - a for a, b in zip(cu, cu[1:]))
    d = x["dt"].double() + (x["bias"].double() if x["bias"] is not None else 0)
    d = torch.log1p(torch.exp(d)) if softplus else d
    slowest = float((d.mean(0) * x["a"].double().abs().amin(1)).min()) if d.numel() else 1.0
    steps = min(T, 1 / max(1e-4, slowest))
    return (2 if gradients else 1) * (steps * 2 ** -20 + 2 ** -17)


SCAN_LENS = [([1], True), ([5], False), ([0, 3, 0, 1, 70, 0], True), ([33, 33], False),
             ([63, 1, 64, 2, 129, 65], True), ([130], False)]
SCAN_CASES = [("bf16", 136, 16, True, True, True, True), ("fp32", 64, 16, False, True, False, True),
              ("fp32", 40, 8, True, False, True, True), ("bf16", 72, 32, False, False, False, False),
              ("bf16", 24, 64, True, True, True, True), ("fp32", 8, 64, True, False, False, False)]


@pytest.mark.parametrize("lens,packed", SCAN_LENS)
@pytest.mark.parametrize("io,D,N,z,skip,init,softplus", SCAN_CASES)
def test_scan(gla, lens, packed, io, D, N, z, skip, init, softplus):
    x, cu = scan_inputs(lens, D, N, io, 7, softplus=softplus)
    if not softplus:
        x["bias"] = None
    for name, keep in (("z", z), ("skip", skip), ("init", init)):
        if not keep:
            x[name] = None
    order = ("u", "dt", "a", "b", "c", "skip", "z", "bias")
    more = (softplus, x["init"], cu, x["dy"], x["df"] if init else None)
    ref = ssm_ref.scan(*[x[k] for k in order], *more)
    size = ssm_ref.scan(*[x[k] for k in order], *more, absolute=True)
    cu_gpu = torch.tensor(cu, dtype=torch.int32).cuda() if packed else None
    L = lambda t: None if t is None else strided(lead(t, lens, packed))  # noqa: E731
    args = (L(x["u"]), L(x["dt"]), gpu(x["a"]), L(x["b"]), L(x["c"]))
    kw = dict(skip=gpu(x["skip"]), z=L(x["z"]), dt_bias=gpu(x["bias"]), softplus=softplus,
              init_state=gpu(x["init"]), cu_seqlens=cu_gpu)
    f = scan_factor(x, cu, softplus)
    y, fin = gla.scan_fwd(*args, **kw, out_dtype=torch.float32)
    near(y.reshape(ref["y"].shape), ref["y"], size["y"], f, "y")
    near(fin, ref["final"], size["final"], f, "final")
    if io == "bf16":
        y16, fin16 = gla.scan_fwd(*args, **kw)
        check_bf16_rounding(y16, y)
        assert torch.equal(fin16, fin)
    if init:
        state = gpu(x["init"]).clone()
        y2, _ = gla.scan_fwd(*args, **{**kw, "init_state": state}, final_state=state,
                             out_dtype=torch.float32)
        assert torch.equal(y2, y) and torch.equal(state, fin)
    f = scan_factor(x, cu, softplus, gradients=True) + max(1, sum(lens)) * 2 ** -24
    names = ("du", "ddt", "da", "db", "dc", "dskip", "dz", "dbias", "d_init")
    grads = {}
    for gd in {DT[io], torch.float32}:
        got = gla.scan_bwd(*args, gpu(lead(x["dy"], lens, packed)), **kw,
                           d_final_state=gpu(x["df"]) if init else None, grad_dtype=gd)
        grads[gd] = dict(zip(names, got))
    for k in names:
        got = grads[torch.float32][k]
        if ref[k] is None:
            assert got is None, k
            continue
        near(got.reshape(ref[k].shape), ref[k], size[k], f, k)
        if io == "bf16":
            low = grads[torch.bfloat16][k]
            if low.dtype == torch.bfloat16:
                check_bf16_rounding(low, got)
            else:
                assert torch.equal(low, got), k
    gla.status_sync()


@pytest.mark.parametrize("io,R,D,N", [("bf16", 1, 8, 16), ("fp32", 3, 72, 8), ("bf16", 9, 520, 16),
                                      ("bf16", 6, 40, 32), ("fp32", 5, 24, 64)])
def test_scan_step_continues_the_prompt(gla, io, R, D, N):
    T = 12
    x, cu = scan_inputs([T] * R, D, N, io, 8)
    order = ("u", "dt", "a", "b", "c", "skip", "z", "bias")
    ref = ssm_ref.scan(*[x[k] for k in order], True, x["init"], cu)
    size = ssm_ref.scan(*[x[k] for k in order], True, x["init"], cu, absolute=True)
    f = scan_factor(x, cu, True)
    rows = {k: x[k].reshape(R, T, -1) for k in ("u", "dt", "b", "c", "z")}
    head = {k: gpu(v[:, :8].contiguous()) for k, v in rows.items()}
    kw = dict(skip=gpu(x["skip"]), dt_bias=gpu(x["bias"]))
    a = gpu(x["a"])
    _, state = gla.scan_fwd(head["u"], head["dt"], a, head["b"], head["c"], z=head["z"],
                            init_state=gpu(x["init"]), **kw)
    pool = torch.full((2 * R + 1, D, N), 9.0, device="cuda")
    perm = torch.randperm(2 * R + 1, generator=torch.Generator().manual_seed(2)).to(torch.int32)
    slots, other = gpu(perm[:R]).contiguous(), gpu(perm[R:2 * R]).contiguous()
    pool[slots.long()] = state
    for t in range(8, T):
        s = {k: strided(v[:, t]) for k, v in rows.items()}
        args = (s["u"], s["dt"], a, s["b"], s["c"])
        old = pool[slots.long()].clone()
        y2 = gla.scan_step(*args, pool, z=s["z"], slots=slots, out_slots=other,
                           out_dtype=torch.float32, **kw)
        assert torch.equal(pool[slots.long()], old)
        if io == "bf16":
            y16 = gla.scan_step(*args, state.clone(), z=s["z"], **kw)
            check_bf16_rounding(y16, y2)
        y = gla.scan_step(*args, state, z=s["z"], out_dtype=torch.float32, **kw)
        slots, other = other, slots
        assert torch.equal(y, y2) and torch.equal(pool[slots.long()], state)
        near(y, ref["y"].reshape(R, T, D)[:, t], size["y"].reshape(R, T, D)[:, t], f, f"y{t}")
    near(state, ref["final"], size["final"], f, "state")
    assert (pool[int(perm[2 * R])] == 9.0).all()
    gla.status_sync()


def test_step_rows_that_do_nothing(gla):
    """-1 in either table: no page and no output is touched; a page outside the pool is reported."""
    D, N, W = 64, 16, 4
    g = torch.Generator().manual_seed(9)
    u = gpu(rnd(g, 5, D, dtype=torch.bfloat16))
    bc = gpu(rnd(g, 5, N, dtype=torch.bfloat16))
    a = -torch.ones(D, N, device="cuda")
    w = torch.ones(D, W, device="cuda")
    slots = torch.tensor([2, -1, 0, 3, 1], dtype=torch.int32, device="cuda")
    outs = torch.tensor([2, 4, -1, 5, 1], dtype=torch.int32, device="cuda")
    for step, pool in ((lambda p, o, s, t: gla.scan_step(u, u, a, bc, bc, p, slots=s, out_slots=t, out=o),
                        torch.randn(6, D, N, device="cuda")),
                       (lambda p, o, s, t: gla.conv_step(u, w, p, slots=s, out_slots=t, out=o),
                        torch.randn(6, W - 1, D, device="cuda").to(torch.bfloat16))):
        before, out = pool.clone(), torch.full((5, D), 7.0, dtype=torch.bfloat16, device="cuda")
        step(pool, out, slots, outs)
        gla.status_sync()
        assert (out[1:3] == 7.0).all() and not (out[0] == 7.0).all()
        assert torch.equal(pool[[0, 3, 4]], before[[0, 3, 4]])
        assert not torch.equal(pool[2], before[2]) and not torch.equal(pool[5], before[5])
        before = pool.clone()
        bad = slots.clone()
        bad[0] = 6
        with pytest.raises(gla.GlaError):
            step(pool, out, bad, None)
            gla.status_sync()
        assert torch.equal(pool[2], before[2])
        gla.status_sync()


def test_malformed_offsets_are_reported(gla):
    D, N = 64, 16
    x = torch.randn(64, D, device="cuda").to(torch.bfloat16)
    bc = x[:, :N].contiguous()
    a, w = -torch.ones(D, N, device="cuda"), torch.ones(D, 4, device="cuda")
    for cu in ([0, 70, 64], [3, 20, 64], [0, 20, 60], [0, 40, 20, 64], [0, -5, 64]):
        c = torch.tensor(cu, dtype=torch.int32, device="cuda")
        for call in (lambda: gla.conv_fwd(x, w, cu_seqlens=c), lambda: gla.conv_bwd(x, w, x, cu_seqlens=c),
                     lambda: gla.scan_fwd(x, x, a, bc, bc, cu_seqlens=c),
                     lambda: gla.scan_bwd(x, x, a, bc, bc, x, cu_seqlens=c)):
            with pytest.raises(gla.GlaError) as e:
                call()
                gla.status_sync()
            assert e.value.status == 1, cu
    gla.status_sync()


def test_extreme_step_sizes(gla):
    """dt of -100 (no step), +100 (the step itself), and a decay that erases the state."""
    D, N = 8, 16
    dt = torch.tensor([-100.0, 0.0, 100.0, -20.0, 20.0, 88.0, -88.0, 1e-3]).repeat(D, 1).t().contiguous()
    u = torch.ones(8, D)
    bc = torch.ones(8, N)
    a = -torch.arange(1, N + 1).float().repeat(D, 1)
    init = torch.ones(1, D, N)
    ref = ssm_ref.scan(u, dt, a, bc, bc, None, None, None, True, init, [0, 8])
    size = ssm_ref.scan(u, dt, a, bc, bc, None, None, None, True, init, [0, 8], absolute=True)
    y, fin = gla.scan_fwd(gpu(u)[None], gpu(dt)[None], gpu(a), gpu(bc)[None], gpu(bc)[None],
                          init_state=gpu(init))
    # exponents up to 16 * 100: their rounding moves a decay by 2^-24 * |exponent|, but
    # exp(-x) x <= 1/e of the state it multiplies
    near(y[0], ref["y"], size["y"], 2 ** -16, "y")
    near(fin, ref["final"], size["final"], 2 ** -16, "final")


def test_layer_in_training_and_serving(gla):
    """conv, scan and their gradients in a row as a layer uses them, packed; then the same
    tokens through the prompt form in two pieces and the single-token forms on pools."""
    D, N, W = 128, 16, 4
    lens = [40, 7, 25]
    cu = cu_of(lens)
    R = sum(lens)
    g = torch.Generator().manual_seed(12)
    bf = torch.bfloat16
    xz = gpu(rnd(g, R, 2 * D, dtype=bf))
    proj = gpu(rnd(g, R, D + 2 * N, std=0.5, dtype=bf))
    w, wb = gpu(rnd(g, D, W, std=0.4)), gpu(rnd(g, D))
    a = gpu(-torch.arange(1, N + 1).float() * (0.5 + torch.rand(D, N, generator=g)))
    skip, bias = gpu(rnd(g, D)), gpu(rnd(g, D) - 4)
    cu_gpu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    x, z = xz[:, :D], xz[:, D:]
    dt, b, c = proj[:, :D], proj[:, D:D + N], proj[:, D + N:]
    u, conv_state = gla.conv_fwd(x, w, wb, cu_seqlens=cu_gpu, activation="silu")
    y, state = gla.scan_fwd(u, dt, a, b, c, skip=skip, z=z, dt_bias=bias, cu_seqlens=cu_gpu)
    dy = gpu(rnd(g, R, D, dtype=bf))
    grads = gla.scan_bwd(u, dt, a, b, c, dy, skip=skip, z=z, dt_bias=bias, cu_seqlens=cu_gpu)
    dx, dw, db, _ = gla.conv_bwd(x, w, grads[0], wb, cu_seqlens=cu_gpu, activation="silu")
    gla.status_sync()
    # against the references fed with the same (bf16) intermediates
    uc = ssm_ref.conv(x, w, wb, None, cu, True, grads[0])
    ua = ssm_ref.conv(x, w, wb, None, cu, True, grads[0], absolute=True)
    near(u, uc["y"], ua["y"] * 1.0, 2 ** -8 + 2 ** -18, "u")      # bf16 result
    near(dx, uc["dx"], ua["dx"], 2 ** -8 + 2 ** -17, "dx")
    near(dw, uc["dw"], ua["dw"], 2 ** -17 + R * 2 ** -24, "dw")
    sc = ssm_ref.scan(u, dt, a, b, c, skip, z, bias, True, None, cu, dy)
    sa = ssm_ref.scan(u, dt, a, b, c, skip, z, bias, True, None, cu, dy, absolute=True)
    near(y, sc["y"], sa["y"], 2 ** -8 + 2 ** -13, "y")
    near(grads[0], sc["du"], sa["du"], 2 ** -8 + 2 ** -12, "du")
    near(grads[2], sc["da"], sa["da"], 2 ** -12, "da")
    # serving: a prompt of all but two tokens, then two single tokens, on pools
    pages = gla.fork_pages([], torch.zeros(8, dtype=torch.int32, device="cuda"),
                           torch.full((3,), gla.PAGE_NEW, dtype=torch.int32, device="cuda"))[0]
    conv_pool = torch.zeros(8, W - 1, D, dtype=bf, device="cuda")
    scan_pool = torch.zeros(8, D, N, device="cuda")
    keep = torch.cat([torch.arange(p, q - 2) for p, q in zip(cu, cu[1:])]).cuda()
    short = torch.tensor(cu_of([n - 2 for n in lens]), dtype=torch.int32, device="cuda")
    u1, cs = gla.conv_fwd(x[keep], w, wb, cu_seqlens=short, activation="silu")
    assert torch.equal(u1, u[keep])
    _, ss = gla.scan_fwd(u1, dt[keep], a, b[keep], c[keep], skip=skip, z=z[keep], dt_bias=bias,
                         cu_seqlens=short)
    conv_pool[pages.long()], scan_pool[pages.long()] = cs, ss
    for back in (2, 1):
        at = torch.tensor([q - back for q in cu[1:]], device="cuda")
        ut = gla.conv_step(x[at], w, conv_pool, wb, activation="silu", slots=pages)
        assert torch.equal(ut, u[at])
        yt = gla.scan_step(ut, dt[at], a, b[at], c[at], scan_pool, skip=skip, z=z[at],
                           dt_bias=bias, slots=pages)
        near(yt, sc["y"][at.cpu()], sa["y"][at.cpu()], 2 ** -8 + 2 ** -13, "token")
    assert torch.equal(conv_pool[pages.long()], conv_state)
    near(scan_pool[pages.long()], sc["final"], sa["final"], 2 ** -13, "state")
    gla.status_sync()


def test_captured_and_on_another_stream(gla):
    """A captured forward, backward and step replay on new inputs; a call on a given stream."""
    D, N = 128, 16
    x, cu = scan_inputs([50, 30], D, N, "bf16", 13)
    t = {k: gpu(v) for k, v in x.items()}
    cu_gpu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    w = torch.randn(D, 4, device="cuda")

    def layer(stream=None):
        u, _ = gla.conv_fwd(t["u"], w, cu_seqlens=cu_gpu, activation="silu", stream=stream)
        y, fin = gla.scan_fwd(u, t["dt"], t["a"], t["b"], t["c"], skip=t["skip"], z=t["z"],
                              dt_bias=t["bias"], cu_seqlens=cu_gpu, stream=stream)
        g = gla.scan_bwd(u, t["dt"], t["a"], t["b"], t["c"], t["dy"], skip=t["skip"], z=t["z"],
                         dt_bias=t["bias"], cu_seqlens=cu_gpu, stream=stream)
        dx = gla.conv_bwd(t["u"], w, g[0], cu_seqlens=cu_gpu, activation="silu", stream=stream)
        return [u, y, fin, *g, *[v for v in dx if v is not None]]

    side = torch.cuda.Stream()
    first = layer()
    torch.cuda.synchronize()
    other = layer(side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = layer()
    t["u"].copy_(t["u"].flip(0))
    t["dt"].mul_(0.5)
    graph.replay()
    fresh = layer()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(held, fresh))
    assert not torch.equal(first[1], fresh[1])
    gla.status_sync()


def test_large_ragged_calls_are_exact_and_repeatable(gla):
    """Full-size packed calls (thousands of blocks in flight): every convolution output
    equals the one computed sequence by sequence, and all operators give the
    same bits five times over."""
    g = torch.Generator(device="cuda").manual_seed(21)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    lens = [1, 0, 7894, 1556, 1186, 571, 11851, 1755, 963, 4023, 38, 3141, 494, 2, 3, 33]
    R, D, N, W = sum(lens), 2048, 16, 4
    cu = cu_of(lens)
    cu_gpu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    x, dy, bc = r(R, 2 * D)[:, :D], r(R, D), r(R, 2 * N)
    w, bias = torch.randn(D, W, generator=g, device="cuda"), torch.randn(D, generator=g, device="cuda")
    init = r(len(lens), W - 1, D)
    a = -torch.rand(D, N, generator=g, device="cuda") * 8 - 0.1
    dt = (r(R, D) - 4).contiguous()

    def everything():
        y, f = gla.conv_fwd(x, w, bias, init_state=init, cu_seqlens=cu_gpu, activation="silu")
        dx = gla.conv_bwd(x, w, dy, bias, init_state=init, cu_seqlens=cu_gpu, activation="silu")
        o, h = gla.scan_fwd(y, dt, a, bc[:, :N], bc[:, N:], z=x, cu_seqlens=cu_gpu)
        grads = gla.scan_bwd(y, dt, a, bc[:, :N], bc[:, N:], dy, z=x, cu_seqlens=cu_gpu)
        return [y, f, *dx, o, h, *[t for t in grads if t is not None]]

    first = everything()
    for _ in range(4):
        assert all(torch.equal(p, q) for p, q in zip(first, everything()))
    for i, (lo, hi) in enumerate(zip(cu, cu[1:])):
        y, f = gla.conv_fwd(x[lo:hi][None], w, bias, init_state=init[i:i + 1], activation="silu")
        assert torch.equal(y[0], first[0][lo:hi]) and torch.equal(f[0], first[1][i])
    # and the last rows of every sequence against the definition
    for i, (lo, hi) in enumerate(zip(cu, cu[1:])):
        seq = torch.cat([init[i], x[lo:hi]]).double()[-(W + 7):]
        k = seq.shape[0] - W + 1
        p = bias.double() + sum(w[:, j].double() * seq[j:j + k] for j in range(W))
        if hi > lo:
            n = min(k, hi - lo)
            err = (first[0][hi - n:hi].double() - (p / (1 + torch.exp(-p)))[-n:]).abs()
            assert float((err - (2 ** -8 + 2 ** -18) * p[-n:].abs()).max()) < 1e-5
    gla.status_sync()
