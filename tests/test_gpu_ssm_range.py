"""The selective scan and the causal convolution over the rest of their documented range,
against the plain 64-bit implementations.

Tolerances as in test_gpu_ssm, per element, as parts of the same sum over the
absolute values of its terms (its decays as they are, so that growth is in it).
"""
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
