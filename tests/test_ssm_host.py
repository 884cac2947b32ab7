"""The selective-scan and page entry points on the host: bad arguments are rejected
before anything touches the GPU, empty calls do nothing, and the tests' own
64-bit gradients agree with finite differences (CPU only)."""
import ctypes
import re

import pytest
import torch

import ssm_ref
from gated_linear_attention_gla_gb300 import _binding, build as glabuild
from test_abi_host import HEADER

E = _binding
A = 1 << 20
P = [A * (i + 1) for i in range(40)]  # fake, aligned, never dereferenced


@pytest.fixture(scope="module")
def L():
    glabuild.build()
    return _binding.lib()


def test_ctypes_signatures_match_header(L):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    for name in ("gla_conv_fwd", "gla_conv_bwd", "gla_conv_bwd_workspace_size", "gla_conv_step",
                 "gla_scan_fwd", "gla_scan_fwd_workspace_size", "gla_scan_bwd",
                 "gla_scan_bwd_workspace_size", "gla_scan_step", "gla_pages_copy",
                 "gla_pages_fork", "gla_pages_compact", "gla_pages_free"):
        params = re.search(name + r"\s*\(([^)]*)\)", text).group(1).split(",")
        assert len(getattr(L, name).argtypes) == len(params), name


def conv_fwd(L, **kw):
    a = dict(x=P[0], xs=64, w=P[1], b=P[2], init=P[3], out=P[4], fin=P[5], cu=None, B=2, T=16,
             D=64, W=4, flags=0)
    a.update(kw)
    return L.gla_conv_fwd(a["x"], a["xs"], a["w"], a["b"], a["init"], a["out"], a["fin"], a["cu"],
                          a["B"], a["T"], a["D"], a["W"], None, a["flags"])


@pytest.mark.parametrize("kw,status", [
    (dict(flags=E.GLA_FLAG_VECTOR_GATE), E.GLA_ERR_INVALID_ARG),
    (dict(flags=E.GLA_FLAG_SOFTPLUS), E.GLA_ERR_INVALID_ARG),
    (dict(B=-1), E.GLA_ERR_INVALID_ARG), (dict(T=-1), E.GLA_ERR_INVALID_ARG),
    (dict(W=1), E.GLA_ERR_UNSUPPORTED), (dict(W=5), E.GLA_ERR_UNSUPPORTED),
    (dict(D=60), E.GLA_ERR_UNSUPPORTED), (dict(D=1 << 25, xs=1 << 25), E.GLA_ERR_UNSUPPORTED),
    (dict(xs=56), E.GLA_ERR_INVALID_ARG),                    # rows overlap
    (dict(xs=68), E.GLA_ERR_MISALIGNED),                     # rows not 16-byte aligned (bf16)
    (dict(x=None), E.GLA_ERR_INVALID_ARG), (dict(w=None), E.GLA_ERR_INVALID_ARG),
    (dict(out=None), E.GLA_ERR_INVALID_ARG),
    (dict(x=P[0] + 8), E.GLA_ERR_MISALIGNED), (dict(w=P[1] + 2), E.GLA_ERR_MISALIGNED),
    (dict(cu=P[6] + 1, B=2, T=16), E.GLA_ERR_MISALIGNED),
    (dict(out=P[0]), E.GLA_ERR_INVALID_ARG), (dict(fin=P[4]), E.GLA_ERR_INVALID_ARG),
    (dict(fin=P[3] + 16), E.GLA_ERR_INVALID_ARG),            # partly over the initial state
    (dict(B=1 << 20, T=1 << 20), E.GLA_ERR_INVALID_ARG),
])
def test_conv_fwd_rejects_before_launch(L, kw, status):
    assert conv_fwd(L, **kw) == status


def test_conv_fwd_rejects_more_blocks_than_a_grid_has(L):
    """A block for every sequence's final state and one for the rows: 2^31 - 1 and one."""
    many = dict(B=2 ** 31 - 1, D=8, xs=8, W=2, cu=1 << 40, fin=1 << 42, init=None)
    assert conv_fwd(L, T=1, **many) == E.GLA_ERR_INVALID_ARG


def test_conv_empty_calls_do_nothing(L):
    assert conv_fwd(L, B=0) == E.GLA_OK and conv_fwd(L, D=0) == E.GLA_OK
    assert conv_fwd(L, T=0, fin=None, x=None, out=None) == E.GLA_OK


def conv_bwd(L, **kw):
    a = dict(x=P[0], xs=64, w=P[1], b=P[2], init=P[3], dy=P[4], df=P[5], dx=P[6], dw=P[7],
             db=P[8], di=P[9], cu=None, B=2, T=16, D=64, W=4, ws=P[20], wb=1 << 20, flags=0)
    a.update(kw)
    return L.gla_conv_bwd(a["x"], a["xs"], a["w"], a["b"], a["init"], a["dy"], a["df"], a["dx"],
                          a["dw"], a["db"], a["di"], a["cu"], a["B"], a["T"], a["D"], a["W"],
                          a["ws"], a["wb"], None, a["flags"])


@pytest.mark.parametrize("kw,status", [
    (dict(flags=1 << 9), E.GLA_ERR_INVALID_ARG), (dict(W=6), E.GLA_ERR_UNSUPPORTED),
    (dict(dw=None), E.GLA_ERR_INVALID_ARG), (dict(dy=None), E.GLA_ERR_INVALID_ARG),
    (dict(dx=P[0]), E.GLA_ERR_INVALID_ARG), (dict(db=P[7] + 16), E.GLA_ERR_INVALID_ARG),
    (dict(ws=P[6]), E.GLA_ERR_INVALID_ARG), (dict(ws=None), E.GLA_ERR_INVALID_ARG),
    (dict(wb=64), E.GLA_ERR_INVALID_ARG), (dict(ws=P[20] + 16), E.GLA_ERR_MISALIGNED),
    (dict(di=P[9] + 4), E.GLA_ERR_MISALIGNED),
    (dict(B=0, cu=P[12]), E.GLA_ERR_INVALID_ARG),            # rows, but no sequence
])
def test_conv_bwd_rejects_before_launch(L, kw, status):
    assert conv_bwd(L, **kw) == status


def conv_step(L, **kw):
    a = dict(x=P[0], xs=64, w=P[1], b=P[2], st=P[3], ns=0, sl=None, os=None, out=P[4], N=4, D=64,
             W=4, flags=0)
    a.update(kw)
    return L.gla_conv_step(a["x"], a["xs"], a["w"], a["b"], a["st"], a["ns"], a["sl"], a["os"],
                           a["out"], a["N"], a["D"], a["W"], None, a["flags"])


@pytest.mark.parametrize("kw,status", [
    (dict(ns=3), E.GLA_ERR_INVALID_ARG), (dict(os=P[7]), E.GLA_ERR_INVALID_ARG),
    (dict(N=-1), E.GLA_ERR_INVALID_ARG), (dict(st=None), E.GLA_ERR_INVALID_ARG),
    (dict(out=P[3]), E.GLA_ERR_INVALID_ARG), (dict(sl=P[6] + 2, ns=8), E.GLA_ERR_MISALIGNED),
    (dict(sl=P[3], ns=8), E.GLA_ERR_INVALID_ARG), (dict(D=12), E.GLA_ERR_UNSUPPORTED),
])
def test_conv_step_rejects_before_launch(L, kw, status):
    assert conv_step(L, **kw) == status
    assert conv_step(L, N=0) == E.GLA_OK


ROWS = dict(u=P[0], us=64, dt=P[1], dts=64, a=P[2], b=P[3], bs=16, c=P[4], cs=16, skip=P[5],
            z=P[6], zs=64, bias=P[7])


def rows_of(a):
    return [a[k] for k in ("u", "us", "dt", "dts", "a", "b", "bs", "c", "cs", "skip", "z", "zs",
                           "bias")]


def scan_fwd(L, **kw):
    a = dict(ROWS, init=P[8], out=P[9], fin=P[10], cu=None, B=2, T=16, D=64, N=16, ws=P[30],
             wb=1 << 20, flags=E.GLA_FLAG_SOFTPLUS)
    a.update(kw)
    return L.gla_scan_fwd(*rows_of(a), a["init"], a["out"], a["fin"], a["cu"], a["B"], a["T"],
                          a["D"], a["N"], a["ws"], a["wb"], None, a["flags"])


SCAN_BAD = [
    (dict(flags=E.GLA_FLAG_SILU), E.GLA_ERR_INVALID_ARG), (dict(B=-2), E.GLA_ERR_INVALID_ARG),
    (dict(N=12), E.GLA_ERR_UNSUPPORTED), (dict(N=128), E.GLA_ERR_UNSUPPORTED),
    (dict(D=62), E.GLA_ERR_UNSUPPORTED), (dict(us=63), E.GLA_ERR_INVALID_ARG),
    (dict(bs=8), E.GLA_ERR_INVALID_ARG), (dict(zs=32), E.GLA_ERR_INVALID_ARG),
    (dict(dts=68), E.GLA_ERR_MISALIGNED), (dict(u=None), E.GLA_ERR_INVALID_ARG),
    (dict(a=None), E.GLA_ERR_INVALID_ARG), (dict(c=None), E.GLA_ERR_INVALID_ARG),
    (dict(u=P[0] + 2), E.GLA_ERR_MISALIGNED), (dict(b=P[3] + 1), E.GLA_ERR_MISALIGNED),
    (dict(a=P[2] + 4), E.GLA_ERR_MISALIGNED), (dict(z=P[6] + 8), E.GLA_ERR_MISALIGNED),
    (dict(B=1 << 20, T=1 << 20), E.GLA_ERR_INVALID_ARG),
]


@pytest.mark.parametrize("kw,status", SCAN_BAD + [
    (dict(out=None), E.GLA_ERR_INVALID_ARG), (dict(out=P[0]), E.GLA_ERR_INVALID_ARG),
    (dict(fin=P[8] + 64), E.GLA_ERR_INVALID_ARG), (dict(out=P[9] + 4), E.GLA_ERR_MISALIGNED),
    (dict(fin=P[6]), E.GLA_ERR_INVALID_ARG),
])
def test_scan_fwd_rejects_before_launch(L, kw, status):
    assert scan_fwd(L, **kw) == status
    assert scan_fwd(L, B=0) == E.GLA_OK
    assert scan_fwd(L, T=0, fin=None) == E.GLA_OK


def scan_bwd(L, **kw):
    a = dict(ROWS, init=P[8], dy=P[9], df=P[10], du=P[11], ddt=P[12], da=P[13], db=P[14],
             dc=P[15], ds=P[16], dz=P[17], dbias=P[18], di=P[19], cu=None, B=2, T=16, D=64, N=16,
             ws=1 << 32, wb=1 << 28, flags=E.GLA_FLAG_SOFTPLUS)
    a.update(kw)
    return L.gla_scan_bwd(*rows_of(a), a["init"], a["dy"], a["df"], a["du"], a["ddt"], a["da"],
                          a["db"], a["dc"], a["ds"], a["dz"], a["dbias"], a["di"], a["cu"],
                          a["B"], a["T"], a["D"], a["N"], a["ws"], a["wb"], None, a["flags"])


@pytest.mark.parametrize("kw,status", SCAN_BAD + [
    (dict(dz=None), E.GLA_ERR_INVALID_ARG), (dict(z=None), E.GLA_ERR_INVALID_ARG),
    (dict(skip=None), E.GLA_ERR_INVALID_ARG), (dict(bias=None), E.GLA_ERR_INVALID_ARG),
    (dict(da=None), E.GLA_ERR_INVALID_ARG), (dict(dy=None), E.GLA_ERR_INVALID_ARG),
    (dict(ws=None), E.GLA_ERR_INVALID_ARG), (dict(wb=1000), E.GLA_ERR_INVALID_ARG),
    (dict(du=P[1]), E.GLA_ERR_INVALID_ARG), (dict(db=P[14] + 4), E.GLA_ERR_MISALIGNED),
    (dict(dc=P[14] + 64), E.GLA_ERR_INVALID_ARG), (dict(ws=P[11]), E.GLA_ERR_INVALID_ARG),
    (dict(B=0, cu=P[21]), E.GLA_ERR_INVALID_ARG),
])
def test_scan_bwd_rejects_before_launch(L, kw, status):
    assert scan_bwd(L, **kw) == status


def scan_step(L, **kw):
    a = dict(ROWS, st=P[8], ns=0, sl=None, os=None, out=P[9], R=4, D=64, N=16,
             flags=E.GLA_FLAG_SOFTPLUS)
    a.update(kw)
    return L.gla_scan_step(*rows_of(a), a["st"], a["ns"], a["sl"], a["os"], a["out"], a["R"],
                           a["D"], a["N"], None, a["flags"])


@pytest.mark.parametrize("kw,status", [
    (dict(N=4), E.GLA_ERR_UNSUPPORTED), (dict(ns=2), E.GLA_ERR_INVALID_ARG),
    (dict(os=P[20]), E.GLA_ERR_INVALID_ARG), (dict(st=None), E.GLA_ERR_INVALID_ARG),
    (dict(out=P[8]), E.GLA_ERR_INVALID_ARG), (dict(u=P[8] + 64), E.GLA_ERR_INVALID_ARG),
    (dict(st=P[8] + 8), E.GLA_ERR_MISALIGNED), (dict(R=-1), E.GLA_ERR_INVALID_ARG),
    (dict(sl=P[20] + 2, ns=4), E.GLA_ERR_MISALIGNED),
])
def test_scan_step_rejects_before_launch(L, kw, status):
    assert scan_step(L, **kw) == status
    assert scan_step(L, R=0) == E.GLA_OK


def pools(*sizes, base=1 << 33):
    arr = (_binding.PagePool * max(1, len(sizes)))()
    for i, n in enumerate(sizes):
        arr[i].base, arr[i].page_bytes = base + (i << 32), n
    return arr


def test_pages_reject_before_launch(L):
    bad, un, mis = E.GLA_ERR_INVALID_ARG, E.GLA_ERR_UNSUPPORTED, E.GLA_ERR_MISALIGNED
    ok = pools(4096)
    copy = lambda p=ok, k=1, S=8, s=P[0], t=P[1], c=P[2], n=3: L.gla_pages_copy(  # noqa: E731
        p, k, S, s, t, c, n, None)
    assert copy(n=-1) == bad and copy(s=None) == bad and copy(c=None) == bad
    assert copy(c=P[0]) == bad and copy(S=E.GLA_MAX_PAGES + 1) == un and copy(S=-1) == bad
    assert copy(p=pools(4090)) == mis and copy(p=pools(0)) == bad and copy(p=pools(4096, base=8)) == mis
    assert copy(s=P[0] + 2) == mis
    assert copy(p=pools(4096, base=P[1])) == bad            # a table inside a pool
    two = pools(4096, 4096)
    two[1].base = two[0].base + 4096
    assert copy(p=two, k=2) == bad                          # pools overlap
    assert copy(n=0) == E.GLA_OK
    fork = lambda u=P[0], uo=P[0], p=P[1], c=P[2], n=3, S=8: L.gla_pages_fork(  # noqa: E731
        ok, 1, S, u, uo, p, c, n, None)
    assert fork(u=None) == bad and fork(uo=None) == bad and fork(p=None) == bad
    assert fork(c=P[1]) == bad and fork(uo=P[0] + 4) == bad and fork(p=P[0]) == bad
    assert fork(n=0) == E.GLA_OK                            # in place, nothing asked for
    comp = lambda u=P[0], uo=P[0], s=P[1], so=P[1], f=P[3], n=3: L.gla_pages_compact(  # noqa: E731
        ok, 1, 8, u, uo, s, so, n, f, None)
    assert comp(f=None) == bad and comp(f=P[0]) == bad and comp(so=P[1] + 4) == bad
    assert comp(s=P[0]) == bad and comp(u=None) == bad
    free = lambda u=P[0], uo=P[0], s=P[1], n=3: L.gla_pages_free(u, uo, 8, s, n, None)  # noqa: E731
    assert free(u=None) == bad and free(s=P[0]) == bad and free(uo=P[0] + 8) == bad
    assert free(n=0) == E.GLA_OK


def test_python_wrappers_refuse_cpu_tensors_and_bad_options():
    import gated_linear_attention_gla_gb300 as gla
    x = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        gla.conv_fwd(x, torch.zeros(64, 4))
    with pytest.raises(ValueError):
        gla.scan_fwd(x, x, torch.zeros(64, 16), x[..., :16], x[..., :16])
    with pytest.raises(ValueError):
        gla.fork_pages([], torch.zeros(4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))


def test_row_strides():
    from gated_linear_attention_gla_gb300._marshal import rows
    t = torch.zeros(3, 5, 32)
    step = lambda v, dtype=torch.float32: rows(v, "t", v.shape, dtype, v.device)[1]  # noqa: E731
    assert step(t) == 32 and step(t[..., 8:16]) == 32 and step(t[0, :, 8:16]) == 32
    assert step(t[:, :1, :8]) == 160                            # one token a sequence
    assert step(t[:1, :1, :8]) == 8 and step(t[0, :1, :8]) == 8  # one row
    assert step(t[:0]) == 32
    assert rows(t[..., 8:16], "t", (3, 5, 8), torch.float32, t.device)[0] == t.data_ptr() + 32
    for bad in (t[:, :4, :8],                                  # rows at two distances
                t[..., ::2],                                   # columns apart
                t[:, :1].expand(3, 5, 32),                     # one row five times
                t.transpose(0, 1), t[None]):
        with pytest.raises(ValueError):
            step(bad)
    with pytest.raises(ValueError):
        step(t, torch.bfloat16)
    with pytest.raises(ValueError):
        rows(t, "t", (3, 5, 31), torch.float32, t.device)


def _differences(f, t, idx, eps=1e-6):
    old = t.view(-1)[idx].item()
    t.view(-1)[idx] = old + eps
    hi = f()
    t.view(-1)[idx] = old - eps
    lo = f()
    t.view(-1)[idx] = old
    return (hi - lo) / (2 * eps)


@pytest.mark.parametrize("act", [False, True])
def test_reference_conv_gradients_against_differences(act):
    g = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    cu = [0, 1, 1, 3, 9]
    for W in (2, 4):
        x, w, b, init, dy, df = rnd(9, 2), rnd(2, W), rnd(2), rnd(4, W - 1, 2), rnd(9, 2), rnd(4, W - 1, 2)

        def loss():
            o = ssm_ref.conv(x, w, b, init, cu, act)
            return float((o["y"] * dy).sum() + (o["final"] * df).sum())

        got = ssm_ref.conv(x, w, b, init, cu, act, dy, df)
        for name, t in (("dx", x), ("dw", w), ("db", b), ("d_init", init)):
            for i in range(t.numel()):
                assert abs(_differences(loss, t, i) - float(got[name].reshape(-1)[i])) < 1e-6, name


@pytest.mark.parametrize("softplus", [False, True])
def test_reference_scan_gradients_against_differences(softplus):
    g = torch.Generator().manual_seed(4)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    cu = [0, 1, 1, 6]
    t = dict(u=rnd(6, 2), dt=rnd(6, 2), a=-rnd(2, 3).abs(), b=rnd(6, 3), c=rnd(6, 3), skip=rnd(2),
             z=rnd(6, 2), bias=rnd(2), init=rnd(3, 2, 3))
    dy, df = rnd(6, 2), rnd(3, 2, 3)
    run = lambda *more: ssm_ref.scan(t["u"], t["dt"], t["a"], t["b"], t["c"], t["skip"], t["z"],  # noqa: E731
                                     t["bias"], softplus, t["init"], cu, *more)

    def loss():
        o = run()
        return float((o["y"] * dy).sum() + (o["final"] * df).sum())

    got = run(dy, df)
    for name, key in (("u", "du"), ("dt", "ddt"), ("a", "da"), ("b", "db"), ("c", "dc"),
                      ("skip", "dskip"), ("z", "dz"), ("bias", "dbias"), ("init", "d_init")):
        for i in range(t[name].numel()):
            assert abs(_differences(loss, t[name], i) - float(got[key].reshape(-1)[i])) < 1e-6, key
