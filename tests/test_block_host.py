"""The recurrence's, the norms' and the feed-forward projections' entry points on the host:
bad arguments are rejected before anything touches the GPU, empty calls do
nothing, and the tests' own 64-bit formulas agree with finite differences (CPU only)."""
import re

import pytest
import torch

import block_ref
import gated_linear_attention_gla_gb300 as gla
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
    for name in ("gla_recur_fwd", "gla_recur_bwd", "gla_recur_bwd_workspace_size", "gla_recur_step",
                 "gla_block_norm_fwd", "gla_block_norm_bwd", "gla_block_norm_bwd_workspace_size",
                 "gla_glu_fwd", "gla_glu_bwd", "gla_glu_bwd_workspace_size"):
        params = re.search(name + r"\s*\(([^)]*)\)", text).group(1).split(",")
        assert len(getattr(L, name).argtypes) == len(params), name
        assert callable(getattr(gla, name[4:], None)) or name.endswith("_size")


ROWS = dict(x=P[0], xs=64, f=P[1], fs=64, i=P[2], is_=64, z=P[3], zs=64, decay=P[4])


def rows_of(a):
    return [a[k] for k in ("x", "xs", "f", "fs", "i", "is_", "z", "zs", "decay")]


def recur_fwd(L, **kw):
    a = dict(ROWS, init=P[5], out=P[6], fin=P[7], cu=None, B=2, T=16, D=64, flags=0)
    a.update(kw)
    return L.gla_recur_fwd(*rows_of(a), a["init"], a["out"], a["fin"], a["cu"], a["B"], a["T"],
                           a["D"], None, a["flags"])


COMMON = [
    (dict(flags=E.GLA_FLAG_SILU), E.GLA_ERR_INVALID_ARG), (dict(D=60), E.GLA_ERR_UNSUPPORTED),
    (dict(D=1 << 25, xs=1 << 25, fs=1 << 25, is_=1 << 25, zs=1 << 25), E.GLA_ERR_UNSUPPORTED),
    (dict(xs=56), E.GLA_ERR_INVALID_ARG), (dict(fs=68), E.GLA_ERR_MISALIGNED),
    (dict(is_=72, flags=E.GLA_FLAG_FP32_IO, zs=66), E.GLA_ERR_MISALIGNED),
    (dict(x=None), E.GLA_ERR_INVALID_ARG), (dict(f=None), E.GLA_ERR_INVALID_ARG),
    (dict(out=None), E.GLA_ERR_INVALID_ARG), (dict(z=P[3] + 8), E.GLA_ERR_MISALIGNED),
    (dict(decay=P[4] + 4), E.GLA_ERR_MISALIGNED), (dict(out=P[1]), E.GLA_ERR_INVALID_ARG),
    (dict(xs=1 << 41), E.GLA_ERR_INVALID_ARG)]


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(B=-1), E.GLA_ERR_INVALID_ARG), (dict(T=-1), E.GLA_ERR_INVALID_ARG),
    (dict(fin=P[6]), E.GLA_ERR_INVALID_ARG), (dict(fin=P[5] + 16), E.GLA_ERR_INVALID_ARG),
    (dict(cu=P[8] + 2), E.GLA_ERR_MISALIGNED), (dict(B=1 << 20, T=1 << 20), E.GLA_ERR_INVALID_ARG),
    (dict(B=2 ** 30, T=1, D=512, xs=512, fs=512, is_=512, zs=512, x=1 << 44, f=2 << 44, i=3 << 44,
          z=4 << 44, out=5 << 44, fin=6 << 44, init=None), E.GLA_ERR_INVALID_ARG)])
def test_recur_fwd_rejects_before_launch(L, kw, status):
    assert recur_fwd(L, **kw) == status


def test_recur_empty_calls_do_nothing(L):
    assert recur_fwd(L, B=0) == E.GLA_OK and recur_fwd(L, D=0) == E.GLA_OK
    assert recur_fwd(L, T=0, fin=None, x=None, f=None, out=None) == E.GLA_OK


def recur_bwd(L, **kw):
    a = dict(ROWS, init=P[5], dy=P[6], dfin=P[7], dx=P[8], df=P[9], di=P[10], dz=P[11], dd=P[12],
             d0=P[13], cu=None, B=2, T=16, D=64, ws=P[20], wb=1 << 20, flags=0)
    a.update(kw)
    return L.gla_recur_bwd(*rows_of(a), a["init"], a["dy"], a["dfin"], a["dx"], a["df"], a["di"],
                           a["dz"], a["dd"], a["d0"], a["cu"], a["B"], a["T"], a["D"], a["ws"],
                           a["wb"], None, a["flags"])


@pytest.mark.parametrize("kw,status", [
    (dict(flags=1 << 9), E.GLA_ERR_INVALID_ARG), (dict(dy=None), E.GLA_ERR_INVALID_ARG),
    (dict(di=None), E.GLA_ERR_INVALID_ARG), (dict(i=None), E.GLA_ERR_INVALID_ARG),
    (dict(z=None), E.GLA_ERR_INVALID_ARG), (dict(decay=None), E.GLA_ERR_INVALID_ARG),
    (dict(dx=P[0]), E.GLA_ERR_INVALID_ARG), (dict(dd=P[9] + 16), E.GLA_ERR_INVALID_ARG),
    (dict(ws=None), E.GLA_ERR_INVALID_ARG), (dict(wb=64), E.GLA_ERR_INVALID_ARG),
    (dict(ws=P[20] + 16), E.GLA_ERR_MISALIGNED), (dict(ws=P[8]), E.GLA_ERR_INVALID_ARG),
    (dict(d0=P[13] + 4), E.GLA_ERR_MISALIGNED), (dict(B=0, cu=P[14]), E.GLA_ERR_INVALID_ARG)])
def test_recur_bwd_rejects_before_launch(L, kw, status):
    assert recur_bwd(L, **kw) == status


def recur_step(L, **kw):
    a = dict(ROWS, st=P[5], ns=0, sl=None, os=None, out=P[6], N=4, D=64, flags=0)
    a.update(kw)
    return L.gla_recur_step(*rows_of(a), a["st"], a["ns"], a["sl"], a["os"], a["out"], a["N"],
                            a["D"], None, a["flags"])


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(ns=3), E.GLA_ERR_INVALID_ARG), (dict(os=P[7]), E.GLA_ERR_INVALID_ARG),
    (dict(N=-1), E.GLA_ERR_INVALID_ARG), (dict(st=None), E.GLA_ERR_INVALID_ARG),
    (dict(st=P[0]), E.GLA_ERR_INVALID_ARG), (dict(sl=P[7] + 2, ns=8), E.GLA_ERR_MISALIGNED),
    (dict(sl=P[5], ns=8), E.GLA_ERR_INVALID_ARG)])
def test_recur_step_rejects_before_launch(L, kw, status):
    assert recur_step(L, **kw) == status
    assert recur_step(L, N=0) == E.GLA_OK


def norm_fwd(L, **kw):
    a = dict(res=P[0], y=P[1], ys=64, z=P[2], zs=64, pw=P[3], pb=P[4], sc=P[5], w=P[6], b=P[7],
             eps=1e-6, ro=P[8], out=P[9], R=16, D=64, flags=0)
    a.update(kw)
    return L.gla_block_norm_fwd(a["res"], a["y"], a["ys"], a["z"], a["zs"], a["pw"], a["pb"],
                                a["sc"], a["w"], a["b"], a["eps"], a["ro"], a["out"], a["R"],
                                a["D"], None, a["flags"])


@pytest.mark.parametrize("kw,status", [
    (dict(flags=E.GLA_FLAG_SILU), E.GLA_ERR_INVALID_ARG), (dict(R=-1), E.GLA_ERR_INVALID_ARG),
    (dict(D=60), E.GLA_ERR_UNSUPPORTED), (dict(D=8200, ys=8200, zs=8200), E.GLA_ERR_UNSUPPORTED),
    (dict(eps=-1.0), E.GLA_ERR_INVALID_ARG), (dict(eps=float("nan")), E.GLA_ERR_INVALID_ARG),
    (dict(eps=float("inf")), E.GLA_ERR_INVALID_ARG), (dict(res=None), E.GLA_ERR_INVALID_ARG),
    (dict(y=None), E.GLA_ERR_INVALID_ARG), (dict(pw=None), E.GLA_ERR_INVALID_ARG),
    (dict(w=None), E.GLA_ERR_INVALID_ARG), (dict(out=None), E.GLA_ERR_INVALID_ARG),
    (dict(out=None, w=None, b=None, ro=None), E.GLA_ERR_INVALID_ARG),
    (dict(ys=56), E.GLA_ERR_INVALID_ARG), (dict(zs=68), E.GLA_ERR_MISALIGNED),
    (dict(sc=P[5] + 8), E.GLA_ERR_MISALIGNED), (dict(out=P[9] + 2), E.GLA_ERR_MISALIGNED),
    (dict(out=P[0]), E.GLA_ERR_INVALID_ARG), (dict(ro=P[0] + 16), E.GLA_ERR_INVALID_ARG),
    (dict(ro=P[9]), E.GLA_ERR_INVALID_ARG), (dict(ro=P[1]), E.GLA_ERR_INVALID_ARG)])
def test_block_norm_fwd_rejects_before_launch(L, kw, status):
    assert norm_fwd(L, **kw) == status
    assert norm_fwd(L, R=0) == E.GLA_OK and norm_fwd(L, D=0) == E.GLA_OK


def norm_bwd(L, **kw):
    a = dict(res=P[0], y=P[1], ys=64, z=P[2], zs=64, pw=P[3], pb=P[4], sc=P[5], w=P[6], eps=1e-6,
             du=P[7], ds=P[8], dr=P[9], dy=P[10], dz=P[11], dpw=P[12], dpb=P[13], dsc=P[14],
             dw=P[15], db=P[16], R=16, D=64, ws=P[20], wb=1 << 20, flags=0)
    a.update(kw)
    return L.gla_block_norm_bwd(a["res"], a["y"], a["ys"], a["z"], a["zs"], a["pw"], a["pb"],
                                a["sc"], a["w"], a["eps"], a["du"], a["ds"], a["dr"], a["dy"],
                                a["dz"], a["dpw"], a["dpb"], a["dsc"], a["dw"], a["db"], a["R"],
                                a["D"], a["ws"], a["wb"], None, a["flags"])


@pytest.mark.parametrize("kw,status", [
    (dict(dr=None), E.GLA_ERR_INVALID_ARG), (dict(dy=None), E.GLA_ERR_INVALID_ARG),
    (dict(dz=None), E.GLA_ERR_INVALID_ARG), (dict(z=None), E.GLA_ERR_INVALID_ARG),
    (dict(pb=None), E.GLA_ERR_INVALID_ARG), (dict(sc=None), E.GLA_ERR_INVALID_ARG),
    (dict(w=None), E.GLA_ERR_INVALID_ARG), (dict(dr=P[0]), E.GLA_ERR_INVALID_ARG),
    (dict(ws=None), E.GLA_ERR_INVALID_ARG), (dict(wb=8), E.GLA_ERR_INVALID_ARG),
    (dict(ws=P[20] + 16), E.GLA_ERR_MISALIGNED), (dict(dw=P[15] + 2), E.GLA_ERR_MISALIGNED),
    (dict(db=P[15]), E.GLA_ERR_INVALID_ARG), (dict(D=16384, ys=16384, zs=16384), E.GLA_ERR_UNSUPPORTED)])
def test_block_norm_bwd_rejects_before_launch(L, kw, status):
    assert norm_bwd(L, **kw) == status
    assert norm_bwd(L, D=0) == E.GLA_OK


def glu(L, bwd, **kw):
    a = dict(x=P[0], xs=64, wg=P[1], wu=P[2], out=P[3], dx=P[4], dwg=P[5], dwu=P[6], R=16, D=64,
             F=128, ws=P[20], wb=1 << 20, flags=0)
    a.update(kw)
    if bwd:
        return L.gla_glu_bwd(a["x"], a["xs"], a["wg"], a["wu"], a["out"], a["dx"], a["dwg"],
                             a["dwu"], a["R"], a["D"], a["F"], a["ws"], a["wb"], None, a["flags"])
    return L.gla_glu_fwd(a["x"], a["xs"], a["wg"], a["wu"], a["out"], a["R"], a["D"], a["F"], None,
                         a["flags"])


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(flags=E.GLA_FLAG_SILU), E.GLA_ERR_INVALID_ARG), (dict(R=-1), E.GLA_ERR_INVALID_ARG),
    (dict(flags=E.GLA_FLAG_FP32_IO), E.GLA_ERR_UNSUPPORTED), (dict(D=60), E.GLA_ERR_UNSUPPORTED),
    (dict(F=100), E.GLA_ERR_UNSUPPORTED), (dict(D=1 << 21, xs=1 << 21), E.GLA_ERR_UNSUPPORTED),
    (dict(x=None), E.GLA_ERR_INVALID_ARG), (dict(wg=None), E.GLA_ERR_INVALID_ARG),
    (dict(out=None), E.GLA_ERR_INVALID_ARG), (dict(xs=56), E.GLA_ERR_INVALID_ARG),
    (dict(xs=68), E.GLA_ERR_MISALIGNED), (dict(wu=P[2] + 8), E.GLA_ERR_MISALIGNED),
    (dict(out=P[3] + 8), E.GLA_ERR_MISALIGNED), (dict(R=2 ** 31 - 1, F=1 << 20), E.GLA_ERR_INVALID_ARG)])
def test_glu_rejects_before_launch(L, bwd, kw, status):
    assert glu(L, bwd, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dx=P[0]), E.GLA_ERR_INVALID_ARG), (dict(dwg=P[6]), E.GLA_ERR_INVALID_ARG),
    (dict(dwu=None), E.GLA_ERR_INVALID_ARG), (dict(ws=None), E.GLA_ERR_INVALID_ARG),
    (dict(wb=8), E.GLA_ERR_INVALID_ARG), (dict(ws=P[20] + 16), E.GLA_ERR_MISALIGNED)])
def test_glu_bwd_rejects_before_launch(L, kw, status):
    assert glu(L, True, **kw) == status


def test_glu_empty_calls_do_nothing(L):
    assert glu(L, False, R=0) == E.GLA_OK and glu(L, False, F=0) == E.GLA_OK
    assert glu(L, False, out=P[0]) == E.GLA_ERR_INVALID_ARG  # the output over x


def test_python_refusals():
    """Arguments the wrappers refuse before the library is called (CPU tensors first)."""
    x = torch.zeros(1, 4, 64)
    for call in (lambda: gla.recur_fwd(x, x), lambda: gla.recur_bwd(x, x, x),
                 lambda: gla.recur_step(x[0], x[0], x[0]), lambda: gla.block_norm_fwd(x, x, weight=x[0, 0]),
                 lambda: gla.block_norm_bwd(x, x), lambda: gla.glu_fwd(x, x[0], x[0]),
                 lambda: gla.glu_bwd(x, x[0], x[0], x)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("decay,unit", [(True, True), (True, False), (False, True), (False, False)])
def test_reference_recurrence_gradients(decay, unit):
    g = torch.Generator().manual_seed(1)
    cu, D = [0, 3, 3, 7], 2
    x, f, i, z = (torch.randn(7, D, generator=g).double().requires_grad_(True) for _ in range(4))
    dec = (-torch.rand(D, generator=g).double() - 0.1).requires_grad_(True) if decay else None
    init = torch.randn(3, D, generator=g).double().requires_grad_(True)
    fn = lambda *a: block_ref.recur(a[0], a[1], a[5] if decay else None, a[2], a[3], unit, a[4], cu)  # noqa: E731
    args = (x, f, i, z, init) + ((dec,) if decay else ())
    assert torch.autograd.gradcheck(fn, args)


@pytest.mark.parametrize("layer", [True, False])
def test_reference_norm_gradients(layer):
    g = torch.Generator().manual_seed(2)
    t = lambda *s: torch.randn(*s, generator=g).double().requires_grad_(True)  # noqa: E731
    args = (t(3, 8), t(3, 8), t(3, 8), t(8), t(8), t(8), t(8), t(8))
    assert torch.autograd.gradcheck(lambda *a: block_ref.block_norm(*a, layer, 1e-3), args)


def test_reference_glu_gradients():
    g = torch.Generator().manual_seed(3)
    x, wg, wu, dh = (torch.randn(*s, generator=g).double() for s in ((5, 6), (4, 6), (4, 6), (5, 4)))
    got = block_ref.glu_all(x, wg, wu, dh)
    leaves = [v.clone().requires_grad_(True) for v in (x, wg, wu)]
    (block_ref.silu(leaves[0] @ leaves[1].t()) * (leaves[0] @ leaves[2].t()) * dh).sum().backward()
    for n, v in zip(("dx", "dwg", "dwu"), leaves):
        assert torch.allclose(got[n][0], v.grad, rtol=1e-10)


def test_build_knows_every_source_file():
    """A change of any file of csrc rebuilds the library."""
    import os
    known = {os.path.basename(p) for p in glabuild._inputs()}
    assert set(os.listdir(glabuild.CSRC)) <= known
