"""What the entry points of the recurrence, the norms and the projections refuse at the ends of their
ranges, before anything touches the GPU (CPU only)."""
import pytest
import torch

import gated_linear_attention_gla_gb300 as gla
from gated_linear_attention_gla_gb300 import _binding as E
import test_block_host as block
import test_ssm_host as ssm
from test_block_host import L, glu  # noqa: F401

FAR = [k << 48 for k in range(1, 16)]  # fake, aligned, never dereferenced, far apart


def test_glu_gradients_have_a_row_limit(L):
    """The weights' gradients are one sum over the rows."""
    most = 1 << 26
    far = dict(x=FAR[0], wg=FAR[1], wu=FAR[2], out=FAR[3], dx=FAR[4], dwg=FAR[5], dwu=FAR[6], ws=FAR[7])
    for rows in (most + 1, 1 << 29, 2 ** 31 - 1):
        assert glu(L, True, R=rows, D=8, F=8, xs=8, **far) == E.GLA_ERR_UNSUPPORTED
        assert L.gla_glu_bwd_workspace_size(rows, 8, 8) == 0
    assert L.gla_glu_bwd_workspace_size(most, 8, 8) == 2 * most * 8 * 2
    # the limit itself passes the check: the next one, of the workspace, speaks
    assert glu(L, True, R=most, D=8, F=8, xs=8, wb=1, **far) == E.GLA_ERR_INVALID_ARG


def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("n", [2 ** 31, 2 ** 32 + 5])
def test_counts_that_no_c_int_holds(n):
    """A count of 2^32 + 5 must not reach the library as 5."""
    w, f = meta(8, 8), meta(8, dtype=torch.float32)
    cu = torch.zeros(2, dtype=torch.int32, device="meta")
    rows, seqs, toks, wide = meta(n, 8), meta(n, 1, 8), meta(1, n, 8), meta(1, n)
    filt, a = meta(8, 4, dtype=torch.float32), meta(8, 8, dtype=torch.float32)
    state = meta(n, 8, dtype=torch.float32)
    calls = [
        lambda: gla.recur_fwd(seqs, seqs), lambda: gla.recur_fwd(toks, toks), lambda: gla.recur_fwd(rows, rows, cu_seqlens=cu),
        lambda: gla.recur_fwd(wide[None], wide[None]), lambda: gla.recur_bwd(toks, toks, toks),
        lambda: gla.recur_fwd(w, w, cu_seqlens=torch.zeros(n + 1, dtype=torch.int32, device="meta")),
        lambda: gla.recur_step(rows, rows, state),
        lambda: gla.block_norm_fwd(rows, weight=f), lambda: gla.block_norm_fwd(meta(n // 8, 8, 8), weight=f),
        lambda: gla.block_norm_fwd(wide, weight=f), lambda: gla.block_norm_bwd(rows, rows, weight=f),
        lambda: gla.glu_fwd(rows, w, w), lambda: gla.glu_bwd(rows, w, w, rows), lambda: gla.glu_fwd(wide, w, w),
        lambda: gla.glu_fwd(w, rows, rows),
        lambda: gla.conv_fwd(toks, filt), lambda: gla.conv_step(rows, filt, meta(n, 3, 8)), lambda: gla.conv_fwd(wide[None], filt),
        lambda: gla.scan_fwd(seqs, seqs, a, seqs, seqs), lambda: gla.scan_step(rows, rows, a, rows, rows, state)]
    for call in calls:
        with pytest.raises(ValueError, match="at most 2.31 - 1"):
            call()


MOST, APART = 2 ** 31 - 1, 1 << 40


def far(*names):
    """Tensors far apart, so that no overlap is found."""
    return {n: (k + 1) << 54 for k, n in enumerate(names)}


RECUR = far("x", "f", "i", "z", "decay", "init", "out", "fin", "dy", "dfin", "dx", "df", "di", "dz", "dd", "d0", "ws", "st")
NORM = far("res", "y", "z", "pw", "pb", "sc", "w", "b", "ro", "out", "du", "ds", "dr", "dy", "dz", "dpw", "dpb", "dsc", "dw", "db", "ws")
GLU = far("x", "wg", "wu", "out", "dx", "dwg", "dwu", "ws")
SSM = far("x", "w", "b", "init", "out", "fin", "u", "dt", "a", "c", "skip", "z", "bias", "ws")


@pytest.mark.parametrize("call,kw", [
    (block.recur_fwd, dict(RECUR, B=MOST, T=MOST, i=None, z=None)), (block.recur_fwd, dict(RECUR, B=1 << 8, T=1 << 16, xs=APART)),
    (block.recur_bwd, dict(RECUR, B=MOST, T=MOST, wb=1 << 62)), (block.recur_bwd, dict(RECUR, B=1, T=1 << 24, fs=APART, wb=1 << 62)),
    (block.recur_step, dict(RECUR, N=1 << 24, zs=APART)), (block.recur_step, dict(RECUR, N=MOST, is_=APART)),
    (block.norm_fwd, dict(NORM, R=MOST, ys=APART)), (block.norm_fwd, dict(NORM, R=1 << 24, zs=APART)),
    (block.norm_bwd, dict(NORM, R=1 << 24, zs=APART, wb=1 << 62)),
    (lambda L, **kw: glu(L, False, **kw), dict(GLU, R=1 << 24, xs=APART)),
    (lambda L, **kw: glu(L, True, **kw), dict(GLU, R=1 << 25, xs=APART, wb=1 << 62)),
    (ssm.conv_fwd, dict(SSM, B=1, T=1 << 24, xs=APART)), (ssm.scan_fwd, dict(SSM, B=1, T=1 << 24, us=APART, wb=1 << 62))])
def test_more_elements_than_64_bits_count(L, call, kw):
    """Rows times their distance beyond 2^63, which wrapped to a small or negative number of elements."""
    assert call(L, **kw) == E.GLA_ERR_INVALID_ARG
