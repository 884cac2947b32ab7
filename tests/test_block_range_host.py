"""What the entry points of the recurrence, the norms and the projections refuse at the ends of their
ranges, before anything touches the GPU (CPU only)."""
import pytest
import torch

import gated_linear_attention_gla_gb300 as gla
from gated_linear_attention_gla_gb300 import _binding as E
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
