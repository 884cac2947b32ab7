"""What the entry points of the recurrence, the norms and the projections refuse at the ends of their
ranges, before anything touches the GPU (CPU only)."""
import pytest

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
