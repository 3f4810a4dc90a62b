"""Host-side edges of the block operators (norm, convolution, scan) on the CPU: the
largest sizes that a call may name, and what a call tells autograd of the tensors it
writes in place."""
import pytest
import torch

from linear_rnn_mlstm_b200 import binding as xb


@pytest.mark.parametrize("dt", (xb.F32, xb.BF16))
def test_norm_workspace_at_the_most_rows(dt):
    """The number of CTAs must not wrap: a full wave, as for any large number of rows."""
    for C in (8, 512, 8192):                                  # a warp per row, and a CTA per row
        want = xb.xlstm_rmsnorm_bwd_workspace_size(1 << 20, C, dt)
        assert want[0] == xb.OK and 0 < want[1] < 1 << 26
        for rows in ((1 << 31) - 8, (1 << 31) - 7, (1 << 31) - 1):
            assert xb.xlstm_rmsnorm_bwd_workspace_size(rows, C, dt) == want, (rows, C)
