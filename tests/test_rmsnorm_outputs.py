"""GPU tests of the RMS norm's ``y=`` argument against the float64 oracle, with the
tolerances of ``test_rmsnorm_parity``."""
import numpy as np
import pytest
import torch

import oracle.block as ob
from blockparity import BF16, EPS32, F32, normal, within
from linear_rnn_mlstm_b200 import binding as xb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", (F32, BF16), ids=("f32", "bf16"))
@pytest.mark.parametrize("C", (24, 2048, 8192))
def test_into_a_given_tensor_and_in_place(C, dtype):
    x0, r, g = normal(1, 5, C, dtype=dtype), normal(2, 5, C, dtype=dtype), normal(3, C, scale=0.2, mean=1.0)
    for residual in (None, r):
        yr, sr, _ = ob.rmsnorm(x0, g, residual)
        for in_place in (False, True):
            x = x0.cuda()
            out = x if in_place else torch.full_like(x, float("nan"))
            y, s, _ = xb.rmsnorm(x, g.cuda(), None if residual is None else residual.cuda(), y=out)
            assert y is out
            within(y, yr, 32 * EPS32 * np.abs(yr), "y")
            if residual is not None:
                within(s, sr, 0.0, "s")
            else:
                assert s is None if in_place else s is x
            if not in_place:
                assert torch.equal(x.cpu(), x0)


def test_a_given_tensor_must_fit():
    x, g = torch.zeros(4, 64, device="cuda"), torch.ones(64, device="cuda")
    with pytest.raises(ValueError, match="y"):
        xb.rmsnorm(x, g, y=torch.zeros(4, 32, device="cuda"))
    with pytest.raises(TypeError):
        xb.rmsnorm(x, g, y=torch.zeros(4, 64, device="cuda", dtype=BF16))
    with pytest.raises(xb.XlstmError):                            # the residual is still to be read
        r = torch.zeros_like(x)
        xb.rmsnorm(x, g, r, y=r)
