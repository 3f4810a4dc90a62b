"""GPU tests of the selective scan at its edges: lanes without a channel, growing
states, long walks of one CTA, infinities and NaN inside a sequence.  The
tolerances are those of the parity tests (``test_scan_parity``, ``test_scan_bwd_parity``)."""
import numpy as np
import pytest
import torch

import oracle.ssm as oscan
from blockparity import BF16, F32, cuda, within
from linear_rnn_mlstm_b200 import autograd as xa
from linear_rnn_mlstm_b200 import binding as xb
from test_scan_parity import bounds, inputs

pytestmark = pytest.mark.gpu


# 64, 32, 16, 8 and 4 states: a warp of 256 threads' worth of lanes is left over in each
@pytest.mark.parametrize("dtype", (F32, BF16), ids=("f32", "bf16"))
@pytest.mark.parametrize("C,N", [(8, 64), (24, 32), (72, 16), (136, 8), (264, 4)])
def test_a_step_whose_last_warp_has_idle_lanes(C, N, dtype):
    """The idle lanes must not read the state of channel 0, which its owner is writing."""
    B = 64
    i = inputs(B, None, C, N, dtype=dtype, seed=C)
    h0 = i.pop("h0")
    d, h = cuda(i), h0.cuda()
    y = xb.ssm_scan_step(h=h, **d)
    one = {k: v[:, None] if k in ("x", "delta", "Bm", "Cm", "z") else v for k, v in i.items()}
    yr, hr = oscan.scan(**one, h0=h0)
    ey, eh = bounds({**one, "h0": h0})
    within(h, hr, eh, "h")
    within(y, yr[:, 0], (ey + 4e-6 * np.abs(yr))[:, 0], "y")


def test_a_state_stepped_before_the_backward_is_refused():
    i = cuda(inputs(2, 8, 16, 16))
    i["x"].requires_grad_()
    y, _ = xa.ssm_scan(**i)
    xb.ssm_scan_step(h=i["h0"], **{k: v.detach()[:, 0].contiguous() if k in ("x", "delta", "Bm", "Cm", "z") else v
                                   for k, v in i.items() if k != "h0"})
    with pytest.raises(RuntimeError, match="inplace operation"):
        y.sum().backward()
    y, h = xa.ssm_scan(**{**i, "h0": None})                       # a state that nothing saved may move on
    xb.ssm_scan_step(h=h.detach(), **{k: v.detach()[:, 0].contiguous() if k in ("x", "delta", "Bm", "Cm", "z") else v
                                      for k, v in i.items() if k != "h0"})
    y.sum().backward()
    assert i["x"].grad is not None
