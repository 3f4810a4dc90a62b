"""GPU tests of a padded batch's lengths taken from inside a vector, and of segmented
prompts with lengths at several state sizes."""
import numpy as np
import pytest
import torch

import oracle.block as ob
import oracle.ssm as oscan
from blockparity import BF16, F32, cuda, normal, within
from linear_rnn_mlstm_b200 import binding as xb
from test_scan_parity import bounds, inputs

pytestmark = pytest.mark.gpu


def test_a_slice_of_the_lengths():
    n = torch.tensor([9, 3, 0, 7, 5], dtype=torch.int32)
    x, w = normal(1, 4, 9, 16), normal(2, 16, 4)
    y, st = xb.causal_conv_fwd(x.cuda(), w.cuda(), lengths=n.cuda()[1:], y=torch.zeros(4, 9, 16, device="cuda"))
    same, st2 = xb.causal_conv_fwd(x.cuda(), w.cuda(), lengths=n[1:].cuda(), y=torch.zeros(4, 9, 16, device="cuda"))
    assert torch.equal(y, same) and torch.equal(st, st2)
    yr, _ = ob.causal_conv(x, w, lengths=n[1:].tolist())
    np.testing.assert_allclose(y.cpu().numpy(), yr, rtol=0, atol=1e-5 * np.abs(yr).max())
    d = cuda(inputs(4, 90, 16, 16))
    got = xb.ssm_scan_fwd(**d, lengths=10 * n.cuda()[1:], y=torch.zeros(4, 90, 16, device="cuda"))
    both = torch.cat((torch.zeros(1, dtype=torch.int32), 10 * n[1:])).cuda()[1:]
    again = xb.ssm_scan_fwd(**d, lengths=both, y=torch.zeros(4, 90, 16, device="cuda"))
    assert both.data_ptr() % 16 and all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("dtype", (F32, BF16), ids=("f32", "bf16"))
@pytest.mark.parametrize("N", (1, 5, 8, 13, 30, 32, 50, 64))
def test_segments_of_a_padded_batch(N, dtype):
    """Few channels: the tokens are cut into segments, some of them past a row's end."""
    n = [0, 1, 63, 64, 200, 421]
    i = inputs(6, 421, 16, N, dtype=dtype, seed=N)
    y = torch.full((6, 421, 16), 5.0, dtype=dtype, device="cuda")
    got, h = xb.ssm_scan_fwd(**cuda(i), lengths=torch.tensor(n, dtype=torch.int32).cuda(), y=y)
    yr, hr = oscan.scan(**i, lengths=n)
    ey, eh = bounds(i, lengths=n)
    within(h, hr, eh, "h")
    for b, m in enumerate(n):
        assert torch.all(got[b, m:] == 5.0)
        if m:
            within(got[b, :m], yr[b, :m], ey[b, :m] + 4e-6 * np.abs(yr[b, :m]), "y")
