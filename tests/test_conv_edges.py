"""GPU tests of the convolution's backward at its edges: a carried state that is not finite."""
import numpy as np
import pytest
import torch

import oracle.block as ob
from blockparity import BF16, F32, cuda, normal
from linear_rnn_mlstm_b200 import binding as xb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", (F32, BF16), ids=("f32", "bf16"))
@pytest.mark.parametrize("K", (2, 3, 4))
@pytest.mark.parametrize("S", (1, 2, 5, 40))
def test_a_bad_carried_input_spoils_only_what_reads_it(S, K, dtype):
    """The last tap never meets a carried input: its gradient stays finite; so do the
    other channels and the gradients of tokens whose outputs did not read it."""
    for bad in (float("nan"), float("inf")):
        a = dict(x=normal(1, 2, S, 16, dtype=dtype), w=normal(2, 16, K), bias=normal(3, 16), state0=normal(4, 2, K - 1, 16, dtype=dtype))
        a["state0"][1, K - 2, 5] = bad                            # the input just before the sequence
        dy = normal(5, 2, S, 16, dtype=dtype)
        for act in ("none", "silu"):
            g = xb.causal_conv_bwd(**cuda(a), dy=dy.cuda(), act=act)
            with np.errstate(all="ignore"):
                ref = ob.causal_conv_grads(a["x"], a["w"], dy, a["bias"], act, a["state0"])
            if act == "none":
                assert np.isfinite(ref["dw"][:, K - 1]).all()
            for nm in ref:
                assert np.array_equal(g[nm].isfinite().cpu().numpy(), np.isfinite(ref[nm])), (nm, act)
