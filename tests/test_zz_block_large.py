"""The block operators on tensors of more than 2^31 elements (offsets past 32 bits),
checked against the same operators on their last part alone, and the binding's
refusal of views that the kernels cannot take (GPU)."""
import pytest
import torch

from blockparity import BF16, normal
from linear_rnn_mlstm_b200 import binding as xb

pytestmark = pytest.mark.gpu

S, C, CUT = 1_050_000, 2048, 1_049_000        # S * C = 2.15e9 > 2^31


def _big(seed):
    """[1, S, C] bf16: 1000 random tokens over and over."""
    return normal(seed, 1, 1000, C, dtype=BF16).cuda().repeat(1, S // 1000, 1)


def test_norm_and_convolution():
    x, gamma, w = _big(1), normal(2, C, mean=1.0).cuda(), normal(3, C, 4, scale=0.5).cuda()
    y, s, rstd = xb.rmsnorm(x, gamma, x)
    yt, st, rt = xb.rmsnorm(x[:, CUT:].contiguous(), gamma, x[:, CUT:].contiguous())
    assert torch.equal(y[:, CUT:], yt) and torch.equal(s[:, CUT:], st) and torch.equal(rstd[:, CUT:], rt)
    dx, _ = xb.rmsnorm_bwd(x, s, gamma, rstd)
    dxt, _ = xb.rmsnorm_bwd(x[:, CUT:].contiguous(), st, gamma, rt)
    assert torch.equal(dx[:, CUT:], dxt)
    del y, s, dx
    q, sc, _ = xb.rmsnorm_fp8(x, gamma)
    qt, sct, _ = xb.rmsnorm_fp8(x[:, CUT:].contiguous(), gamma)
    assert torch.equal(q[:, CUT:].contiguous().view(torch.uint8), qt.view(torch.uint8)) and torch.equal(sc[:, CUT:], sct)
    del q, sc
    y, last = xb.causal_conv_fwd(x, w)
    yt, lastt = xb.causal_conv_fwd(x[:, CUT:].contiguous(), w, state0=x[:, CUT - 3:CUT].contiguous())
    assert torch.equal(y[:, CUT:], yt) and torch.equal(last, lastt)
    g = xb.causal_conv_bwd(x, w, y)
    gt = xb.causal_conv_bwd(x[:, CUT:].contiguous(), w, yt, state0=x[:, CUT - 3:CUT].contiguous())
    assert torch.equal(g["dx"][:, CUT:], gt["dx"])


def test_scan():
    x, delta = _big(4), _big(5)
    A, bias = -torch.exp(normal(6, C, 16)).cuda(), torch.full((C,), -3.0).cuda()
    bc = normal(7, 2, 1, 1000, 1, 16, dtype=BF16).cuda().repeat(1, 1, S // 1000, 1, 1)
    y, h = xb.ssm_scan_fwd(x, delta, A, bc[0], bc[1], delta_bias=bias)
    cut = CUT - 3000
    cuts = lambda sl: [t[:, sl].contiguous() for t in (x, delta, bc[0], bc[1])]
    first = cuts(slice(0, cut))
    _, hc = xb.ssm_scan_fwd(first[0], first[1], A, first[2], first[3], delta_bias=bias)
    del first
    part = cuts(slice(cut, None))
    # one pass over the tokens in either call: the same operations from the same state
    yt, ht = xb.ssm_scan_fwd(part[0], part[1], A, part[2], part[3], delta_bias=bias, h0=hc)
    assert torch.equal(y[:, cut:], yt) and torch.equal(h, ht)
    del y
    g = xb.ssm_scan_bwd(x, delta, A, bc[0], bc[1], x, delta_bias=bias)
    gt = xb.ssm_scan_bwd(part[0], part[1], A, part[2], part[3], part[0], delta_bias=bias, h0=hc)
    for nm in ("dx", "ddelta", "dBm", "dCm"):
        # other segment borders, hence other roundings of the states; one bf16 rounding each
        a, b = g[nm][:, CUT:].float(), gt[nm][:, CUT - cut:].float()
        assert float((a - b).abs().max()) <= 2.0 ** -7 * float(b.abs().max()), nm


def test_views_the_kernels_cannot_take_are_refused():
    x, g, w = torch.zeros(2, 8, 64, device="cuda"), torch.ones(64, device="cuda"), torch.zeros(64, 4, device="cuda")
    halves = torch.zeros(2, 8, 128, device="cuda")[..., :64]                  # a half of a projection: rows apart
    with pytest.raises(ValueError, match="contiguous"):
        xb.rmsnorm(halves, g)
    with pytest.raises(ValueError, match="contiguous"):
        xb.causal_conv_fwd(halves, w)
    with pytest.raises(ValueError, match="contiguous"):
        xb.ssm_scan_fwd(x, halves, -torch.ones(64, 8, device="cuda"), torch.zeros(2, 8, 1, 8, device="cuda"),
                        torch.zeros(2, 8, 1, 8, device="cuda"))
    off = torch.zeros(2 * 8 * 64 + 1, device="cuda")[1:].view(2, 8, 64)       # dense, four bytes past a boundary
    with pytest.raises(xb.XlstmError) as e:
        xb.rmsnorm(off, g)
    assert e.value.status == xb.ERR_ALIGN
    with pytest.raises(ValueError, match="shape"):
        xb.causal_conv_fwd(x, w, state0=torch.zeros(2, 2, 64, device="cuda"))
    with pytest.raises(TypeError):
        xb.causal_conv_fwd(x, w, lengths=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(TypeError):
        xb.ssm_scan_step(x[:, 0].contiguous(), x[:, 0].contiguous(), -torch.ones(64, 8, device="cuda"), torch.zeros(2, 1, 8, device="cuda"),
                         torch.zeros(2, 1, 8, device="cuda"), torch.zeros(2, 64, 8, device="cuda", dtype=BF16))


def test_batches_of_nothing():
    w, A = torch.zeros(64, 4, device="cuda"), -torch.ones(64, 8, device="cuda")
    x, bc = torch.zeros(0, 5, 64, device="cuda"), torch.zeros(0, 5, 1, 8, device="cuda")
    y, st = xb.causal_conv_fwd(x, w)
    assert y.shape == (0, 5, 64) and st.shape == (0, 3, 64)
    y, h = xb.ssm_scan_fwd(x, x, A, bc, bc)
    assert y.shape == (0, 5, 64) and h.shape == (0, 64, 8)
    g = xb.ssm_scan_bwd(x, x, A, bc, bc, x)
    assert not g["dA"].any()
    g = xb.causal_conv_bwd(x, w, x)
    assert not g["dw"].any()
    assert xb.causal_conv_step(x[:, 0], w, st).shape == (0, 64)
    assert xb.ssm_scan_step(x[:, 0], x[:, 0], A, bc[:, 0], bc[:, 0], h).shape == (0, 64)
    y, s, rstd = xb.rmsnorm(x, torch.ones(64, device="cuda"))
    assert y.shape == x.shape and rstd.shape == (0, 5)
