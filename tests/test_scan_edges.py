"""GPU tests of the selective scan at its edges: lanes without a channel, growing
states, long walks of one CTA, infinities and NaN inside a sequence.  The
tolerances are those of the parity tests (``test_scan_parity``, ``test_scan_bwd_parity``)."""
import numpy as np
import pytest
import torch

import oracle.ssm as oscan
from blockparity import BF16, EPS32, F32, cuda, within
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


# ------------------------------------------------------------ growing states
# exp(step A) over a segment is past fp32 although no state, cotangent or gradient is.
STEP = 1.625                                                      # sums of it are exact; 64 of them: e^104


@pytest.mark.parametrize("dtype", (F32, BF16), ids=("f32", "bf16"))
def test_growth_of_a_state_that_is_still_zero(dtype):
    i = inputs(1, 2048, 16, 16, dtype=dtype, seed=3)
    i.update(A=0.5 + torch.rand(16, 16, generator=torch.Generator().manual_seed(1)) / 2, delta=torch.full_like(i["delta"], STEP),
             delta_bias=None, h0=None)
    i["x"][:, :-20] = 0                                           # a prompt padded on the left
    y, h = xb.ssm_scan_fwd(**cuda(i), softplus=False)
    yr, hr = oscan.scan(**i, softplus=False)
    ey, eh = bounds(i, softplus=False)
    within(h, hr, eh, "h")
    within(y, yr, ey + 4e-6 * np.abs(yr), "y")


@pytest.mark.parametrize("dtype", (F32, BF16), ids=("f32", "bf16"))
def test_growth_of_a_small_state(dtype):
    i = inputs(1, 2048, 16, 16, dtype=dtype, seed=4)
    i.update(A=torch.ones(16, 16), delta=torch.full_like(i["delta"], STEP), delta_bias=None, h0=1e-15 * torch.rand(1, 16, 16))
    i["x"].zero_()
    i["delta"][:, 64:] = 0                                        # and no further
    y, h = xb.ssm_scan_fwd(**cuda(i), softplus=False)
    yr, hr = oscan.scan(**i, softplus=False)
    ey, eh = bounds(i, softplus=False)
    within(h, hr, eh, "h")
    within(y, yr, ey + 4e-6 * np.abs(yr), "y")


@pytest.mark.parametrize("dtype", (F32, BF16), ids=("f32", "bf16"))
@pytest.mark.parametrize("C,N", [(16, 16), (16, 5), (2048, 16)])
def test_gradients_of_growing_states(C, N, dtype):
    """All inputs are positive, so no term cancels another and every gradient is relatively
    as exact as its factors: (6 + 35 * 1.625) EPS a token for a state and for a cotangent,
    64 tokens each, and 600 EPS for the chains of sums: under 9000 EPS."""
    pos = lambda seed, *shape: (0.1 + torch.rand(shape, generator=torch.Generator().manual_seed(seed)))
    S = 256
    zero_then = lambda t, a, b: t * torch.tensor([float(a <= k < b) for k in range(S)]).view(1, S, 1)
    base = dict(delta=torch.full((1, S, C), STEP), A=torch.ones(C, N), Bm=pos(1, 1, S, 1, N), Cm=pos(2, 1, S, 1, N),
                D=None, z=None, delta_bias=None)
    first = {**base, "x": zero_then(pos(3, 1, S, C), S - 20, S), "h0": None, "dy": zero_then(pos(4, 1, S, C), 0, 20)}
    small = {**base, "x": zero_then(1e-15 * pos(3, 1, S, C), 0, 64), "h0": 1e-15 * pos(5, 1, C, N),
             "dy": zero_then(1e-15 * pos(4, 1, S, C), 63, 64), "delta": zero_then(base["delta"], 0, 64)}
    for i in (first, small):
        i = {k: v.to(dtype) if k in ("x", "delta", "Bm", "Cm", "dy") else v for k, v in i.items()}
        got = xb.ssm_scan_bwd(**cuda(i), softplus=False)
        ref = oscan.scan_grads(**i, softplus=False)
        assert max(np.abs(r).max() for r in (ref["dx"], ref["dh0"])) > 1e10
        for nm, g in got.items():
            if g is not None:
                within(g, ref[nm], 9000 * EPS32 * np.abs(ref[nm]), nm)


# ------------------------------------------- infinities and NaN inside a sequence
def _same_finite(got, ref, room, what):
    """Finite where the reference is, and there within its bound."""
    got, ref = got.detach().cpu().double().numpy(), np.asarray(ref, np.float64)
    assert np.array_equal(np.isfinite(got), np.isfinite(ref)), what
    ok = np.isfinite(ref)
    got, ref, room = got[ok], ref[ok], room[ok]
    assert np.all(np.abs(got - ref) <= room + 2.0 ** -23 * (np.abs(ref) + room) + 1e-37), what


BAD = (float("nan"), float("inf"), float("-inf"))


@pytest.mark.parametrize("bad", BAD, ids=("nan", "inf", "-inf"))
@pytest.mark.parametrize("name", ("x", "Bm", "Cm", "z"))
@pytest.mark.parametrize("C,N", [(16, 16), (4096, 16), (16, 5)])
def test_a_value_that_is_not_finite_spoils_what_the_definition_says(C, N, name, bad):
    """In segments and in one pass: earlier tokens, other channels and other rows stay finite."""
    i = inputs(2, 200, C, N, seed=11)
    clean = {k: v.clone() if v is not None else None for k, v in i.items()}
    i[name][(0, 90, 3) if name in ("x", "z") else (0, 90, 0, 2)] = bad
    y, h = xb.ssm_scan_fwd(**cuda(i))
    with np.errstate(all="ignore"):
        yr, hr = oscan.scan(**i)
    ey, eh = bounds(clean)
    _same_finite(y, yr, ey + 4e-6 * np.abs(np.nan_to_num(yr, posinf=0, neginf=0)), "y")
    _same_finite(h, hr, eh, "h")


@pytest.mark.parametrize("C,N", [(16, 16), (4096, 16), (16, 5)])
def test_a_nan_step_size(C, N):
    i = inputs(2, 200, C, N, seed=12)
    i["delta"][0, 90, 3] = float("nan")
    d = cuda(i)
    y, h = xb.ssm_scan_fwd(**d)
    with np.errstate(all="ignore"):
        yr, hr = oscan.scan(**i)
    assert np.array_equal(y.isfinite().cpu().numpy(), np.isfinite(yr)) and np.array_equal(h.isfinite().cpu().numpy(), np.isfinite(hr))
    dy = torch.zeros(2, 200, C)
    dy[:, 95:] = 1.0                                              # and none where the NaN stands
    g = xb.ssm_scan_bwd(**d, dy=dy.cuda())
    with np.errstate(all="ignore"):
        ref = oscan.scan_grads(**i, dy=dy.numpy())
    for nm in ref:
        if nm != "dz":                                            # a zero cotangent of a NaN is a NaN, or not, by the order of its factors
            assert np.array_equal(g[nm].isfinite().cpu().numpy(), np.isfinite(ref[nm])), nm


def test_a_cotangent_that_is_not_finite():
    i = inputs(2, 200, 16, 16, seed=13)
    for bad in BAD:
        dy = torch.ones(2, 200, 16)
        dy[1, 130, 5] = bad
        g = xb.ssm_scan_bwd(**cuda(i), dy=dy.cuda())
        with np.errstate(all="ignore"):
            ref = oscan.scan_grads(**i, dy=dy.numpy())
        for nm in ref:
            assert np.array_equal(g[nm].isfinite().cpu().numpy(), np.isfinite(ref[nm])), (nm, bad)


@pytest.mark.parametrize("C,N", [(16, 16), (2048, 16), (16, 5), (16, 12)])
def test_gradients_before_an_infinite_step_size(C, N):
    """It ends the memory (its decay is zero): what came before stays finite."""
    i = inputs(2, 200, C, N, seed=14)
    i["delta"][0, 90, 3] = float("inf")
    for first, last in ((0, 200), (0, 90), (95, 200)):
        dy = torch.zeros(2, 200, C)
        dy[:, first:last] = 1.0
        g = xb.ssm_scan_bwd(**cuda(i), dy=dy.cuda())
        with np.errstate(all="ignore"):
            ref = oscan.scan_grads(**i, dy=dy.numpy())
        assert np.isfinite(ref["dx"][0, :90, 3]).all()
        for nm in ref:
            if nm != "dz":
                assert np.array_equal(g[nm].isfinite().cpu().numpy(), np.isfinite(ref[nm])), (nm, first, last)
