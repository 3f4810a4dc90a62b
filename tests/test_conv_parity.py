"""GPU parity of the short causal convolution (``xlstm_causal_conv_*``) against
the float64 oracle (``oracle.block``).

Tolerances, from the arithmetic (EPS = 2^-24): with P = |bias| + sum |w x|, the
pre-activation is off by at most (K + 1) EPS P, its Swish by 1.1 times that plus
the fast sigmoid's error (3e-6 relative for the |pre| < 20 here): 1e-5 of |y| and
of EPS-weighted P together stay below 8 EPS P + 4e-6 |y|.  A slope is off by at
most 0.5 of the pre-activation's error and 5e-6; dx and dw are sums of at most 4
and 64 + 64 such terms in a row: 1e-5 of the sums of magnitudes (|dy| (1 + P)
times |w| or |x|)."""
import numpy as np
import pytest
import torch

import oracle.block as ob
from blockparity import BF16, EPS32, F32, cuda, normal, within
from linear_rnn_mlstm_b200 import autograd as xa
from linear_rnn_mlstm_b200 import binding as xb

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1, 8, 4), (2, 2, 16, 4), (1, 3, 8, 4), (3, 17, 24, 3), (2, 65, 264, 4), (1, 130, 2048, 2), (5, 16, 40, 4), (1, 1021, 72, 3)]


def _inputs(B, S, C, K, dtype, seed=0):
    return dict(x=normal(seed, B, S, C, dtype=dtype), w=normal(seed + 1, C, K, scale=0.5), bias=normal(seed + 2, C, scale=0.3),
                state0=normal(seed + 3, B, K - 1, C, dtype=dtype))


def _size(a):
    """P = |bias| + sum |w x|, per output."""
    m = {k: np.abs(ob.f64(v)) for k, v in a.items()}
    return ob.causal_conv(m["x"], m["w"], m["bias"], "none", m["state0"])[0]


@pytest.mark.parametrize("dtype", (F32, BF16), ids=("f32", "bf16"))
@pytest.mark.parametrize("act", ("silu", "none"))
@pytest.mark.parametrize("B,S,C,K", SHAPES)
def test_forward(B, S, C, K, act, dtype):
    a = _inputs(B, S, C, K, dtype)
    for bare in (False, True):
        if bare:
            a = {**a, "bias": torch.zeros(C), "state0": torch.zeros(B, K - 1, C, dtype=dtype)}
        d = cuda(a)
        y, st = xb.causal_conv_fwd(d["x"], d["w"], None if bare else d["bias"], act, None if bare else d["state0"])
        yr, sr = ob.causal_conv(a["x"], a["w"], a["bias"], act, a["state0"])
        within(y, yr, 8 * EPS32 * _size(a) + 4e-6 * np.abs(yr), "y")
        np.testing.assert_array_equal(st.cpu().double().numpy(), sr)


@pytest.mark.parametrize("dtype", (F32, BF16), ids=("f32", "bf16"))
def test_lengths_leave_what_stands_behind_them(dtype):
    B, S, C, K = 6, 33, 40, 4
    a = _inputs(B, S, C, K, dtype)
    n = torch.tensor([0, 1, 2, 33, 99, -4], dtype=torch.int32)              # the last two are held to 33 and 0
    for b, m in enumerate((0, 1, 2, 33, 33, 0)):
        a["x"][b, m:] = float("nan")                                        # not to be read into anything
    d = cuda(a)
    y = torch.full((B, S, C), 5.0, dtype=dtype, device="cuda")
    got, st = xb.causal_conv_fwd(d["x"], d["w"], d["bias"], "silu", d["state0"], lengths=n.cuda(), y=y)
    clean = {**a, "x": torch.nan_to_num(a["x"])}
    yr, sr = ob.causal_conv(clean["x"], a["w"], a["bias"], "silu", a["state0"], lengths=n.tolist())
    for b, m in enumerate((0, 1, 2, 33, 33, 0)):
        assert torch.all(got[b, m:] == 5.0)
        if m:
            within(got[b, :m], yr[b, :m], 8 * EPS32 * _size(clean)[b, :m] + 4e-6 * np.abs(yr[b, :m]), "y")
    np.testing.assert_array_equal(st.cpu().double().numpy(), sr)


@pytest.mark.parametrize("dtype", (F32, BF16), ids=("f32", "bf16"))
@pytest.mark.parametrize("K", (2, 3, 4))
def test_steps_continue_a_prompt(K, dtype):
    B, S, C = 3, 9, 136
    a = _inputs(B, S, C, K, dtype)
    d = cuda(a)
    whole, last = xb.causal_conv_fwd(d["x"], d["w"], d["bias"], "silu", d["state0"])
    y, st = xb.causal_conv_fwd(d["x"][:, :4].contiguous(), d["w"], d["bias"], "silu", d["state0"])
    assert torch.equal(y, whole[:, :4])
    for t in range(4, S):
        y = xb.causal_conv_step(d["x"][:, t].contiguous(), d["w"], st, d["bias"], "silu")
        assert torch.equal(y, whole[:, t])
    assert torch.equal(st, last)


@pytest.mark.parametrize("dtype", (F32, BF16), ids=("f32", "bf16"))
@pytest.mark.parametrize("B,C,K", [(1, 8, 2), (41, 1032, 4), (300, 256, 3), (2, 65536, 4), (257, 2400, 4)])
@pytest.mark.parametrize("act", ("silu", "none"))
def test_step_over_many_rows_and_channels(B, C, K, act, dtype):
    a = _inputs(B, 1, C, K, dtype)
    d = cuda(a)
    y = xb.causal_conv_step(d["x"][:, 0].contiguous(), d["w"], d["state0"], d["bias"], act)
    yr, sr = ob.causal_conv(a["x"], a["w"], a["bias"], act, a["state0"])
    within(y, yr[:, 0], (8 * EPS32 * _size(a) + 4e-6 * np.abs(yr))[:, 0], "y")
    np.testing.assert_array_equal(d["state0"].cpu().double().numpy(), sr)


def test_an_empty_prompt_hands_the_state_on():
    d = cuda(_inputs(2, 0, 16, 4, F32))
    y, st = xb.causal_conv_fwd(d["x"], d["w"], d["bias"], "silu", d["state0"])
    assert y.shape == (2, 0, 16) and torch.equal(st, d["state0"])


def test_far_pre_activations():
    x = torch.tensor([-1e4, -200.0, -90.0, -88.5, 0.0, 90.0, 1e4, 3e38]).repeat(1, 1, 1).cuda()
    w = torch.tensor([[0.0, 1.0]]).repeat(8, 1).cuda()
    y, _ = xb.causal_conv_fwd(x, w)
    ref = ob.causal_conv(x.cpu(), w.cpu())[0]
    within(y, ref, 2e-5 * np.abs(ref) + 1e-36, "y")


@pytest.mark.parametrize("dtype", (F32, BF16), ids=("f32", "bf16"))
@pytest.mark.parametrize("act", ("silu", "none"))
@pytest.mark.parametrize("B,S,C,K", SHAPES + [(2, 700, 512, 4), (3, 0, 8, 3)])
def test_backward(B, S, C, K, act, dtype):
    a = _inputs(B, S, C, K, dtype)
    dy, dst = normal(7, B, S, C, dtype=dtype), normal(8, B, K - 1, C, dtype=dtype)
    d = cuda({**a, "dy": dy, "dstate": dst})
    got = xb.causal_conv_bwd(d["x"], d["w"], d["dy"], d["bias"], act, d["state0"], d["dstate"])
    ref = ob.causal_conv_grads(a["x"], a["w"], dy, a["bias"], act, a["state0"], dst)
    m = np.abs(ob.f64(dy)) * (1 + _size(a))
    sizes = ob.causal_conv_grads(np.abs(ob.f64(a["x"])), np.abs(ob.f64(a["w"])), m, None, "none", np.abs(ob.f64(a["state0"])),
                                 np.abs(ob.f64(dst)))
    for nm in ("dx", "dstate0", "dw", "dbias"):
        within(got[nm], ref[nm], 1e-5 * sizes[nm], nm)
    again = xb.causal_conv_bwd(d["x"], d["w"], d["dy"], d["bias"], act, d["state0"], d["dstate"])
    assert all(torch.equal(got[nm], again[nm]) for nm in got)
    bare = xb.causal_conv_bwd(d["x"], d["w"], d["dy"], act=act)
    refb = ob.causal_conv_grads(a["x"], a["w"], dy, None, act)
    assert bare["dbias"] is None and bare["dstate0"] is None
    for nm in ("dx", "dw"):
        within(bare[nm], refb[nm], 1e-5 * sizes[nm], nm)


def test_autograd_with_the_carried_state():
    a = _inputs(2, 6, 16, 4, F32)
    t = {k: v.cuda().requires_grad_() for k, v in a.items()}
    y, st = xa.causal_conv(t["x"], t["w"], t["bias"], "silu", t["state0"])
    wy, ws = normal(5, *y.shape).cuda(), normal(6, *st.shape).cuda()
    ((y * wy).sum() + (st * ws).sum()).backward()
    ref = ob.causal_conv_grads(a["x"], a["w"], wy.cpu(), a["bias"], "silu", a["state0"], ws.cpu())
    for nm in a:
        np.testing.assert_allclose(t[nm].grad.cpu().numpy(), ref["d" + nm], rtol=0, atol=2e-5 * np.abs(ref["d" + nm]).max(), err_msg=nm)
