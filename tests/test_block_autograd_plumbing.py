"""Host logic of the differentiable block operators (``linear_rnn_mlstm_b200.autograd``)
on the CPU: the library's calls are replaced by stand-ins that compute with the
float64 oracles, so what is checked is which tensors reach which call and which
gradients come back (the kernels have their own parity tests)."""
import numpy as np
import pytest
import torch

import oracle.block as ob
import oracle.ssm as oscan
from linear_rnn_mlstm_b200 import autograd as xa
from linear_rnn_mlstm_b200 import binding as xb


def _t(x, like):
    return None if x is None else torch.from_numpy(np.asarray(x)).to(like.dtype)


@pytest.fixture
def stand_ins(monkeypatch):
    seen = {}

    def rmsnorm(x, gamma, residual=None, eps=1e-5):
        y, s, rstd = ob.rmsnorm(x, gamma, residual, eps)
        return _t(y, x), x if residual is None else _t(s, x), torch.from_numpy(rstd).float()

    def rmsnorm_bwd(dy, s, gamma, rstd, ds=None):
        seen["norm"] = dict(ds=ds, dy=dy)
        dx, dg = ob.rmsnorm_grads(dy, s, gamma, ds=ds, rstd=rstd)
        return _t(dx, s), _t(dg, gamma)

    def conv_fwd(x, w, bias=None, act="silu", state0=None):
        y, st = ob.causal_conv(x, w, bias, act, state0)
        return _t(y, x), _t(st, x)

    def conv_bwd(x, w, dy, bias=None, act="silu", state0=None, dstate=None):
        seen["conv"] = dict(dstate=dstate, dy=dy)
        g = ob.causal_conv_grads(x, w, dy, bias, act, state0, dstate)
        return dict(dx=_t(g["dx"], x), dw=_t(g["dw"], w), dbias=None if bias is None else _t(g["dbias"], bias),
                    dstate0=None if state0 is None else _t(g["dstate0"], x))

    def scan_fwd(x, delta, A, Bm, Cm, D=None, z=None, delta_bias=None, h0=None, softplus=True):
        y, h = oscan.scan(x, delta, A, Bm, Cm, D, z, delta_bias, h0, softplus)
        return _t(y, x), torch.from_numpy(h).float()

    def scan_bwd(x, delta, A, Bm, Cm, dy, D=None, z=None, delta_bias=None, h0=None, dh=None, softplus=True):
        seen["scan"] = dict(dh=dh, dy=dy)
        g = oscan.scan_grads(x, delta, A, Bm, Cm, dy, D, z, delta_bias, h0, dh, softplus)
        args = dict(x=x, delta=delta, A=A, Bm=Bm, Cm=Cm, D=D, z=z, delta_bias=delta_bias, h0=h0)
        return {"d" + k: None if v is None else _t(g["d" + k], v) for k, v in args.items()}

    for name, fn in (("rmsnorm", rmsnorm), ("rmsnorm_bwd", rmsnorm_bwd), ("causal_conv_fwd", conv_fwd), ("causal_conv_bwd", conv_bwd),
                     ("ssm_scan_fwd", scan_fwd), ("ssm_scan_bwd", scan_bwd)):
        monkeypatch.setattr(xb, name, fn)
    return seen


def _n(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64).float().requires_grad_()


def test_norm_with_and_without_a_residual(stand_ins):
    x, r, g = _n(0, 3, 8), _n(1, 3, 8), _n(2, 8)
    y, s = xa.rmsnorm(x, g, r)
    (y.sum() + 2 * s.sum()).backward()
    dx, dg = ob.rmsnorm_grads(np.ones((3, 8)), (x + r).detach(), g.detach(), ds=np.full((3, 8), 2.0))
    for t in (x, r):
        np.testing.assert_allclose(t.grad.numpy(), dx, rtol=1e-4, atol=1e-5)
    np.testing.assert_allclose(g.grad.numpy(), dg, rtol=1e-4, atol=1e-5)
    x2 = _n(3, 3, 8)
    y, s = xa.rmsnorm(x2, g.detach())
    assert s is x2
    y.sum().backward()
    assert stand_ins["norm"]["ds"] is None and x2.grad is not None
    y, s = xa.rmsnorm(x2, g.detach(), r)                     # the stream alone is used
    s.sum().backward()
    assert not stand_ins["norm"]["dy"].any()


def test_convolution_state_carries_gradients(stand_ins):
    t = dict(x=_n(0, 2, 5, 8), w=_n(1, 8, 4), bias=_n(2, 8), state0=_n(3, 2, 3, 8))
    y, st = xa.causal_conv(t["x"], t["w"], t["bias"], "silu", t["state0"])
    (y.sum() + (3 * st).sum()).backward()
    ref = ob.causal_conv_grads(*(t[k].detach() for k in ("x", "w")), np.ones((2, 5, 8)), t["bias"].detach(), "silu", t["state0"].detach(),
                               np.full((2, 3, 8), 3.0))
    for k in t:
        np.testing.assert_allclose(t[k].grad.numpy(), ref["d" + k], rtol=1e-4, atol=1e-5, err_msg=k)
    y, _ = xa.causal_conv(t["x"], t["w"])
    y.sum().backward()
    assert stand_ins["conv"]["dstate"] is None


def test_scan_gradients_reach_every_input(stand_ins):
    B, S, C, N, G = 2, 4, 8, 3, 2
    t = dict(x=_n(0, B, S, C), delta=_n(1, B, S, C), A=_n(2, C, N), Bm=_n(3, B, S, G, N), Cm=_n(4, B, S, G, N), D=_n(5, C),
             z=_n(6, B, S, C), delta_bias=_n(7, C), h0=_n(8, B, C, N))
    y, h = xa.ssm_scan(**t)
    (y.sum() + (2 * h).sum()).backward()
    ref = oscan.scan_grads(**{k: v.detach() for k, v in t.items()}, dy=np.ones((B, S, C)), dh=np.full((B, C, N), 2.0))
    for k in t:
        np.testing.assert_allclose(t[k].grad.numpy(), ref["d" + k], rtol=1e-4, atol=1e-4, err_msg=k)
    y, h = xa.ssm_scan(t["x"], t["delta"], t["A"], t["Bm"], t["Cm"])
    h.sum().backward()
    assert stand_ins["scan"]["dh"].dtype == torch.float32 and not stand_ins["scan"]["dy"].any()


def test_cotangents_that_start_off_a_16_byte_boundary_are_moved(stand_ins):
    """Cutting up a concatenation's gradient gives contiguous slices at any offset."""
    one = _n(9, 1)
    cut = lambda t, w: (torch.cat((one, t.flatten())) * w).sum()
    x, g, w4 = _n(0, 3, 8), _n(1, 8), _n(2, 8, 4)
    wy, wxs = _n(3, 25).detach(), _n(4, 41).detach()
    cut(xa.rmsnorm(x, g)[0], wy).backward()
    np.testing.assert_allclose(g.grad.numpy(), ob.rmsnorm_grads(wy[1:].reshape(3, 8), x.detach(), g.detach())[1], rtol=1e-4, atol=1e-5)
    xs = _n(5, 1, 5, 8)
    y, st = xa.causal_conv(xs, w4)
    (cut(y, wxs) + cut(st, wy)).backward()
    t = dict(x=xs, delta=xs.detach() * 0.5, A=_n(6, 8, 3), Bm=_n(7, 1, 5, 1, 3), Cm=_n(8, 1, 5, 1, 3))
    y, h = xa.ssm_scan(**t)
    (cut(y, wxs) + cut(h, wy)).backward()
    for call, names in (("norm", ["dy"]), ("conv", ["dy", "dstate"]), ("scan", ["dy", "dh"])):
        for nm in names:
            assert stand_ins[call][nm].data_ptr() % 16 == 0 and stand_ins[call][nm].is_contiguous(), (call, nm)
