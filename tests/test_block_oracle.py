"""Pins of the block operators' oracle (``oracle.block``): hand-worked values,
torch's own float64 routines, central differences for every gradient, and the
e4m3 rounding against torch's conversion."""
import numpy as np
import torch

import oracle.block as ob


def _g(seed):
    return np.random.default_rng(seed)


def test_rmsnorm_by_hand():
    # s = (3, 4): mean square 12.5; eps 3.5 makes the root 4
    y, s, rstd = ob.rmsnorm([[1.0, 4.0]], [2.0, 0.5], [[2.0, 0.0]], eps=3.5)
    np.testing.assert_allclose(s, [[3, 4]])
    np.testing.assert_allclose(rstd, [0.25])
    np.testing.assert_allclose(y, [[1.5, 0.5]])


def test_rmsnorm_is_layer_norm_of_centred_rows():
    g = _g(1)
    x = g.normal(size=(5, 16))
    x -= x.mean(1, keepdims=True)
    y, _, _ = ob.rmsnorm(x, np.ones(16), eps=0.1)
    ref = torch.nn.functional.layer_norm(torch.from_numpy(x), (16,), eps=0.1).numpy()
    np.testing.assert_allclose(y, ref, rtol=1e-12, atol=1e-12)


def test_e4m3_is_torchs_conversion():
    g = _g(2)
    v = np.concatenate([g.normal(size=4000) * 2.0 ** g.integers(-12, 8, 4000), np.arange(-64, 64) * 2.0 ** -10,
                        [0.0, 448.0, -448.0, 17.0, 19.0]]).astype(np.float32)
    v = np.clip(v, -448, 448)
    ref = torch.from_numpy(v).to(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(ob.e4m3(v), ref)


def test_quantise_scales_and_zero_groups():
    y = np.zeros((2, 64))
    y[0, :32] = np.linspace(-896, 896, 32)
    q, scale = ob.quantise(y, 32)
    assert scale.shape == (2, 2) and scale[0, 0] == 2.0 and scale[0, 1] == ob.SCALE_MIN
    assert np.abs(q).max() == 448 and not q[1].any()
    assert ob.quantise(y, 0)[1].shape == (2, 1)


def _difference(f, x, v, h=1e-6):
    return (f(x + h * v) - f(x - h * v)) / (2 * h)


def test_rmsnorm_gradients_against_differences():
    g = _g(3)
    s, gamma, dy, ds = g.normal(size=(3, 8)), g.normal(size=8), g.normal(size=(3, 8)), g.normal(size=(3, 8))
    dx, dgamma = ob.rmsnorm_grads(dy, s, gamma, 0.01, ds)

    def loss(a, b):
        y, st, _ = ob.rmsnorm(a, b, eps=0.01)
        return (dy * y).sum() + (ds * st).sum()

    v, u = g.normal(size=s.shape), g.normal(size=8)
    np.testing.assert_allclose((dx * v).sum(), _difference(lambda a: loss(a, gamma), s, v), rtol=1e-7)
    np.testing.assert_allclose((dgamma * u).sum(), _difference(lambda b: loss(s, b), gamma, u), rtol=1e-7)


def test_conv_by_hand():
    x = [[[1.0], [2.0], [3.0]]]
    y, state = ob.causal_conv(x, [[10.0, 1.0]], [0.5], "none", [[[7.0]]])
    np.testing.assert_allclose(y[0, :, 0], [71.5, 12.5, 23.5])
    np.testing.assert_allclose(state, [[[3.0]]])
    y, state = ob.causal_conv(x, [[10.0, 1.0]], None, "none", [[[7.0]]], lengths=[0])
    assert not y.any() and state[0, 0, 0] == 7.0


def test_conv_is_torchs_padded_convolution():
    g = _g(4)
    x, w, b = g.normal(size=(2, 9, 8)), g.normal(size=(8, 4)), g.normal(size=8)
    y, _ = ob.causal_conv(x, w, b, "silu")
    t = torch.nn.functional.conv1d(torch.from_numpy(x).transpose(1, 2), torch.from_numpy(w)[:, None], torch.from_numpy(b),
                                   padding=3, groups=8)[..., :9]
    np.testing.assert_allclose(y, torch.nn.functional.silu(t).transpose(1, 2).numpy(), rtol=1e-12, atol=1e-12)


def test_conv_in_two_halves_with_the_carried_state():
    g = _g(5)
    x, w = g.normal(size=(2, 7, 8)), g.normal(size=(8, 3))
    whole, last = ob.causal_conv(x, w)
    a, st = ob.causal_conv(x[:, :1], w)
    b, st = ob.causal_conv(x[:, 1:], w, state0=st)
    np.testing.assert_allclose(np.concatenate([a, b], 1), whole, rtol=1e-13, atol=1e-13)
    np.testing.assert_array_equal(st, last)


def test_conv_gradients_against_differences():
    g = _g(6)
    for act in ("silu", "none"):
        for S in (1, 2, 6):
            a = dict(x=g.normal(size=(2, S, 3)), w=g.normal(size=(3, 4)), bias=g.normal(size=3), state0=g.normal(size=(2, 3, 3)))
            dy, dst = g.normal(size=(2, S, 3)), g.normal(size=(2, 3, 3))
            grads = ob.causal_conv_grads(dy=dy, dstate=dst, act=act, **a)

            def loss(**kw):
                y, st = ob.causal_conv(act=act, **{**a, **kw})
                return (y * dy).sum() + (st * dst).sum()

            for nm in a:
                v = g.normal(size=a[nm].shape)
                got = _difference(lambda t: loss(**{nm: t}), a[nm], v)
                np.testing.assert_allclose((grads["d" + nm] * v).sum(), got, rtol=1e-6, err_msg=nm)
