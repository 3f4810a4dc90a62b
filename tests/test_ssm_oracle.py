"""Pins of the selective scan's oracle (``oracle.ssm``): a hand-worked case, the
closed form of a constant input, a cumulative sum as the case without decay, two
halves joined by the state, and central differences for every gradient."""
import numpy as np

import oracle.ssm as os_


def _inputs(B=2, S=5, C=6, N=3, G=2, seed=0):
    g = np.random.default_rng(seed)
    n = lambda *s: g.normal(size=s)
    return dict(x=n(B, S, C), delta=n(B, S, C), A=-np.exp(n(C, N)), Bm=n(B, S, G, N), Cm=n(B, S, G, N), D=n(C), z=n(B, S, C),
                delta_bias=n(C), h0=n(B, C, N))


def test_by_hand():
    ln2 = np.log(2.0)
    y, h = os_.scan([[[3.0], [1.0]]], [[[1.0], [2.0]]], [[-ln2]], [[[[2.0]], [[5.0]]]], [[[[1.0]], [[10.0]]]], D=[0.5], h0=[[[4.0]]],
                    softplus=False)
    # h1 = 4 / 2 + 1 * 3 * 2 = 8, y1 = 8 + 1.5; h2 = 8 / 4 + 2 * 1 * 5 = 12, y2 = 120 + 0.5
    np.testing.assert_allclose(y[0, :, 0], [9.5, 120.5])
    np.testing.assert_allclose(h, [[[12.0]]])


def test_constant_input_reaches_the_geometric_sum():
    S, a = 40, 0.8
    one = np.ones((1, S, 1))
    y, h = os_.scan(one, one, [[np.log(a)]], one[..., None], one[..., None], softplus=False)
    np.testing.assert_allclose(y[0, :, 0], (1 - a ** np.arange(1, S + 1)) / (1 - a), rtol=1e-12)


def test_without_decay_it_is_a_running_sum_and_softplus_is_torchs():
    import torch
    i = _inputs(G=1, N=1)
    i["A"] = np.zeros_like(i["A"])
    y, _ = os_.scan(i["x"], i["delta"], i["A"], np.ones_like(i["Bm"]), np.ones_like(i["Cm"]))
    d = torch.nn.functional.softplus(torch.from_numpy(i["delta"])).numpy()
    np.testing.assert_allclose(y, np.cumsum(d * i["x"], 1), rtol=1e-10)


def test_two_halves_and_lengths():
    i = _inputs()
    y, h = os_.scan(**i)
    cut = lambda s: {k: v[:, s] if k in ("x", "delta", "Bm", "Cm", "z") else v for k, v in i.items()}
    y1, h1 = os_.scan(**cut(slice(0, 2)))
    y2, h2 = os_.scan(**{**cut(slice(2, None)), "h0": h1})
    np.testing.assert_allclose(np.concatenate([y1, y2], 1), y, rtol=1e-13)
    np.testing.assert_allclose(h2, h, rtol=1e-13)
    y3, h3 = os_.scan(**i, lengths=[2, 0])
    np.testing.assert_allclose(y3[0, :2], y1[0])
    np.testing.assert_allclose(h3, np.stack([h1[0], i["h0"][1]]))
    assert not y3[0, 2:].any() and not y3[1].any()


def test_gradients_against_differences():
    for softplus in (True, False):
        i = _inputs(seed=3)
        if not softplus:
            i["delta"], i["delta_bias"] = np.abs(i["delta"]) * 0.3, np.abs(i["delta_bias"]) * 0.3
        g = np.random.default_rng(9)
        dy, dh = g.normal(size=i["x"].shape), g.normal(size=i["h0"].shape)
        grads = os_.scan_grads(dy=dy, dh=dh, softplus=softplus, **i)

        def loss(**kw):
            y, h = os_.scan(softplus=softplus, **{**i, **kw})
            return (y * dy).sum() + (h * dh).sum()

        for nm in i:
            v = g.normal(size=i[nm].shape)
            e = 1e-6
            diff = (loss(**{nm: i[nm] + e * v}) - loss(**{nm: i[nm] - e * v})) / (2 * e)
            np.testing.assert_allclose((grads["d" + nm] * v).sum(), diff, rtol=2e-6, err_msg=nm)
