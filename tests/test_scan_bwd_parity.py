"""GPU parity of the selective scan's backward (``xlstm_ssm_scan_bwd``) against
the float64 oracle (``oracle.ssm``).

Tolerances: bounds on the fp32 error, carried along both recurrences in 64 bits
(EPS = 2^-24).  A decay is within (4 + 35 |d A|) EPS, a step size within 32 EPS, the
gate and its slope within 70 EPS (4e-6) of their values, a product or sum adds EPS;
so for the states' magnitudes Mh and errors Eh
  Eh_t = a (Eh + (6 + 35 |d A|) EPS Mh) + 36 EPS |d x B|,
and the same for the cotangents g (Mg, Eg) from the last token on, with
|C e| (2 + 70) EPS entering at each token.  A gradient is a sum of products of
these; its error is the products' plus EPS times the longest chain of additions in
any place (at most 40 over states and channels, 130 over tokens) times the sum of
magnitudes."""
import numpy as np
import pytest
import torch

import oracle.ssm as oscan
from oracle.block import f64, sigmoid
from blockparity import BF16, EPS32, F32, cuda, normal, within
from linear_rnn_mlstm_b200 import autograd as xa
from linear_rnn_mlstm_b200 import binding as xb
from test_scan_parity import inputs

pytestmark = pytest.mark.gpu

KE = 70 * EPS32


def bounds(i, dy, dh, softplus=True):
    x, A, Bm, Cm = f64(i["x"]), np.abs(f64(i["A"])), np.abs(f64(i["Bm"])), np.abs(f64(i["Cm"]))
    B, S, C = x.shape
    N, G = A.shape[1], Bm.shape[2]
    d, slope = oscan._steps(i["delta"], i["delta_bias"], softplus)
    ax, u = np.abs(x), np.abs(d * x)
    skip = np.zeros(C) if i["D"] is None else np.abs(f64(i["D"]))
    z = None if i["z"] is None else f64(i["z"])
    ady = np.abs(f64(dy))
    e = ady if z is None else ady * np.abs(z * sigmoid(z))
    Mh = np.zeros((B, C, N)) if i.get("h0") is None else np.abs(f64(i["h0"]))
    Eh = np.zeros_like(Mh)
    hs = [(Mh, Eh)]
    out = {k: np.zeros_like(x) for k in ("dx", "ddelta", "dz")}
    sums = lambda v: v.reshape(B, G, C // G, N).sum(2)
    for t in range(S):
        ad = d[:, t, :, None] * A
        a, ub = np.exp(-ad), u[:, t, :, None] * oscan._rows(Bm, t, C)
        Eh = a * (Eh + (6 + 35 * ad) * EPS32 * Mh) + 36 * EPS32 * ub
        Mh = a * Mh + ub
        hs.append((Mh, Eh))
        if z is not None:
            y = (Mh * oscan._rows(Cm, t, C)).sum(2) + skip * ax[:, t]
            Ey = ((Eh + (N + 2) * EPS32 * Mh) * oscan._rows(Cm, t, C)).sum(2) + 2 * EPS32 * skip * ax[:, t]
            out["dz"][:, t] = ady[:, t] * 1.1 * (Ey + (KE + 4 * EPS32) * (1 + np.abs(z[:, t])) * y)
    Mr = np.zeros((B, C, N)) if dh is None else np.abs(f64(dh))
    Er = np.zeros_like(Mr)
    out.update(dA=np.zeros_like(A), dBm=np.zeros_like(Bm), dCm=np.zeros_like(Cm))
    dbm = np.zeros_like(x)
    for t in reversed(range(S)):
        et, ut, dt_ = e[:, t, :, None], u[:, t, :, None], d[:, t, :, None]
        Bt, Ct = oscan._rows(Bm, t, C), oscan._rows(Cm, t, C)
        Mg, Eg = Ct * et + Mr, Ct * et * (KE + 2 * EPS32) + Er
        Mh, Eh = hs[t + 1]
        out["dCm"][:, t] = sums(et * (Eh + (KE + 42 * EPS32) * Mh))
        out["dBm"][:, t] = sums(ut * (Eg + 76 * EPS32 * Mg))
        M1, E1 = (Bt * Mg).sum(2), (Bt * (Eg + 20 * EPS32 * Mg)).sum(2)
        ad = dt_ * A
        Mr, Er = np.exp(-ad) * Mg, np.exp(-ad) * (Eg + (6 + 35 * ad) * EPS32 * Mg)
        Mp, Ep = hs[t]
        Mw, Ew = Mr * Mp, Er * Mp + Mr * Ep + 2 * EPS32 * Mr * Mp
        M2, E2 = (A * Mw).sum(2), (A * (Ew + 25 * EPS32 * Mw)).sum(2)
        out["dA"] += (dt_ * (Ew + (34 + 130) * EPS32 * Mw)).sum(0)
        out["dx"][:, t] = d[:, t] * (E1 + 36 * EPS32 * M1) + skip * e[:, t] * (KE + 3 * EPS32)
        dbm[:, t] = slope[:, t] * (M2 + M1 * ax[:, t])
        out["ddelta"][:, t] = slope[:, t] * (E2 + E1 * ax[:, t]) + 50 * EPS32 * dbm[:, t]
    out["dh0"] = Er
    out["dD"] = (e * ax * (KE + 130 * EPS32)).sum((0, 1))
    out["ddelta_bias"] = (out["ddelta"] + 130 * EPS32 * dbm).sum((0, 1))
    return out


def check(i, softplus=True, seed=90, with_dh=True):
    B, S, C = i["x"].shape
    dy = normal(seed, B, S, C, dtype=i["x"].dtype)
    dh = normal(seed + 1, B, C, i["A"].shape[1]) if with_dh else None
    d = cuda({**i, "dy": dy, "dh": dh})
    got = xb.ssm_scan_bwd(**d, softplus=softplus)
    ref = oscan.scan_grads(**i, dy=dy, dh=dh, softplus=softplus)
    room = bounds(i, dy, dh, softplus)
    for nm, g in got.items():
        if i.get(nm[1:]) is None:
            assert g is None, nm
        else:
            within(g, ref[nm], room[nm], nm)
    again = xb.ssm_scan_bwd(**d, softplus=softplus)
    assert all(g is None or torch.equal(g, again[nm]) for nm, g in got.items())


@pytest.mark.parametrize("dtype", (F32, BF16), ids=("f32", "bf16"))
@pytest.mark.parametrize("N", (1, 3, 4, 8, 13, 16, 17, 32, 33, 64))
def test_over_state_sizes(N, dtype):
    check(inputs(2, 70, 24, N, dtype=dtype, seed=N))


@pytest.mark.parametrize("dtype", (F32, BF16), ids=("f32", "bf16"))
@pytest.mark.parametrize("B,S,C,N,G", [(1, 1, 8, 16, 1), (3, 2, 40, 16, 1), (1, 8, 16, 8, 2), (2, 9, 8, 16, 1), (2, 63, 72, 16, 1),
                                       (2, 64, 264, 16, 1), (1, 65, 48, 16, 2), (1, 700, 24, 16, 1), (2, 257, 80, 4, 5), (1, 130, 2048, 16, 1), (1, 2200, 8, 5, 1)])
def test_over_shapes(B, S, C, N, G, dtype):
    check(inputs(B, S, C, N, G, dtype=dtype, seed=S))


# enough CTAs for two channel groups a warp in bf16
@pytest.mark.parametrize("dtype", (F32, BF16), ids=("f32", "bf16"))
@pytest.mark.parametrize("B,S,C,N,G", [(2, 200, 2048, 16, 1), (2, 137, 2064, 16, 2), (2, 200, 1024, 32, 1), (3, 137, 520, 50, 1)])
def test_over_shapes_that_fill_the_sms(B, S, C, N, G, dtype):
    check(inputs(B, S, C, N, G, dtype=dtype, seed=S))


@pytest.mark.parametrize("with_dh", (False, True))
@pytest.mark.parametrize("full", (False, True))
def test_with_and_without_each_option(full, with_dh):
    i = inputs(2, 75, 16, 16, full=full)
    check(i, with_dh=with_dh)
    i["delta"], i["delta_bias"] = torch.rand_like(i["delta"]) * 0.2, None
    check(i, softplus=False, with_dh=with_dh)


def test_a_long_memory():
    check(inputs(1, 1500, 16, 16, step=1e-3, seed=2))


def test_without_tokens():
    i = inputs(2, 0, 16, 16)
    dh = normal(1, 2, 16, 16)
    g = xb.ssm_scan_bwd(**cuda({**i, "dy": i["x"], "dh": dh}))
    assert torch.equal(g["dh0"].cpu(), dh) and not g["dA"].any() and not g["dD"].any()


def test_gradients_against_differences_of_the_forward_kernel():
    i = inputs(2, 70, 16, 16, seed=7)
    d = cuda(i)
    dy, dh = normal(1, 2, 70, 16).cuda(), normal(2, 2, 16, 16).cuda()
    g = xb.ssm_scan_bwd(**d, dy=dy, dh=dh)

    def loss(**kw):
        y, h = xb.ssm_scan_fwd(**{**d, **kw})
        return float((y.double() * dy).sum() + (h.double() * dh).sum())

    base = loss()
    for k, nm in enumerate(("x", "delta", "A", "Bm", "Cm", "D", "z", "delta_bias", "h0")):
        v = normal(20 + k, *d[nm].shape).cuda()
        e = 1e-2
        diff = (loss(**{nm: d[nm] + e * v}) - loss(**{nm: d[nm] - e * v})) / (2 * e)
        got = float((g["d" + nm].double() * v).sum())
        # the difference's own error: e^2 of the third derivative and the forward's rounding over e
        scale = float((g["d" + nm].double() ** 2).sum().sqrt() * (v.double() ** 2).sum().sqrt())
        assert abs(got - diff) <= 5e-3 * scale + 1e-4 * abs(base), nm


def test_autograd_through_the_scan():
    i = inputs(2, 40, 16, 8, G=2)
    t = {k: v.cuda().requires_grad_() for k, v in i.items()}
    y, h = xa.ssm_scan(**t)
    wy, wh = normal(1, *y.shape).cuda(), normal(2, *h.shape).cuda()
    ((y * wy).sum() + (h * wh).sum()).backward()
    ref = oscan.scan_grads(**i, dy=wy.cpu(), dh=wh.cpu())
    room = bounds(i, wy.cpu(), wh.cpu())
    for nm in i:
        within(t[nm].grad, ref["d" + nm], room["d" + nm], nm)
    t2 = {k: v.detach().requires_grad_(k in ("x", "A")) for k, v in t.items()}
    y, h = xa.ssm_scan(**t2)
    h.sum().backward()                                            # the state alone, some inputs without gradients
    assert t2["x"].grad is not None and t2["delta"].grad is None


def test_a_captured_backward_replays_on_new_inputs():
    a, b = cuda(inputs(1, 200, 40, 16, dtype=BF16, seed=1)), cuda(inputs(1, 200, 40, 16, dtype=BF16, seed=50))
    for k, src in enumerate((a, b)):
        src["dy"] = normal(k, 1, 200, 40, dtype=BF16).cuda()
    held = {k: v.clone() for k, v in a.items()}
    xb.ssm_scan_bwd(**held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = xb.ssm_scan_bwd(**held)
    for src in (b, a):
        for k in held:
            held[k].copy_(src[k])
        graph.replay()
        want = xb.ssm_scan_bwd(**src)
        assert all(torch.equal(g[nm], want[nm]) for nm in g if g[nm] is not None)
