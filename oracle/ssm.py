"""Float64 numpy oracle of the selective state-space scan and its gradients,
token by token from the definition in ``include/xlstm_mlstm.h`` (test
infrastructure only; nothing is shared with the kernels)."""
from __future__ import annotations

import numpy as np

from .block import f64, sigmoid


def _steps(delta, delta_bias, softplus):
    v = f64(delta)
    if delta_bias is not None:
        v = v + f64(delta_bias)
    return (np.logaddexp(v, 0.0), sigmoid(v)) if softplus else (v, np.ones_like(v))


def _rows(m, t, C):
    """[B, S, G, N] at token t, one row per channel: [B, C, N]."""
    return np.repeat(m[:, t], C // m.shape[2], axis=1)


def scan(x, delta, A, Bm, Cm, D=None, z=None, delta_bias=None, h0=None, softplus=True, lengths=None):
    """(y [B, S, C], h [B, C, N]); y is zero behind a row's length."""
    x, A, Bm, Cm = f64(x), f64(A), f64(Bm), f64(Cm)
    B, S, C = x.shape
    d, _ = _steps(delta, delta_bias, softplus)
    h = np.zeros((B, C, A.shape[1])) if h0 is None else f64(h0).copy()
    n = np.full(B, S) if lengths is None else np.clip(f64(lengths), 0, S)
    y = np.zeros_like(x)
    for t in range(S):
        new = np.exp(d[:, t, :, None] * A) * h + (d[:, t] * x[:, t])[..., None] * _rows(Bm, t, C)
        live = (t < n)[:, None]
        h = np.where(live[..., None], new, h)
        v = (_rows(Cm, t, C) * h).sum(2)
        if D is not None:
            v = v + f64(D) * x[:, t]
        if z is not None:
            zt = f64(z)[:, t]
            v = v * zt * sigmoid(zt)
        y[:, t] = np.where(live, v, 0)
    return y, h


def scan_grads(x, delta, A, Bm, Cm, dy, D=None, z=None, delta_bias=None, h0=None, dh=None, softplus=True):
    """dict dx, ddelta, dA, dBm, dCm, dD, dz, ddelta_bias, dh0 of sum(dy y) + sum(dh h)."""
    x, A, Bm, Cm, dy = f64(x), f64(A), f64(Bm), f64(Cm), f64(dy)
    B, S, C = x.shape
    N, G = A.shape[1], Bm.shape[2]
    d, slope = _steps(delta, delta_bias, softplus)
    h = np.zeros((B, C, N)) if h0 is None else f64(h0)
    hs = [h]
    for t in range(S):
        hs.append(np.exp(d[:, t, :, None] * A) * hs[-1] + (d[:, t] * x[:, t])[..., None] * _rows(Bm, t, C))
    skip = np.zeros(C) if D is None else f64(D)
    out = {}
    if z is not None:
        zz = f64(z)
        sg = sigmoid(zz)
        y = np.stack([(_rows(Cm, t, C) * hs[t + 1]).sum(2) for t in range(S)], 1) if S else np.zeros_like(x)
        out["dz"] = dy * (y + skip * x) * sg * (1 + zz * (1 - sg))
        dy = dy * zz * sg
    g = np.zeros((B, C, N)) if dh is None else f64(dh).copy()
    out.update(dx=np.zeros_like(x), ddelta=np.zeros_like(x), dA=np.zeros_like(A), dBm=np.zeros_like(Bm), dCm=np.zeros_like(Cm))
    for t in reversed(range(S)):
        g = g + _rows(Cm, t, C) * dy[:, t, :, None]
        out["dCm"][:, t] = (hs[t + 1] * dy[:, t, :, None]).reshape(B, G, -1, N).sum(2)
        out["dBm"][:, t] = (g * (d[:, t] * x[:, t])[..., None]).reshape(B, G, -1, N).sum(2)
        du = (g * _rows(Bm, t, C)).sum(2)
        ga = g * np.exp(d[:, t, :, None] * A)
        w = ga * hs[t]
        out["dA"] += (w * d[:, t, :, None]).sum(0)
        out["dx"][:, t] = du * d[:, t] + dy[:, t] * skip
        out["ddelta"][:, t] = ((w * A).sum(2) + du * x[:, t]) * slope[:, t]
        g = ga
    out.update(dh0=g, dD=(dy * x).sum((0, 1)), ddelta_bias=out["ddelta"].sum((0, 1)))
    return out
