"""Float64 numpy oracles of the block's operators around the cells (test
infrastructure only): the residual addition with root-mean-square norm and its
e4m3 output, and the short causal convolution, each with its gradients.

Everything is written per token or per tap from the definitions in
``include/xlstm_mlstm.h``; nothing is shared with the kernels.
"""
from __future__ import annotations

import numpy as np

F8_MAX = 448.0                # largest finite e4m3 value
SCALE_MIN = 2.0 ** -126


def f64(x):
    """Any array or torch tensor (any dtype) as float64; None stays None."""
    if x is None:
        return None
    if hasattr(x, "detach"):
        x = x.detach().to("cpu").double().numpy()
    return np.asarray(x, dtype=np.float64)


def sigmoid(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


# -------------------------------------------------------------------- norm
def rmsnorm(x, gamma, residual=None, eps=1e-5):
    """(y, s, rstd) over the last axis."""
    s = f64(x) if residual is None else f64(x) + f64(residual)
    rstd = 1.0 / np.sqrt((s * s).mean(-1) + eps)
    return s * rstd[..., None] * f64(gamma), s, rstd


def e4m3(v):
    """To the nearest e4m3 number, ties to even, held to +-448."""
    v = f64(v)
    e = np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6)))
    step = 2.0 ** (e - 3)                       # 2^-9 below the smallest normal, 2^-6
    return np.clip(np.rint(v / step) * step, -F8_MAX, F8_MAX)


def quantise(y, group):
    """(q, scales): one scale per ``group`` channels, one per row for 0."""
    C = y.shape[-1]
    g = y.reshape(*y.shape[:-1], -1, group or C)
    scale = np.maximum(np.abs(g).max(-1) / F8_MAX, SCALE_MIN)
    return e4m3(g / scale[..., None]).reshape(y.shape), scale


def rmsnorm_grads(dy, s, gamma, eps=1e-5, ds=None, rstd=None):
    """(dx, dgamma) of sum(dy y) + sum(ds s)."""
    dy, s, gamma = f64(dy), f64(s), f64(gamma)
    rstd = 1.0 / np.sqrt((s * s).mean(-1) + eps) if rstd is None else f64(rstd)
    n = s * rstd[..., None]
    g = dy * gamma
    dx = rstd[..., None] * (g - n * (g * n).mean(-1, keepdims=True))
    if ds is not None:
        dx = dx + f64(ds)
    return dx, (dy * n).reshape(-1, n.shape[-1]).sum(0)


# -------------------------------------------------------------- convolution
def _pre(x, w, bias, state0):
    x, w = f64(x), f64(w)
    B, S, C = x.shape
    K = w.shape[1]
    before = np.zeros((B, K - 1, C)) if state0 is None else f64(state0)
    seen = np.concatenate([before, x], axis=1)
    pre = np.zeros((B, S, C)) if bias is None else np.tile(f64(bias), (B, S, 1))
    for t in range(S):
        for k in range(K):
            pre[:, t] += w[:, k] * seen[:, t + k]
    return pre, seen


def causal_conv(x, w, bias=None, act="silu", state0=None, lengths=None):
    """(y, state): y [B, S, C] (zero behind a row's length), state [B, K-1, C]."""
    pre, seen = _pre(x, w, bias, state0)
    y = pre * sigmoid(pre) if act == "silu" else pre
    B, S, _ = y.shape
    K = f64(w).shape[1]
    n = [S] * B if lengths is None else [min(max(int(v), 0), S) for v in lengths]
    state = np.stack([seen[b, n[b]:n[b] + K - 1] for b in range(B)]) if B else seen[:, :K - 1]
    for b in range(B):
        y[b, n[b]:] = 0
    return y, state


def causal_conv_grads(x, w, dy, bias=None, act="silu", state0=None, dstate=None):
    """dict dx, dw, dbias, dstate0 of sum(dy y) + sum(dstate state)."""
    pre, seen = _pre(x, w, bias, state0)
    w, d = f64(w), f64(dy)
    if act == "silu":
        sg = sigmoid(pre)
        d = d * sg * (1.0 + pre * (1.0 - sg))
    K, S = w.shape[1], pre.shape[1]
    dseen, dw = np.zeros_like(seen), np.zeros_like(w)
    for k in range(K):
        dseen[:, k:k + S] += w[:, k] * d
        dw[:, k] = (d * seen[:, k:k + S]).sum((0, 1))
    if dstate is not None:
        dseen[:, S:] += f64(dstate)
    return dict(dx=dseen[:, K - 1:], dstate0=dseen[:, :K - 1], dw=dw, dbias=d.sum((0, 1)))
