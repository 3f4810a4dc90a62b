"""The mLSTM cell as a differentiable PyTorch op: ``xlstm_mlstm_fwd`` forward,
``xlstm_mlstm_bwd`` backward, through the ctypes binding (argument marshalling
only; every step runs in the library's kernels).

``mlstm_cell(q, k, v, i_pre, f_pre, o_pre)`` returns ``(h, C, n, m)`` for a
zero initial state; h and the final stabilised state (C', n') carry gradients
to q, k, v and the three gate pre-activations.  m, the stabiliser, is
bookkeeping of the stabilised units and is returned without a gradient.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import binding as xb

BWD_MAX_CHUNK = 64       # the backward kernels hold a chunk of tokens per thread


class MLSTMCellFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, i_pre, f_pre, o_pre, chunk, fgate):
        h, C, n, m = xb.mlstm_fwd(q, k, v, i_pre, f_pre, o_pre, chunk=chunk, fgate=fgate)
        ctx.save_for_backward(q, k, v, i_pre, f_pre, o_pre)
        ctx.chunk = min(chunk, BWD_MAX_CHUNK)
        ctx.fgate = fgate
        ctx.mark_non_differentiable(m)
        return h, C, n, m

    @staticmethod
    def backward(ctx, dh, dC, dn, dm):
        q, k, v, i_pre, f_pre, o_pre = ctx.saved_tensors
        if dh is None:
            dh = torch.zeros_like(q)
        g = xb.mlstm_bwd(q, k, v, i_pre, f_pre, o_pre, dh.to(q.dtype).contiguous(),
                         dC=None if dC is None else dC.float().contiguous(),
                         dn=None if dn is None else dn.float().contiguous(),
                         chunk=ctx.chunk, fgate=ctx.fgate)
        return g["dq"], g["dk"], g["dv"], g["di"], g["df"], g["do"], None, None


def mlstm_cell(q, k, v, i_pre, f_pre, o_pre, chunk=64, fgate="sigmoid"):
    """Differentiable mLSTM cell forward from a zero state: (h, C, n, m)."""
    return MLSTMCellFunction.apply(q, k, v, i_pre, f_pre, o_pre, chunk, fgate)


# ---------------------------------------------------- the block around the cell
# A backward pass may be captured into a CUDA graph; torch requires that no eager
# autograd graph of the same leaves is alive while it is.
def _cotangent(g, dtype):
    """A cotangent as the kernels take it: contiguous, on a 16-byte boundary (a slice of
    another operator's gradient may start anywhere)."""
    if g is None:
        return None
    g = g.to(dtype).contiguous()
    return g.clone() if g.data_ptr() % 16 else g


class RMSNormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gamma, residual, eps):
        y, s, rstd = xb.rmsnorm(x, gamma, residual=residual, eps=eps)
        ctx.save_for_backward(s, gamma, rstd)
        ctx.with_residual = residual is not None
        ctx.set_materialize_grads(False)
        return (y, s) if residual is not None else y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, ds=None):
        s, gamma, rstd = ctx.saved_tensors
        dy = torch.zeros_like(s) if dy is None else _cotangent(dy, s.dtype)
        dx, dgamma = xb.rmsnorm_bwd(dy, s, gamma, rstd, ds=_cotangent(ds, s.dtype))
        return dx, dgamma, dx if ctx.with_residual else None, None


def rmsnorm(x, gamma, residual=None, eps=1e-5):
    """Differentiable (y, s): s = x + residual (x itself without one), y its RMS norm."""
    if residual is None:
        return RMSNormFunction.apply(x, gamma, None, eps), x
    return RMSNormFunction.apply(x, gamma, residual, eps)


class CausalConvFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, bias, state0, act):
        y, state = xb.causal_conv_fwd(x, w, bias=bias, act=act, state0=state0)
        ctx.save_for_backward(x, w, bias, state0)
        ctx.act = act
        ctx.set_materialize_grads(False)
        return y, state

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dstate):
        x, w, bias, state0 = ctx.saved_tensors
        dy = torch.zeros_like(x) if dy is None else _cotangent(dy, x.dtype)
        g = xb.causal_conv_bwd(x, w, dy, bias=bias, act=ctx.act, state0=state0, dstate=_cotangent(dstate, x.dtype))
        return g["dx"], g["dw"], g["dbias"], g["dstate0"], None


def causal_conv(x, w, bias=None, act="silu", state0=None):
    """Differentiable causal convolution: (y, state), the state being the last K-1 inputs."""
    return CausalConvFunction.apply(x, w, bias, state0, act)


class SSMScanFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, delta, A, Bm, Cm, D, z, delta_bias, h0, softplus):
        y, h = xb.ssm_scan_fwd(x, delta, A, Bm, Cm, D=D, z=z, delta_bias=delta_bias, h0=h0, softplus=softplus)
        ctx.save_for_backward(x, delta, A, Bm, Cm, D, z, delta_bias, h0)
        ctx.softplus = softplus
        ctx.set_materialize_grads(False)
        return y, h

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh):
        x, delta, A, Bm, Cm, D, z, delta_bias, h0 = ctx.saved_tensors
        dy = torch.zeros_like(x) if dy is None else _cotangent(dy, x.dtype)
        g = xb.ssm_scan_bwd(x, delta, A, Bm, Cm, dy, D=D, z=z, delta_bias=delta_bias, h0=h0,
                            dh=_cotangent(dh, torch.float32), softplus=ctx.softplus)
        return tuple(g["d" + nm] for nm in ("x", "delta", "A", "Bm", "Cm", "D", "z", "delta_bias", "h0")) + (None,)


def ssm_scan(x, delta, A, Bm, Cm, D=None, z=None, delta_bias=None, h0=None, softplus=True):
    """Differentiable selective scan: (y, h), h the state after the last token."""
    return SSMScanFunction.apply(x, delta, A, Bm, Cm, D, z, delta_bias, h0, softplus)
