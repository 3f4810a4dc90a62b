"""The block operators run together, as a model runs them (GPU): residual norm ->
projection -> causal convolution -> cell -> gate, with the mLSTM cell and its
epilogue and with the selective scan; prompts, token by token from the carried
states, a captured decode step, and gradients through a whole block.

Tolerances: fp32 throughout.  Each operator is within 1e-5 of its terms'
magnitudes (their own tests); a block chains four of them and two matrix products
of width <= 64 whose fp32 rounding is 64 EPS = 4e-6 of their magnitudes, so 1e-4
of an output's scale (max |y|) bounds both the comparison with 64 bits and that of
two orders of the same computation."""
import numpy as np
import pytest
import torch

import oracle
import oracle.block as ob
import oracle.ssm as oscan
from oracle.headnorm import headnorm_gate as oracle_headnorm
from blockparity import normal
from linear_rnn_mlstm_b200 import autograd as xa
from linear_rnn_mlstm_b200 import binding as xb

pytestmark = pytest.mark.gpu

B, S, C, N, K = 2, 37, 64, 16, 4


def _weights():
    return dict(gamma=normal(1, C, scale=0.1, mean=1.0), w_in=normal(2, C, 2 * C, scale=C ** -0.5), conv=normal(3, C, K, scale=0.5),
                bias=normal(4, C, scale=0.1), w_d=normal(5, C, C, scale=0.3 * C ** -0.5), delta_bias=normal(6, C, scale=0.5, mean=-3.0),
                w_bc=normal(7, C, 2 * N, scale=C ** -0.5), A=-torch.arange(1, N + 1) * torch.exp(normal(8, C, N, scale=0.2)),
                D=normal(9, C, scale=0.1, mean=1.0), w_out=normal(10, C, C, scale=C ** -0.5))


def _scan_block(x, residual, p, conv_state, h, op):
    """One block on [B, T, C] by the given operators; returns (out, stream, conv state, h)."""
    y, s = op.norm(x, p["gamma"], residual)
    u, z = (y @ p["w_in"]).split(C, dim=-1)
    u, conv_state = op.conv(u.contiguous(), p["conv"], p["bias"], conv_state)
    bc = (u @ p["w_bc"]).unsqueeze(-2)
    y, h = op.scan(u, u @ p["w_d"], p["A"], bc[..., :N].contiguous(), bc[..., N:].contiguous(), p["D"], z.contiguous(),
                   p["delta_bias"], h)
    return y @ p["w_out"], s, conv_state, h


class Own:
    norm = staticmethod(lambda x, g, r: xa.rmsnorm(x, g, r))
    conv = staticmethod(lambda u, w, b, st: xa.causal_conv(u, w, b, "silu", st))
    scan = staticmethod(lambda *a: xa.ssm_scan(*a))


class Reference:
    """The same operators in 64 bits by torch's differentiable elementary operations."""

    @staticmethod
    def norm(x, g, r):
        s = x + r
        return s * torch.rsqrt(s.square().mean(-1, keepdim=True) + 1e-5) * g, s

    @staticmethod
    def conv(u, w, b, st):
        x = torch.cat([st, u], 1)
        y = sum(w[:, k] * x[:, k:k + u.shape[1]] for k in range(K)) + b
        return torch.nn.functional.silu(y), x[:, u.shape[1]:]

    @staticmethod
    def scan(u, delta, A, Bm, Cm, D, z, bias, h):
        d, ys = torch.nn.functional.softplus(delta + bias), []
        for t in range(u.shape[1]):
            h = torch.exp(d[:, t, :, None] * A) * h + (d[:, t] * u[:, t])[..., None] * Bm[:, t]
            ys.append((h * Cm[:, t]).sum(-1) + D * u[:, t])
        return torch.stack(ys, 1) * torch.nn.functional.silu(z), h


def _start():
    return normal(20, B, S, C), normal(21, B, S, C), normal(22, B, K - 1, C), normal(23, B, C, N)


def test_gradients_through_a_block():
    p, (x, r, st, h) = _weights(), _start()
    leaves = {**p, "x": x, "r": r, "st": st, "h": h}
    results = []
    for op, put in ((Own, lambda t: t.cuda()), (Reference, lambda t: t.double())):
        q = {k: put(v).requires_grad_() for k, v in leaves.items()}
        out, s, st1, h1 = _scan_block(q["x"], q["r"], q, q["st"], q["h"], op)
        out2, s2, _, _ = _scan_block(out, s, q, st1, h1, op)              # a second one on the stream and the states
        loss = (out2 * put(normal(30, B, S, C))).sum() + (s2 * put(normal(31, B, S, C))).sum()
        loss.backward()
        results.append((out2.detach().cpu(), {k: v.grad.cpu() for k, v in q.items()}))
    (y, g), (yr, gr) = results
    assert float((y - yr).abs().max()) <= 1e-4 * float(yr.abs().max())
    for k in leaves:
        assert float((g[k] - gr[k]).abs().max()) <= 2e-4 * float(gr[k].abs().max()), k


def _scan_tokens(p, x, r, st, h, step):
    """The block token by token from the carried states, through the single-token calls."""
    outs = []
    for t in range(x.shape[1]):
        outs.append(step(p, x[:, t].contiguous(), r[:, t].contiguous(), st, h))
    return torch.stack(outs, 1)


def _token(p, x, r, st, h):
    y, s, _ = xb.rmsnorm(x, p["gamma"], r)
    u, z = (y @ p["w_in"]).split(C, dim=-1)
    u = xb.causal_conv_step(u.contiguous(), p["conv"], st, p["bias"])
    bc = (u @ p["w_bc"]).unsqueeze(-2)
    y = xb.ssm_scan_step(u, u @ p["w_d"], p["A"], bc[..., :N].contiguous(), bc[..., N:].contiguous(), h, D=p["D"], z=z.contiguous(),
                         delta_bias=p["delta_bias"])
    return y @ p["w_out"]


def test_prompt_then_tokens_is_the_whole_prompt():
    p = {k: v.cuda() for k, v in _weights().items()}
    x, r, st, h = (t.cuda() for t in _start())
    whole, _, st_end, h_end = _scan_block(x, r, p, st, h, Own)
    cut = 21
    first, _, st1, h1 = _scan_block(x[:, :cut].contiguous(), r[:, :cut].contiguous(), p, st, h, Own)
    rest = _scan_tokens(p, x[:, cut:], r[:, cut:], st1, h1, _token)
    scale = float(whole.abs().max())
    assert float((torch.cat([first, rest], 1) - whole).abs().max()) <= 1e-4 * scale
    assert float((st1 - st_end).abs().max()) <= 1e-4 * float(st_end.abs().max())
    assert float((h1 - h_end).abs().max()) <= 1e-4 * float(h_end.abs().max())


def test_a_captured_decode_step_replays():
    p = {k: v.cuda() for k, v in _weights().items()}
    x, r, st, h = (t.cuda() for t in _start())
    want = _scan_tokens(p, x[:, :8], r[:, :8], st.clone(), h.clone(), _token)
    xt, rt, stt, ht = x[:, 0].contiguous(), r[:, 0].contiguous(), st.clone(), h.clone()
    _token(p, xt, rt, stt, ht)                                             # warm: library handles, allocations
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = _token(p, xt, rt, stt, ht)
    stt.copy_(st)
    ht.copy_(h)
    for t in range(8):
        xt.copy_(x[:, t])
        rt.copy_(r[:, t])
        graph.replay()
        assert torch.equal(y, want[:, t])


def test_a_captured_training_step_replays():
    """Forward and backward in one graph, on leaves that no eager autograd graph holds while it is captured."""
    p, (x, r, st, h) = _weights(), _start()
    w = normal(30, B, S, C).cuda()

    def step(q):
        out, s, _, h1 = _scan_block(q["x"], q["r"], q, q["st"], q["h"], Own)
        ((out * w).sum() + s.sum() + h1.sum()).backward()

    def leaves(x0):
        return {k: v.clone().cuda().requires_grad_() for k, v in dict(p, x=x0, r=r, st=st, h=h).items()}

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(leaves(x))                                                    # warm: library handles, allocations
    torch.cuda.current_stream().wait_stream(side)
    held, other = leaves(x), normal(40, B, S, C)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(held)
    for x0 in (other, x):
        with torch.no_grad():
            held["x"].copy_(x0)
        graph.replay()
        want = leaves(x0)
        step(want)
        for k in held:
            assert float((held[k].grad - want[k].grad).abs().max()) <= 1e-4 * float(want[k].grad.abs().max()), k


def test_norm_and_convolution_around_the_mlstm_cell():
    """norm -> convolution -> mLSTM cell -> epilogue with the convolution's output as the skip."""
    NH, DH = 4, 16
    x, r, gamma = normal(1, B, S, C), normal(2, B, S, C), normal(3, C, scale=0.1, mean=1.0)
    w, bias = normal(4, C, K, scale=0.5), normal(5, C, scale=0.1)
    gates = dict(i_pre=normal(6, B, NH, S), f_pre=normal(7, B, NH, S, mean=3.0))
    z, gg, gb, sw = normal(8, B, S, C), normal(9, C, scale=0.1, mean=1.0), normal(10, C, scale=0.1), normal(11, C, scale=0.5)
    inf = torch.full((B, NH, S, DH), float("inf"))

    def heads(t):
        return t.reshape(B, S, NH, DH).transpose(1, 2).contiguous()

    y, s, _ = xb.rmsnorm(x.cuda(), gamma.cuda(), r.cuda())
    u, _ = xb.causal_conv_fwd(y, w.cuda(), bias.cuda())
    h, _, _, _ = xb.mlstm_fwd(heads(u), heads(u), heads(y), gates["i_pre"].cuda(), gates["f_pre"].cuda(), inf.cuda(), chunk=16)
    out = xb.mlstm_headnorm_gate(h, gg.cuda(), gb.cuda(), z.cuda(), sw.cuda(), u)

    yr, sr, _ = ob.rmsnorm(x, gamma, r)
    ur, _ = ob.causal_conv(yr, w, bias)
    hd = lambda t: np.ascontiguousarray(t.reshape(B, S, NH, DH).transpose(0, 2, 1, 3))
    hr, _, _, _ = oracle.fwd(hd(ur), hd(ur), hd(yr), gates["i_pre"].numpy(), gates["f_pre"].numpy(), inf.numpy(), "sigmoid")
    ref = oracle_headnorm(hr, gg, gb, z, sw, ur, eps=1e-5)
    assert np.abs(out.cpu().numpy() - ref).max() <= 1e-4 * max(1.0, np.abs(ref).max())
    assert np.abs(s.cpu().numpy() - sr).max() <= 1e-6 * np.abs(sr).max()


def test_padded_batch_serves_like_rows_alone():
    """Convolution and scan of a padded batch of prompts give what each prompt gives alone."""
    n = [5, 0, 37, 1]
    w, A = normal(1, C, K).cuda(), -torch.exp(normal(2, C, N)).cuda()
    x, delta, bc = normal(3, 4, S, C).cuda(), normal(4, 4, S, C, mean=-2.0).cuda(), normal(5, 4, S, 2, 1, N).cuda()
    lengths = torch.tensor(n, dtype=torch.int32).cuda()
    u, st = xb.causal_conv_fwd(x, w, lengths=lengths, y=torch.zeros_like(x))
    y, h = xb.ssm_scan_fwd(u, delta, A, bc[:, :, 0].contiguous(), bc[:, :, 1].contiguous(), lengths=lengths, y=torch.zeros_like(x))
    for b, m in enumerate(n):
        u1, st1 = xb.causal_conv_fwd(x[b:b + 1, :m].contiguous(), w)
        y1, h1 = xb.ssm_scan_fwd(u1, delta[b:b + 1, :m].contiguous(), A, bc[b:b + 1, :m, 0].contiguous(), bc[b:b + 1, :m, 1].contiguous())
        assert torch.equal(u[b:b + 1, :m], u1) and torch.equal(st[b:b + 1], st1)
        for got, ref in ((y[b:b + 1, :m], y1), (h[b:b + 1], h1)):
            assert float((got - ref).abs().max() if got.numel() else 0.0) <= 1e-4 * max(1.0, float(ref.abs().max() if ref.numel() else 0.0))
