"""GPU parity of the selective scan's forward and step (``xlstm_ssm_scan_*``)
against the float64 oracle (``oracle.ssm``).

Tolerance: a bound on the fp32 recurrence's error, carried along with it in 64
bits.  With EPS = 2^-24, the step size d is within 32 EPS of its value (the
softplus: its exponential 4 + 2|v| EPS for |v| < 10, division and series 6), an
exponential within ULP = 4 EPS (2^-22, the hardware's stated error) plus the
error of its exponent, |d A| (32 + 3) EPS; each product and sum adds EPS.  For
the magnitudes M_t = a M_{t-1} + |d x B| the error obeys
  E_t = a (E_{t-1} + (4 + 35 |d A| + 2) EPS M_{t-1}) + 36 EPS |d x B|.
y adds N products and sums in any order, (E + (N + 2) EPS M) |C|, the skip's two
roundings, and the gate's 4e-6 relative.  Where the tokens are cut into segments
the decay over a whole segment is one exponential of a sum of d: its error is
smaller than the per-token errors the bound adds up over that segment."""
import numpy as np
import pytest
import torch

import oracle.ssm as oscan
from oracle.block import f64, sigmoid
from blockparity import BF16, EPS32, F32, cuda, normal, within
from linear_rnn_mlstm_b200 import binding as xb

pytestmark = pytest.mark.gpu


def inputs(B, S, C, N, G=1, dtype=F32, seed=0, full=True, step=None):
    """Step sizes around ``step`` (default log-spread over 1e-3..0.3), decay rates around 1..N."""
    shape = (B, C) if S is None else (B, S, C)
    g = torch.Generator().manual_seed(seed)
    d0 = torch.exp(torch.rand(C, generator=g) * np.log(300.0) + np.log(1e-3)) if step is None else torch.full((C,), step)
    i = dict(x=normal(seed + 1, *shape, dtype=dtype), delta=normal(seed + 2, *shape, dtype=dtype, scale=0.5),
             A=-torch.arange(1, N + 1) * torch.exp(normal(seed + 3, C, N, scale=0.2)),
             Bm=normal(seed + 4, *shape[:-1], G, N, dtype=dtype), Cm=normal(seed + 5, *shape[:-1], G, N, dtype=dtype),
             D=None, z=None, delta_bias=torch.log(torch.expm1(d0)))
    if full:
        i.update(D=normal(seed + 6, C), z=normal(seed + 7, *shape, dtype=dtype), h0=normal(seed + 8, B, C, N))
    return i


def bounds(i, softplus=True, lengths=None):
    """(bound on y, bound on h) for inputs with a token axis."""
    x, A, Bm, Cm = f64(i["x"]), f64(i["A"]), np.abs(f64(i["Bm"])), np.abs(f64(i["Cm"]))
    B, S, C = x.shape
    N = A.shape[1]
    d, _ = oscan._steps(i["delta"], i["delta_bias"], softplus)
    h0 = i.get("h0")
    M = np.zeros((B, C, N)) if h0 is None else np.abs(f64(h0))
    E, ey = np.zeros_like(M), np.zeros_like(x)
    n = np.full(B, S) if lengths is None else np.clip(f64(lengths), 0, S)
    for t in range(S):
        ad = np.abs(d[:, t, :, None] * A)
        a, ub = np.exp(d[:, t, :, None] * A), np.abs(d[:, t] * x[:, t])[..., None] * oscan._rows(Bm, t, C)
        live = (t < n)[:, None, None]
        E = np.where(live, a * (E + (6 + 35 * ad) * EPS32 * M) + 36 * EPS32 * ub, E)
        M = np.where(live, a * M + ub, M)
        ey[:, t] = ((E + (N + 2) * EPS32 * M) * oscan._rows(Cm, t, C)).sum(2)
        if i["D"] is not None:
            ey[:, t] += 2 * EPS32 * np.abs(f64(i["D"]) * x[:, t])
        if i["z"] is not None:
            z = f64(i["z"])[:, t]
            ey[:, t] *= 1.01 * np.abs(z * sigmoid(z))
    return ey, E


def check_forward(i, softplus=True):
    d = cuda(i)
    y, h = xb.ssm_scan_fwd(**d, softplus=softplus)
    yr, hr = oscan.scan(**i, softplus=softplus)
    ey, eh = bounds(i, softplus)
    within(y, yr, ey + 4e-6 * np.abs(yr), "y")
    within(h, hr, eh, "h")


@pytest.mark.parametrize("dtype", (F32, BF16), ids=("f32", "bf16"))
@pytest.mark.parametrize("N", (1, 2, 4, 5, 8, 13, 16, 17, 32, 33, 64))
def test_forward_over_state_sizes(N, dtype):
    check_forward(inputs(2, 70, 24, N, dtype=dtype, seed=N))


@pytest.mark.parametrize("dtype", (F32, BF16), ids=("f32", "bf16"))
@pytest.mark.parametrize("B,S,C,N,G", [(1, 1, 8, 16, 1), (3, 2, 40, 16, 1), (1, 31, 16, 8, 2), (2, 32, 8, 16, 1), (2, 33, 264, 16, 1),
                                       (1, 65, 48, 16, 2), (1, 700, 24, 16, 1), (2, 257, 80, 4, 5), (1, 2050, 8, 16, 1), (4, 97, 2048, 16, 1)])
def test_forward_over_shapes(B, S, C, N, G, dtype):
    check_forward(inputs(B, S, C, N, G, dtype=dtype, seed=S))


@pytest.mark.parametrize("full", (False, True))
def test_forward_with_and_without_each_option(full):
    check_forward(inputs(2, 40, 16, 16, full=full))
    i = inputs(2, 300, 16, 16, full=full)                         # several segments
    check_forward(i)
    i["delta"], i["delta_bias"] = torch.rand_like(i["delta"]) * 0.2, None
    check_forward(i, softplus=False)


def test_a_long_memory():
    check_forward(inputs(1, 4096, 32, 16, step=1e-3, seed=2))     # one pass holds hundreds of tokens in mind


def test_the_state_only_or_the_output_only():
    d = cuda(inputs(1, 90, 16, 16))
    y, h = xb.ssm_scan_fwd(**d)
    y2, none = xb.ssm_scan_fwd(**d, state_out=False)
    assert none is None and torch.equal(y, y2)


@pytest.mark.parametrize("dtype", (F32, BF16), ids=("f32", "bf16"))
@pytest.mark.parametrize("S,C", [(70, 24), (400, 16), (65, 4096)])
def test_lengths_leave_what_stands_behind_them(S, C, dtype):
    n = [0, 1, 33, S, S + 9, -3]
    held = [min(max(v, 0), S) for v in n]
    i = inputs(6, S, C, 16, dtype=dtype)
    dirty = {k: v.clone() if v is not None else None for k, v in i.items()}
    for b, m in enumerate(held):
        for nm in ("x", "delta", "Bm", "Cm", "z"):
            dirty[nm][b, m:] = float("nan")                       # not to be read into anything
    y = torch.full((6, S, C), 5.0, dtype=dtype, device="cuda")
    got, h = xb.ssm_scan_fwd(**cuda(dirty), lengths=torch.tensor(n, dtype=torch.int32).cuda(), y=y)
    yr, hr = oscan.scan(**i, lengths=held)
    ey, eh = bounds(i, lengths=held)
    within(h, hr, eh, "h")
    for b, m in enumerate(held):
        assert torch.all(got[b, m:] == 5.0)
        if m:
            within(got[b, :m], yr[b, :m], ey[b, :m] + 4e-6 * np.abs(yr[b, :m]), "y")


def test_an_empty_prompt_hands_the_state_on():
    d = cuda(inputs(2, 0, 16, 16))
    y, h = xb.ssm_scan_fwd(**d)
    assert y.shape == (2, 0, 16) and torch.equal(h, d["h0"])


@pytest.mark.parametrize("dtype", (F32, BF16), ids=("f32", "bf16"))
@pytest.mark.parametrize("B,C,N,G", [(1, 8, 16, 1), (3, 40, 1, 1), (2, 24, 4, 3), (5, 16, 5, 2), (2, 8, 8, 1), (3, 16, 13, 1), (2, 264, 16, 1),
                                     (2, 8, 30, 1), (1, 24, 32, 1), (2, 16, 50, 2), (3, 8, 64, 1), (33, 2056, 16, 1), (40, 1024, 8, 2)])
@pytest.mark.parametrize("full", (False, True))
def test_step(B, C, N, G, full, dtype):
    i = inputs(B, None, C, N, G, dtype=dtype, full=full)
    h0 = i.pop("h0", torch.zeros(B, C, N))
    d = cuda(i)
    h = h0.cuda()
    y = xb.ssm_scan_step(h=h, **d)
    one = {k: v[:, None] if k in ("x", "delta", "Bm", "Cm", "z") and v is not None else v for k, v in i.items()}
    yr, hr = oscan.scan(**one, h0=h0)
    ey, eh = bounds({**one, "h0": h0})
    within(h, hr, eh, "h")
    within(y, yr[:, 0], (ey + 4e-6 * np.abs(yr))[:, 0], "y")


def test_steps_continue_a_prompt():
    B, S, C, N = 2, 37, 48, 16
    i = inputs(B, S, C, N, G=2, dtype=F32)
    d = cuda(i)
    yr, hr = oscan.scan(**i)
    ey, eh = bounds(i)
    part = {k: v[:, :30].contiguous() if k in ("x", "delta", "Bm", "Cm", "z") else v for k, v in d.items()}
    _, h = xb.ssm_scan_fwd(**part)
    d.pop("h0")
    for t in range(30, S):
        y = xb.ssm_scan_step(h=h, **{k: v[:, t].contiguous() if k in ("x", "delta", "Bm", "Cm", "z") else v for k, v in d.items()})
        within(y, yr[:, t], ey[:, t] + 4e-6 * np.abs(yr[:, t]), "y")
    within(h, hr, eh, "h")


def test_far_step_sizes():
    # softplus at both ends: e^v where v is far below zero, v itself far above
    v = torch.tensor([-80.0, -30.0, -10.0, -1.0, 0.0, 1.0, 30.0, 1000.0])
    i = dict(x=torch.ones(1, 1, 8), delta=v.view(1, 1, 8), A=torch.full((8, 1), -1e-3), Bm=torch.ones(1, 1, 1, 1), Cm=torch.ones(1, 1, 1, 1))
    y, _ = xb.ssm_scan_fwd(**cuda(i))
    ref = oscan.scan(**i)[0]
    within(y, ref, (10 + 3 * v.abs().numpy()) * EPS32 * np.abs(ref), "softplus")


def test_a_captured_call_replays_on_new_inputs():
    for B, C in ((1, 16), (2, 2048)):                             # with segments, and in one pass
        a, b = cuda(inputs(B, 200, C, 16, dtype=BF16, seed=1)), cuda(inputs(B, 200, C, 16, dtype=BF16, seed=50))
        held = {k: v.clone() for k, v in a.items()}
        xb.ssm_scan_fwd(**held)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y, h = xb.ssm_scan_fwd(**held)
        for src in (b, a):
            for k in held:
                held[k].copy_(src[k])
            graph.replay()
            yr, hr = xb.ssm_scan_fwd(**src)
            assert torch.equal(y, yr) and torch.equal(h, hr)


def test_two_calls_at_once_on_two_streams():
    a, b = cuda(inputs(1, 600, 16, 16, dtype=BF16, seed=1)), cuda(inputs(1, 600, 16, 16, dtype=BF16, seed=50))
    want = [xb.ssm_scan_fwd(**v) for v in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for s, v in zip(streams, (a, b)):
            with torch.cuda.stream(s):
                got.append(xb.ssm_scan_fwd(**v))
        torch.cuda.synchronize()
        for (y, h), (yr, hr) in zip(got, want):
            assert torch.equal(y, yr) and torch.equal(h, hr)
