"""GPU parity of the selective scan over long walks of one CTA, against the float64
oracle: the pipeline's steady state (more than 4 tiles of 32 tokens in flight) and the
reuse of its ring (more than 8), in one pass and in segments, at every number of lanes
a channel; the backward's two channel groups a warp for up to 8 states; two streams.

Tolerances: those of ``test_scan_parity`` and ``test_scan_bwd_parity``.  A segment of n
tokens (at most 450 here) is decayed by one exponential of a sum of d, formed by 32 and
then by tile: its exponent e is off by at most (32 + 15 + 3) EPS |e|, where the bound has
35 EPS |e| + 6 n EPS, which is more for |e| < 180 (and past that nothing is left)."""
import numpy as np
import pytest
import torch

import oracle.ssm as oscan
from blockparity import BF16, F32, cuda, normal, within
from linear_rnn_mlstm_b200 import binding as xb
from test_scan_bwd_parity import check as check_backward
from test_scan_parity import bounds, check_forward, inputs

pytestmark = pytest.mark.gpu

SMS = 148


def ctas(B, C, N, G):
    """CTAs of one segment: 4 to 32 lanes a channel (two states each), 32 to 8 channels."""
    cb = 32 if N <= 8 else 16 if N <= 32 else 8
    return B * G * -(-(C // G) // cb)


def needs_one_pass(B, S, C, N, G):
    assert 2 * ctas(B, C, N, G) >= SMS
    assert xb.xlstm_ssm_scan_fwd_workspace_size(B, S, C, N, G, xb.BF16) == (xb.OK, 0)


@pytest.mark.parametrize("dtype", (F32, BF16), ids=("f32", "bf16"))
@pytest.mark.parametrize("B,C,N,G", [(4, 600, 5, 1), (4, 608, 8, 1), (2, 592, 13, 1), (2, 592, 16, 1), (2, 600, 16, 3), (2, 592, 30, 1),
                                     (2, 592, 32, 2), (2, 296, 50, 1), (2, 296, 64, 1)])
def test_one_pass_over_many_tiles(B, C, N, G, dtype):
    for S in (333, 288):                                          # 11 tiles, the last short; 9 whole ones
        needs_one_pass(B, S, C, N, G)
        check_forward(inputs(B, S, C, N, G, dtype=dtype, seed=N))


@pytest.mark.parametrize("dtype", (F32, BF16), ids=("f32", "bf16"))
@pytest.mark.parametrize("N,full", [(8, False), (13, True), (16, False), (64, True)])
def test_one_pass_over_many_tiles_of_a_padded_batch(N, full, dtype):
    B, S, C = 4, 333, 600
    needs_one_pass(B, S, C, N, 1)
    n = [333, 0, 130, 257]
    i = inputs(B, S, C, N, dtype=dtype, seed=N, full=full)
    y = torch.full((B, S, C), 5.0, dtype=dtype, device="cuda")
    got, h = xb.ssm_scan_fwd(**cuda(i), lengths=torch.tensor(n, dtype=torch.int32).cuda(), y=y)
    yr, hr = oscan.scan(**i, lengths=n)
    ey, eh = bounds(i, lengths=n)
    within(h, hr, eh, "h")
    for b, m in enumerate(n):
        assert torch.all(got[b, m:] == 5.0)
        if m:
            within(got[b, :m], yr[b, :m], ey[b, :m] + 4e-6 * np.abs(yr[b, :m]), "y")


@pytest.mark.parametrize("dtype", (F32, BF16), ids=("f32", "bf16"))
@pytest.mark.parametrize("N", (5, 8, 13, 16, 17, 32, 50, 64))
def test_short_segments(N, dtype):
    check_forward(inputs(1, 700, 16, N, dtype=dtype, seed=N))     # 11 segments of two tiles


@pytest.mark.parametrize("dtype", (F32, BF16), ids=("f32", "bf16"))
@pytest.mark.parametrize("C,N,G", [(1920, 5, 1), (1920, 8, 2), (960, 13, 1), (960, 16, 1), (960, 30, 1), (480, 50, 1), (480, 64, 1)])
def test_segments_of_many_tiles(C, N, G, dtype):
    assert ctas(1, C, N, G) == 60                                 # 4 segments of 14 tiles
    check_forward(inputs(1, 1700, C, N, G, dtype=dtype, seed=N, step=2e-3))


# bf16, more than one CTA of two groups per SM: B * G * (blocks of 128 channels) * (segments of 64 tokens) > 148
@pytest.mark.parametrize("dtype", (F32, BF16), ids=("f32", "bf16"))
@pytest.mark.parametrize("B,S,C,N,G", [(3, 200, 2048, 8, 1), (3, 200, 2064, 5, 2), (4, 200, 2048, 4, 1), (3, 193, 2056, 1, 1)])
def test_backward_of_two_groups_a_warp_for_few_states(B, S, C, N, G, dtype):
    assert B * G * -(-(C // G) // 128) * -(-S // 64) > SMS
    check_backward(inputs(B, S, C, N, G, dtype=dtype, seed=S + N))


def test_two_backward_calls_at_once_on_two_streams():
    for shape in ((1, 600, 16, 16), (3, 130, 2048, 8)):
        calls = [cuda({**inputs(*shape, dtype=BF16, seed=k), "dy": normal(k + 60, *shape[:3], dtype=BF16)}) for k in (1, 30)]
        want = [xb.ssm_scan_bwd(**c) for c in calls]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        for _ in range(5):
            got = []
            for s, c in zip(streams, calls):
                with torch.cuda.stream(s):
                    got.append(xb.ssm_scan_bwd(**c))
            torch.cuda.synchronize()
            for g, w in zip(got, want):
                assert all(torch.equal(g[nm], w[nm]) for nm in w)


def test_two_backward_calls_of_norm_and_convolution_at_once():
    def operands(k):
        s, dy = normal(k, 4, 300, 512, dtype=BF16).cuda(), normal(k + 1, 4, 300, 512, dtype=BF16).cuda()
        g, w = normal(k + 2, 512, mean=1.0).cuda(), normal(k + 3, 512, 4).cuda()
        return s, dy, g, w, xb.rmsnorm(s, g)[2]

    def both(s, dy, g, w, rstd):
        c = xb.causal_conv_bwd(s, w, dy)
        return (*xb.rmsnorm_bwd(dy, s, g, rstd), c["dx"], c["dw"])

    calls = [operands(1), operands(40)]
    want = [both(*c) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for s, c in zip(streams, calls):
            with torch.cuda.stream(s):
                got.append(both(*c))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))
