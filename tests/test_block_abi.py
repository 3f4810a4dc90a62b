"""Host-side refusals of the block operators (norm, convolution, scan): bad arguments
are rejected before any device work, so fake device addresses are never used.
And the binding's own checks, on the CPU."""
import pytest
import torch

from linear_rnn_mlstm_b200 import binding as xb

FAKE = 1 << 40


def _call(fn, base, over):
    """``base`` names every argument; pointers are distinct aligned fakes."""
    args = {k: (FAKE + 4096 * i if v == "p" else v) for i, (k, v) in enumerate(base.items())}
    for k, v in over.items():
        args[k] = args[v[1:]] if isinstance(v, str) and v.startswith("=") else v
    return fn(*args.values())


NORM = dict(x="p", residual="p", gamma="p", s="p", y="p", q="p", scales="p", rstd="p", rows=4, C=256, group=128, eps=1e-5,
            dt=xb.BF16, stream=None)


@pytest.mark.parametrize("over,expect", [
    (dict(x=None), xb.ERR_NULL),
    (dict(gamma=None), xb.ERR_NULL),
    (dict(y=None, q=None, scales=None), xb.ERR_NULL),
    (dict(q=None), xb.ERR_NULL),                         # scales without codes
    (dict(scales=None), xb.ERR_NULL),
    (dict(residual=None), xb.ERR_UNSUPPORTED),           # a stream output without a residual
    (dict(group=48), xb.ERR_UNSUPPORTED),
    (dict(group=-1), xb.ERR_UNSUPPORTED),
    (dict(C=264), xb.ERR_UNSUPPORTED),                   # not whole groups
    (dict(C=4), xb.ERR_SHAPE),
    (dict(C=260), xb.ERR_SHAPE),
    (dict(C=8200), xb.ERR_SHAPE),
    (dict(rows=-1), xb.ERR_SHAPE),
    (dict(dt=2), xb.ERR_DTYPE),
    (dict(eps=0.0), xb.ERR_UNSUPPORTED),
    (dict(eps=float("nan")), xb.ERR_UNSUPPORTED),
    (dict(eps=float("inf")), xb.ERR_UNSUPPORTED),
    (dict(x=FAKE + 8), xb.ERR_ALIGN),
    (dict(scales=FAKE + 4), xb.ERR_ALIGN),
    (dict(s="=x"), xb.ERR_UNSUPPORTED),
    (dict(y="=residual"), xb.ERR_UNSUPPORTED),
    (dict(y="=s"), xb.ERR_UNSUPPORTED),
    (dict(q="=y"), xb.ERR_UNSUPPORTED),
    (dict(rstd="=scales"), xb.ERR_UNSUPPORTED),
    (dict(rstd="=gamma"), xb.ERR_UNSUPPORTED),
    (dict(rows=0), xb.OK),
    (dict(rows=0, x=None), xb.OK),
])
def test_rmsnorm_fwd_refusals(over, expect):
    assert _call(xb.xlstm_rmsnorm_fwd, NORM, over) == expect


NORM_BWD = dict(dy="p", ds="p", s="p", gamma="p", rstd="p", dx="p", dgamma="p", rows=4, C=256, dt=xb.BF16, workspace="p",
                workspace_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("over,expect", [
    (dict(dy=None), xb.ERR_NULL),
    (dict(s=None), xb.ERR_NULL),
    (dict(rstd=None), xb.ERR_NULL),
    (dict(dgamma=None), xb.ERR_NULL),
    (dict(dx="=dy"), xb.ERR_UNSUPPORTED),
    (dict(dx="=ds"), xb.ERR_UNSUPPORTED),
    (dict(dgamma="=gamma"), xb.ERR_UNSUPPORTED),
    (dict(dx="=dgamma"), xb.ERR_UNSUPPORTED),
    (dict(workspace=None), xb.ERR_WORKSPACE),
    (dict(workspace_bytes=64), xb.ERR_WORKSPACE),
    (dict(workspace=FAKE + 4), xb.ERR_ALIGN),
    (dict(C=12), xb.ERR_SHAPE),
    (dict(dt=-1), xb.ERR_DTYPE),
])
def test_rmsnorm_bwd_refusals(over, expect):
    assert _call(xb.xlstm_rmsnorm_bwd, NORM_BWD, over) == expect


CONV = dict(x="p", w="p", bias="p", state0="p", lengths="p", y="p", state_out="p", B=2, S=8, C=64, K=4, dt=xb.BF16,
            act=xb.CONV_SILU, stream=None)


@pytest.mark.parametrize("over,expect", [
    (dict(x=None), xb.ERR_NULL),
    (dict(w=None), xb.ERR_NULL),
    (dict(y=None), xb.ERR_NULL),
    (dict(K=1), xb.ERR_SHAPE),
    (dict(K=5), xb.ERR_SHAPE),
    (dict(C=20), xb.ERR_SHAPE),
    (dict(C=65544), xb.ERR_SHAPE),
    (dict(S=-1), xb.ERR_SHAPE),
    (dict(B=-1), xb.ERR_SHAPE),
    (dict(S=1 << 30, B=1 << 20), xb.ERR_SHAPE),
    (dict(dt=5), xb.ERR_DTYPE),
    (dict(act=2), xb.ERR_DTYPE),
    (dict(bias=FAKE + 4), xb.ERR_ALIGN),
    (dict(y="=x"), xb.ERR_UNSUPPORTED),
    (dict(state_out="=state0"), xb.ERR_UNSUPPORTED),
    (dict(state_out="=y"), xb.ERR_UNSUPPORTED),
    (dict(y="=lengths"), xb.ERR_UNSUPPORTED),
    (dict(B=0, x=None), xb.OK),
])
def test_conv_fwd_refusals(over, expect):
    assert _call(xb.xlstm_causal_conv_fwd, CONV, over) == expect


STEP = dict(x="p", w="p", bias="p", state="p", y="p", B=2, C=64, K=4, dt=xb.BF16, act=xb.CONV_SILU, stream=None)


@pytest.mark.parametrize("over,expect", [
    (dict(state=None), xb.ERR_NULL),
    (dict(y=None), xb.ERR_NULL),
    (dict(state="=x"), xb.ERR_UNSUPPORTED),
    (dict(y="=x"), xb.ERR_UNSUPPORTED),
    (dict(y="=state"), xb.ERR_UNSUPPORTED),
    (dict(state=FAKE + 2), xb.ERR_ALIGN),
    (dict(K=6), xb.ERR_SHAPE),
    (dict(B=0), xb.OK),
])
def test_conv_step_refusals(over, expect):
    assert _call(xb.xlstm_causal_conv_step, STEP, over) == expect


CONV_BWD = dict(x="p", w="p", bias="p", state0="p", dy="p", dstate="p", dx="p", dw="p", dbias="p", dstate0="p", B=2, S=8, C=64,
                K=4, dt=xb.BF16, act=xb.CONV_SILU, workspace="p", workspace_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("over,expect", [
    (dict(dy=None), xb.ERR_NULL),
    (dict(dx=None), xb.ERR_NULL),
    (dict(dw=None), xb.ERR_NULL),
    (dict(dx="=dy"), xb.ERR_UNSUPPORTED),
    (dict(dw="=w"), xb.ERR_UNSUPPORTED),
    (dict(dstate0="=dstate"), xb.ERR_UNSUPPORTED),
    (dict(dstate0="=dx"), xb.ERR_UNSUPPORTED),
    (dict(workspace_bytes=128), xb.ERR_WORKSPACE),
    (dict(workspace=None), xb.ERR_WORKSPACE),
    (dict(act=-1), xb.ERR_DTYPE),
])
def test_conv_bwd_refusals(over, expect):
    assert _call(xb.xlstm_causal_conv_bwd, CONV_BWD, over) == expect


def test_workspace_sizes():
    assert xb.xlstm_rmsnorm_bwd_workspace_size(0, 64, xb.F32) == (xb.OK, 0)
    st, n = xb.xlstm_rmsnorm_bwd_workspace_size(1 << 20, 2048, xb.BF16)
    assert st == xb.OK and 0 < n < 1 << 25               # bounded: a share per resident CTA
    assert xb.xlstm_rmsnorm_bwd_workspace_size(4, 10, xb.F32)[0] == xb.ERR_SHAPE
    st, n = xb.xlstm_causal_conv_bwd_workspace_size(2, 100, 64, 4, xb.F32)
    assert st == xb.OK and n >= 2 * 64 * 5 * 4
    assert xb.xlstm_causal_conv_bwd_workspace_size(2, 100, 64, 9, xb.F32)[0] == xb.ERR_SHAPE


def test_the_binding_refuses_host_tensors_and_bad_options():
    x, g = torch.zeros(2, 64), torch.ones(64)
    w = torch.zeros(64, 4)
    for call in (lambda: xb.rmsnorm(x, g), lambda: xb.rmsnorm_fp8(x, g, group=32), lambda: xb.rmsnorm_bwd(x, x, g, torch.ones(2)),
                 lambda: xb.causal_conv_fwd(x[None], w), lambda: xb.causal_conv_step(x, w, torch.zeros(2, 3, 64)),
                 lambda: xb.causal_conv_bwd(x[None], w, x[None])):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
    with pytest.raises(ValueError, match="group"):
        xb.rmsnorm_fp8(x, g, group=48)
    with pytest.raises(ValueError, match="act"):
        xb.causal_conv_fwd(x[None], w, act="relu")
    with pytest.raises(ValueError, match="K 2, 3 or 4"):
        xb.causal_conv_fwd(x[None], torch.zeros(64, 5))
    with pytest.raises(TypeError):
        xb.rmsnorm(x.half(), g)


SCAN = dict(x="p", delta="p", A="p", Bm="p", Cm="p", D="p", z="p", delta_bias="p", h0="p", lengths="p", y="p", h_out="p", B=2, S=8,
            C=64, N=16, G=2, dt=xb.BF16, act=xb.DELTA_SOFTPLUS, workspace="p", workspace_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("over,expect", [
    (dict(x=None), xb.ERR_NULL),
    (dict(delta=None), xb.ERR_NULL),
    (dict(A=None), xb.ERR_NULL),
    (dict(Bm=None), xb.ERR_NULL),
    (dict(Cm=None), xb.ERR_NULL),
    (dict(y=None), xb.ERR_NULL),
    (dict(N=0), xb.ERR_SHAPE),
    (dict(N=65), xb.ERR_SHAPE),
    (dict(C=60), xb.ERR_SHAPE),
    (dict(G=3), xb.ERR_SHAPE),
    (dict(G=16), xb.ERR_SHAPE),                          # groups of four channels
    (dict(G=0), xb.ERR_SHAPE),
    (dict(B=65536), xb.ERR_SHAPE),
    (dict(S=-1), xb.ERR_SHAPE),
    (dict(S=1 << 30, B=60000), xb.ERR_SHAPE),
    (dict(dt=3), xb.ERR_DTYPE),
    (dict(act=2), xb.ERR_DTYPE),
    (dict(z=FAKE + 8), xb.ERR_ALIGN),
    (dict(y="=x"), xb.ERR_UNSUPPORTED),
    (dict(y="=z"), xb.ERR_UNSUPPORTED),
    (dict(h_out="=h0"), xb.ERR_UNSUPPORTED),
    (dict(h_out="=y"), xb.ERR_UNSUPPORTED),
    (dict(S=4096, workspace_bytes=64), xb.ERR_WORKSPACE),   # few channels: the tokens are cut into segments
    (dict(S=4096, workspace=None), xb.ERR_WORKSPACE),
    (dict(B=0, x=None), xb.OK),
])
def test_scan_fwd_refusals(over, expect):
    assert _call(xb.xlstm_ssm_scan_fwd, SCAN, over) == expect


SCAN_STEP = dict(x="p", delta="p", A="p", Bm="p", Cm="p", D="p", z="p", delta_bias="p", h="p", y="p", B=2, C=64, N=16, G=1, dt=xb.BF16,
                 act=xb.DELTA_SOFTPLUS, stream=None)


@pytest.mark.parametrize("over,expect", [
    (dict(h=None), xb.ERR_NULL),
    (dict(y=None), xb.ERR_NULL),
    (dict(h="=x"), xb.ERR_UNSUPPORTED),
    (dict(y="=x"), xb.ERR_UNSUPPORTED),
    (dict(y="=h"), xb.ERR_UNSUPPORTED),
    (dict(h=FAKE + 4), xb.ERR_ALIGN),
    (dict(N=-1), xb.ERR_SHAPE),
    (dict(B=0), xb.OK),
])
def test_scan_step_refusals(over, expect):
    assert _call(xb.xlstm_ssm_scan_step, SCAN_STEP, over) == expect


SCAN_BWD = dict(x="p", delta="p", A="p", Bm="p", Cm="p", D="p", z="p", delta_bias="p", h0="p", dy="p", dh="p", dx="p", ddelta="p",
                dA="p", dBm="p", dCm="p", dD="p", dz="p", ddelta_bias="p", dh0="p", B=2, S=8, C=64, N=16, G=1, dt=xb.BF16,
                act=xb.DELTA_SOFTPLUS, workspace="p", workspace_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("over,expect", [
    (dict(dy=None), xb.ERR_NULL),
    (dict(dx=None), xb.ERR_NULL),
    (dict(dA=None), xb.ERR_NULL),
    (dict(dCm=None), xb.ERR_NULL),
    (dict(z=None), xb.ERR_NULL),                         # a gradient of a gate that is not there
    (dict(dz=None), xb.ERR_NULL),                        # and a gate without its gradient
    (dict(dx="=x"), xb.ERR_UNSUPPORTED),
    (dict(dz="=dy"), xb.ERR_UNSUPPORTED),
    (dict(dBm="=dCm"), xb.ERR_UNSUPPORTED),
    (dict(dh0="=dh"), xb.ERR_UNSUPPORTED),
    (dict(dD="=D"), xb.ERR_UNSUPPORTED),
    (dict(dA=FAKE + 4), xb.ERR_ALIGN),
    (dict(dh=FAKE + 8), xb.ERR_ALIGN),
    (dict(workspace=None), xb.ERR_WORKSPACE),
    (dict(workspace_bytes=1024), xb.ERR_WORKSPACE),
    (dict(S=64 * 65535 + 1), xb.ERR_SHAPE),
    (dict(N=65), xb.ERR_SHAPE),
    (dict(act=-1), xb.ERR_DTYPE),
])
def test_scan_bwd_refusals(over, expect):
    assert _call(xb.xlstm_ssm_scan_bwd, SCAN_BWD, over) == expect


def test_scan_workspace_is_for_few_channels_alone():
    st, few = xb.xlstm_ssm_scan_fwd_workspace_size(1, 4096, 64, 16, 1, xb.BF16)
    assert st == xb.OK and few > 0
    assert xb.xlstm_ssm_scan_fwd_workspace_size(8, 4096, 4096, 16, 1, xb.BF16) == (xb.OK, 0)
    assert xb.xlstm_ssm_scan_fwd_workspace_size(1, 0, 64, 16, 1, xb.BF16) == (xb.OK, 0)


def test_the_scan_refuses_host_tensors_and_bad_shapes():
    x, bc = torch.zeros(1, 4, 16), torch.zeros(1, 4, 1, 8)
    with pytest.raises(ValueError, match="CUDA tensor"):
        xb.ssm_scan_fwd(x, x, -torch.ones(16, 8), bc, bc)
    with pytest.raises(ValueError, match="CUDA tensor"):
        xb.ssm_scan_bwd(x, x, -torch.ones(16, 8), bc, bc, x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        xb.ssm_scan_step(x[:, 0], x[:, 0], -torch.ones(16, 8), bc[:, 0], bc[:, 0], torch.zeros(1, 16, 8))


def test_sizes_past_an_int_are_refused():
    """2^32 + 5 tokens would reach the library as 5."""
    long = torch.empty(1, dtype=torch.bfloat16).expand(1, (1 << 32) + 5, 8)
    flat = torch.empty(1, dtype=torch.bfloat16).expand((1 << 32) + 5, 8)
    w, A = torch.zeros(8, 4), torch.zeros(8, 16)
    state = torch.zeros(1, 3, 8, dtype=torch.bfloat16)
    calls = (lambda: xb._rows(flat), lambda: xb._rows(flat.T), lambda: xb.causal_conv_fwd(long, w),
             lambda: xb.causal_conv_bwd(long, w, long), lambda: xb.causal_conv_step(flat, w, state),
             lambda: xb._scan_args(long, long, A, long[:, :, None], long[:, :, None], None, None, None),
             lambda: xb._scan_args(long[:, :5], long[:, :5], A, flat[None, None], flat[None, None], None, None, None))
    for call in calls:
        with pytest.raises(ValueError, match="at most 2"):
            call()
