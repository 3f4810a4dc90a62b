"""Host-side edges of the block operators (norm, convolution, scan) on the CPU: the
largest sizes that a call may name, and what a call tells autograd of the tensors it
writes in place."""
import pytest
import torch

from linear_rnn_mlstm_b200 import binding as xb


@pytest.mark.parametrize("dt", (xb.F32, xb.BF16))
def test_norm_workspace_at_the_most_rows(dt):
    """The number of CTAs must not wrap: a full wave, as for any large number of rows."""
    for C in (8, 512, 8192):                                  # a warp per row, and a CTA per row
        want = xb.xlstm_rmsnorm_bwd_workspace_size(1 << 20, C, dt)
        assert want[0] == xb.OK and 0 < want[1] < 1 << 26
        for rows in ((1 << 31) - 8, (1 << 31) - 7, (1 << 31) - 1):
            assert xb.xlstm_rmsnorm_bwd_workspace_size(rows, C, dt) == want, (rows, C)


# ---------------------------------------------------- what autograd is told
@pytest.fixture
def launches(monkeypatch):
    """The binding's conveniences on host tensors: every launch of the library is a
    stand-in that reports success (what it would write is set by the test)."""
    import contextlib
    monkeypatch.setattr(xb, "_check", lambda *a: None)
    monkeypatch.setattr(xb, "_on", lambda *a: contextlib.nullcontext())
    monkeypatch.setattr(xb, "_stream", lambda dev: None)
    for name in ("xlstm_rmsnorm_fwd", "xlstm_causal_conv_fwd", "xlstm_causal_conv_step", "xlstm_ssm_scan_fwd", "xlstm_ssm_scan_step",
                 "xlstm_mlstm_fwd", "xlstm_mlstm_step", "xlstm_mlstm_headnorm_gate", "xlstm_mlstm_seg_state", "xlstm_mlstm_state_combine"):
        monkeypatch.setattr(xb, name, lambda *a: xb.OK)
    return monkeypatch


def test_what_a_call_writes_in_place_counts_as_changed(launches):
    z = torch.zeros
    x, w, A, bc = z(2, 5, 64), z(64, 4), z(64, 8), z(2, 5, 1, 8)
    q, g, o = z(2, 1, 5, 64), z(2, 1, 5), z(2, 1, 5, 64)
    y, y1, conv, h = z(2, 5, 64), z(2, 64), z(2, 3, 64), z(2, 64, 8)
    C, n, m, hm, hs = z(2, 1, 64, 64), z(2, 1, 64), z(2, 1), z(2, 1, 5, 64), z(2, 1, 64)
    packed = z(xb.seg_state_floats(2, 1, 64))
    token = (x[:, 0], x[:, 0], A, bc[:, 0], bc[:, 0])
    qt, gt = q[:, :, 0], g[:, :, 0]
    for written, read, call in (
            ([y], [x], lambda: xb.rmsnorm(x, z(64), y=y)),
            ([y], [x, w], lambda: xb.causal_conv_fwd(x, w, y=y)),
            ([conv, y1], [x, w], lambda: xb.causal_conv_step(x[:, 0], w, conv, y=y1)),
            ([conv], [x, w], lambda: xb.causal_conv_step(x[:, 0], w, conv)),
            ([y], [x, A, bc, h], lambda: xb.ssm_scan_fwd(x, x, A, bc, bc, h0=h, y=y)),
            ([h, y1], [x, A, bc], lambda: xb.ssm_scan_step(*token, h, y=y1)),
            ([h], [x, A, bc], lambda: xb.ssm_scan_step(*token, h)),
            ([hm], [q, g, C, n, m], lambda: xb.mlstm_fwd(q, q, q, g, g, o, C0=C, n0=n, m0=m, h=hm)),
            ([C, n, m, hs], [q, g], lambda: xb.mlstm_step(qt, qt, qt, gt, gt, qt, C, n, m, h=hs)),
            ([C, n, m], [q, g], lambda: xb.mlstm_step(qt, qt, qt, gt, gt, qt, C, n, m)),
            ([y], [q, x], lambda: xb.mlstm_headnorm_gate(q, z(64), z(64), x, y=y)),
            ([packed], [q, g], lambda: xb.mlstm_seg_state(q, q, g, g, packed=packed)),
            ([C, n, m], [packed], lambda: xb.mlstm_state_combine(packed[None], 1, 2, 1, 64, out=(C, n, m)))):
        before = [t._version for t in written], [t._version for t in read]
        call()
        assert all(t._version > v for t, v in zip(written, before[0]))
        assert [t._version for t in read] == before[1]


def test_a_state_stepped_after_the_forward_is_refused_by_its_backward(launches):
    """The scan and the convolution save the state they started from; a step moves it on in place."""
    from linear_rnn_mlstm_b200 import autograd as xa
    z = torch.zeros
    leaf = lambda *shape: z(*shape).requires_grad_()
    launches.setattr(xb, "causal_conv_bwd", lambda *a, **k: pytest.fail("ran on a changed state"))
    launches.setattr(xb, "ssm_scan_bwd", lambda *a, **k: pytest.fail("ran on a changed state"))
    x, w, A, bc, conv, h = leaf(2, 5, 64), leaf(64, 4), leaf(64, 8), leaf(2, 5, 1, 8), z(2, 3, 64), z(2, 64, 8)
    y, _ = xa.causal_conv(x, w, state0=conv)
    xb.causal_conv_step(x[:, 0].detach(), w.detach(), conv)
    with pytest.raises(RuntimeError, match="inplace operation"):
        y.sum().backward()
    y, _ = xa.ssm_scan(x, x, A, bc, bc, h0=h)
    xb.ssm_scan_step(*(t.detach() for t in (x[:, 0], x[:, 0], A, bc[:, 0], bc[:, 0])), h)
    with pytest.raises(RuntimeError, match="inplace operation"):
        y.sum().backward()
    u = leaf(2, 5, 64)                                        # a saved input that is another call's y
    y, _ = xa.causal_conv(u * 1.0, w)
    s = u * 1.0
    y, _ = xa.rmsnorm(s, leaf(64))
    with torch.no_grad():
        xb.causal_conv_fwd(x.detach(), w.detach(), y=s)
    with pytest.raises(RuntimeError, match="inplace operation"):
        y.sum().backward()


def test_a_norm_in_its_inputs_place_returns_no_stream(launches):
    """x holds y afterwards: handed on as s it would give wrong gradients."""
    x, r, g = torch.zeros(4, 64), torch.zeros(4, 64), torch.ones(64)
    y, s, rstd = xb.rmsnorm(x, g, y=x)
    assert y is x and s is None and rstd.shape == (4,)
    y, s, _ = xb.rmsnorm(x, g, y=x.view(4, 64))
    assert s is None
    y, s, _ = xb.rmsnorm(x, g)
    assert s is x and y is not x
    none = torch.zeros(0, 64)
    assert xb.rmsnorm(none, g)[1] is none
    y, s, _ = xb.rmsnorm(x, g, r, y=x)                        # with a residual the stream is a tensor of its own
    assert y is x and s.data_ptr() not in (x.data_ptr(), r.data_ptr())


def test_tensors_made_in_inference_mode_can_be_written(launches):
    with torch.inference_mode():
        h, conv = torch.zeros(2, 64, 8), torch.zeros(2, 3, 64)
        x, bc = torch.zeros(2, 64), torch.zeros(2, 1, 8)
        xb.ssm_scan_step(x, x, torch.zeros(64, 8), bc, bc, h)
        xb.causal_conv_step(x, torch.zeros(64, 4), conv, y=torch.zeros(2, 64))


# ------------------------------------------------------------------- lengths
def test_lengths_may_start_anywhere_in_a_batchs_vector():
    """They are read one by one: a slice of a dense vector passes (a later refusal shows it)."""
    from test_block_abi import CONV, FAKE, SCAN, _call
    for fn, base in ((xb.xlstm_causal_conv_fwd, CONV), (xb.xlstm_ssm_scan_fwd, SCAN)):
        assert _call(fn, base, dict(lengths=FAKE + 4, y="=x")) == xb.ERR_UNSUPPORTED
        assert _call(fn, base, dict(lengths=FAKE + 2, y="=x")) == xb.ERR_ALIGN
