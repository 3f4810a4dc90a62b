"""GPU parity of ``xlstm_rmsnorm_fwd`` / ``_bwd`` against the float64 oracle
(``oracle.block``).

Tolerances, from the arithmetic (EPS = 2^-24, half an fp32 step):
 * the mean square is a sum of squares with at most 16 serial and 10 tree
   additions, so rstd is off by at most 13 EPS from it, 4 EPS from rsqrt and the
   division, and y by 3 more: 32 EPS |y| covers it;
 * an e4m3 code is off by half a step of its value (2^-4 relative, 2^-10 scale
   below the smallest normal), the scale by 32 EPS;
 * dx = rstd (g - n m): every term is formed with at most 32 relative roundings,
   so the error is at most 48 EPS of the terms' magnitudes;
 * dgamma adds at most 64 terms one after another in any place: 64 EPS of the
   sum of magnitudes."""
import numpy as np
import pytest
import torch

import oracle.block as ob
from blockparity import BF16, EPS32, F32, cuda, normal, within
from linear_rnn_mlstm_b200 import autograd as xa
from linear_rnn_mlstm_b200 import binding as xb

pytestmark = pytest.mark.gpu

# one channel vector, part of a warp, a whole warp's vectors, one past it, CTA forms, the widest
WIDTHS = (8, 24, 256, 264, 512, 1032, 2048, 4104, 8192)


def _inputs(rows, C, dtype, residual, seed=0):
    x = dict(x=normal(seed, rows, C, dtype=dtype), gamma=normal(seed + 1, C, scale=0.2, mean=1.0),
             residual=normal(seed + 2, rows, C, dtype=dtype, scale=3.0) if residual else None)
    if rows > 2:
        x["x"][1] = 0
        if residual:
            x["residual"][1] = 0                                   # a row of zeros
    return x


@pytest.mark.parametrize("dtype", (F32, BF16), ids=("f32", "bf16"))
@pytest.mark.parametrize("residual", (False, True))
@pytest.mark.parametrize("C", WIDTHS)
def test_forward(C, residual, dtype):
    for rows in (1, 13):
        x = _inputs(rows, C, dtype, residual, seed=C)
        d = cuda(x)
        y, s, rstd = xb.rmsnorm(d["x"], d["gamma"], d["residual"], eps=1e-5)
        yr, sr, rr = ob.rmsnorm(x["x"], x["gamma"], x["residual"], eps=1e-5)
        within(rstd, rr, 20 * EPS32 * rr, "rstd")
        within(y, yr, 32 * EPS32 * np.abs(yr), "y")
        if residual:
            within(s, sr, 0.0, "s")
        else:
            assert s is d["x"]


@pytest.mark.parametrize("dtype", (F32, BF16), ids=("f32", "bf16"))
@pytest.mark.parametrize("C,group", [(8, 0), (128, 32), (128, 128), (192, 64), (640, 128), (2048, 0), (2048, 128), (4224, 32),
                                     (8192, 128), (8184, 0)])
def test_eight_bit_output(C, group, dtype):
    x = _inputs(9, C, dtype, True, seed=C + group)
    d = cuda(x)
    q, scales, s = xb.rmsnorm_fp8(d["x"], d["gamma"], d["residual"], group=group)
    yr, sr, _ = ob.rmsnorm(x["x"], x["gamma"], x["residual"])
    _, scr = ob.quantise(yr, group)
    within(scales, scr, 32 * EPS32 * scr, "scales")
    within(s, sr, 0.0, "s")
    got = (q.float().cpu().double().numpy().reshape(*scr.shape, -1) * scales.cpu().double().numpy()[..., None])
    ref, step = yr.reshape(got.shape), scr[..., None]
    room = 2.0 ** -4 * np.abs(ref) + 2.0 ** -10 * step + 64 * EPS32 * np.abs(ref)
    assert np.all(np.abs(got - ref) <= room * (1 + 2.0 ** -4))
    assert not q[1].float().any() and float(scales[1].max()) == ob.SCALE_MIN       # the row of zeros
    assert float(q.float().abs().max()) == ob.F8_MAX


def test_both_outputs_in_one_call_and_streams_updated_in_place():
    x = cuda(_inputs(7, 512, BF16, True))
    y0, s0, _ = xb.rmsnorm(x["x"], x["gamma"], x["residual"])
    q0, sc0, _ = xb.rmsnorm_fp8(x["x"], x["gamma"], x["residual"], group=64)
    q, sc = torch.empty_like(q0), torch.empty_like(sc0)
    # s in the residual's place and y in x's
    st = xb.xlstm_rmsnorm_fwd(x["x"].data_ptr(), x["residual"].data_ptr(), x["gamma"].data_ptr(), x["residual"].data_ptr(),
                              x["x"].data_ptr(), q.data_ptr(), sc.data_ptr(), None, 7, 512, 64, 1e-5, xb.BF16,
                              torch.cuda.current_stream().cuda_stream)
    assert st == xb.OK
    torch.cuda.synchronize()
    assert torch.equal(x["residual"], s0) and torch.equal(x["x"], y0)
    assert torch.equal(q.view(torch.uint8), q0.view(torch.uint8)) and torch.equal(sc, sc0)


def test_a_nan_or_infinity_stays_in_its_row():
    x = _inputs(4, 256, F32, False)
    x["x"][0, 17] = float("nan")
    x["x"][2, 3] = float("inf")
    d = cuda(x)
    y, _, _ = xb.rmsnorm(d["x"], d["gamma"])
    q, sc, _ = xb.rmsnorm_fp8(d["x"], d["gamma"], group=128)
    assert y[0].isnan().all() and q[0].float().isnan().all()
    assert y[2, 3].isnan() and not y[2, :3].any()                   # rstd = 0: inf * 0 and finite * 0
    assert y[1].isfinite().all() and y[3].isfinite().all() and sc[3].isfinite().all()


@pytest.mark.parametrize("dtype", (F32, BF16), ids=("f32", "bf16"))
@pytest.mark.parametrize("with_ds", (False, True))
@pytest.mark.parametrize("rows,C", [(1, 8), (37, 24), (700, 256), (5, 1032), (1500, 2048), (64, 4104), (9, 8192)])
def test_backward(rows, C, with_ds, dtype):
    s, gamma = normal(C, rows, C, dtype=dtype, scale=2.0), normal(1, C, scale=0.2, mean=1.0)
    dy, ds = normal(2, rows, C, dtype=dtype), normal(3, rows, C, dtype=dtype) if with_ds else None
    _, _, rstd = ob.rmsnorm(s, gamma)
    rstd = torch.from_numpy(rstd).float()
    d = cuda(dict(dy=dy, s=s, gamma=gamma, rstd=rstd, ds=ds))
    dx, dgamma = xb.rmsnorm_bwd(**d)
    dxr, dgr = ob.rmsnorm_grads(dy, s, gamma, ds=ds, rstd=rstd)
    n = np.abs(ob.f64(s)) * ob.f64(rstd)[:, None]
    g = np.abs(ob.f64(dy) * ob.f64(gamma))
    size = ob.f64(rstd)[:, None] * (g + n * (g * n).mean(1, keepdims=True)) + (np.abs(ob.f64(ds)) if with_ds else 0)
    within(dx, dxr, 48 * EPS32 * size, "dx")
    within(dgamma, dgr, 64 * EPS32 * (np.abs(ob.f64(dy)) * n).sum(0), "dgamma")
    again = xb.rmsnorm_bwd(**d)
    assert torch.equal(dx, again[0]) and torch.equal(dgamma, again[1])


def test_backward_without_rows_writes_zero_dgamma():
    e = torch.empty(0, 64, device="cuda")
    dx, dgamma = xb.rmsnorm_bwd(e, e, torch.ones(64, device="cuda"), torch.empty(0, device="cuda"))
    assert dx.shape == (0, 64) and not dgamma.any()


def test_autograd_of_the_stream_and_the_norm():
    x, r, gamma = (t.cuda().requires_grad_() for t in (normal(0, 2, 5, 64), normal(1, 2, 5, 64), normal(2, 64, mean=1.0)))
    wy, ws = normal(3, 2, 5, 64).cuda(), normal(4, 2, 5, 64).cuda()
    y, s = xa.rmsnorm(x, gamma, r)
    ((y * wy).sum() + (s * ws).sum()).backward()
    dx, dg = ob.rmsnorm_grads(wy.cpu(), (x + r).detach().cpu(), gamma.detach().cpu(), ds=ws.cpu())
    for t in (x, r):
        np.testing.assert_allclose(t.grad.cpu().numpy(), dx, rtol=0, atol=2e-5 * np.abs(dx).max())
    np.testing.assert_allclose(gamma.grad.cpu().numpy(), dg, rtol=0, atol=2e-5 * np.abs(dg).max())
    y, s = xa.rmsnorm(x, gamma)
    assert s is x
