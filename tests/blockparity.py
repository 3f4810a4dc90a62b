"""Shared helpers of the block operators' GPU tests: seeded inputs and the
element-by-element comparison with a float64 reference."""
import numpy as np
import torch

F32, BF16 = torch.float32, torch.bfloat16
EPS32 = 2.0 ** -24            # half a step of fp32, relative


def normal(seed, *shape, dtype=F32, scale=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale + mean).to(dtype)


def cuda(d):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in d.items()}


def within(got, ref, bound, what):
    """|got - ref| <= bound + the rounding of the output's own type, everywhere.
    ``bound`` is the error of the fp32 arithmetic, as each test derives it."""
    half = torch.finfo(got.dtype).eps / 2
    tiny = torch.finfo(got.dtype).tiny
    got = got.detach().cpu().double().numpy()
    ref = np.asarray(ref, np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    room = bound + half * (np.abs(ref) + bound) + tiny
    worst = float(np.max(np.abs(got - ref) / room, initial=0.0))
    assert worst <= 1.0, f"{what}: {worst:.3g} of its bound"
