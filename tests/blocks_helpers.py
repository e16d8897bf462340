"""Shared helpers of the tests of the operators around the recurrences.

Tolerances are sums of rounding errors.  `U` is half a step of fp32; a value
rounded to the I/O type is off by half a step of that type relative to
itself; a sum of n products in fp32 by at most (n + 1) U times the sum of
their magnitudes, whatever the order."""
import numpy as np
import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def randn(rng, shape, dtype, scale=1.0, shift=0.0):
    """A CPU tensor of `dtype` and its exact values as float64."""
    t = torch.from_numpy(rng.standard_normal(shape) * scale + shift).to(dtype)
    return t, t.double().numpy()


def within(name, got, ref, tol):
    """Every element of the tensor `got` within `tol` of `ref` (nothing NaN)."""
    g = got.detach().cpu().double().numpy()
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    if not g.size:
        return
    tol = np.broadcast_to(np.asarray(tol, dtype=np.float64), ref.shape)
    bad = ~(np.abs(g - ref) <= tol)
    if bad.any():
        i = tuple(int(k) for k in np.argwhere(bad)[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.size} outside, first at {i}: {g[i]!r} against "
                             f"{ref[i]!r}, tolerance {tol[i]:.3e}")


def as_view(t, kind):
    """The CPU tensor on the GPU: "plain" contiguous, "half" the second half
    of rows twice as wide, "odd" rows one element longer (no wide alignment),
    "wide" rows padded by a multiple of 16 bytes, "time" time-major memory."""
    if t is None:
        return None
    t = t.cuda()
    if kind == "plain":
        return t
    B, T, D = t.shape
    if kind == "time":
        return t.transpose(0, 1).contiguous().transpose(0, 1)
    pad, at = {"half": (D, D), "odd": (1, 1), "wide": (16, 8)}[kind]
    full = torch.full((B, T, D + pad), float("nan"), dtype=t.dtype, device="cuda")
    full[..., at:at + D] = t
    return full[..., at:at + D]
