"""Shared helpers of the tests of the operators between a block's projections.

Tolerances.  U[dtype] bounds the relative error of one rounding to a type.
E = 2^-24 is float32's; a sum of n terms in a tree of depth d is within d E of
the sum of the terms' magnitudes.  Every bound below is
    U[out] |ref| + (float32 error of the computation before it),
with the second part from the depth of the kernel's sums.
"""
import numpy as np
import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 1e-38, torch.bfloat16: 1e-38, torch.float16: 2.0 ** -24}  # subnormal steps
E = 2.0 ** -24
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def draw(rng, shape, dtype=torch.float32, std=1.0):
    """A GPU tensor of rounded normal values, and the same values in float64."""
    t = torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32)).to(dtype)
    return t.cuda(), t.double().numpy()


def f64(t):
    return t.detach().cpu().double().numpy()


def strided(t, pad, lead=0):
    """The same values as rows of a wider buffer whose other places hold NaN."""
    wide = torch.full((*t.shape[:-1], lead + t.shape[-1] + pad), float("nan"), dtype=t.dtype, device=t.device)
    view = wide[..., lead:lead + t.shape[-1]]
    view.copy_(t)
    return view


def check(got, ref, dtype, mag, what=""):
    """|got - ref| <= U |ref| + mag, non-finite places alike."""
    got = f64(got)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    fine = np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{what}: NaN in other places"
    assert np.array_equal(got[~fine & ~np.isnan(ref)], ref[~fine & ~np.isnan(ref)]), f"{what}: infinities differ"
    tol = np.broadcast_to(U[dtype] * np.abs(ref) * (1 + 2.0 ** -8) + mag + TINY[dtype], ref.shape)
    off = np.abs(np.where(fine, got - np.where(fine, ref, 0.0), 0.0))
    bad = fine & ~(off <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} outside, first at "
                           f"{np.argwhere(bad)[0].tolist()}: {got[bad][:3]} for {ref[bad][:3]}, worst "
                           f"{np.max(off[fine] / tol[fine]):.3g} times the bound")
