"""Shared by the tests of the selective block's operators: types, tolerances and inputs.

Tolerances, relative in the 2-norm: an output rounded once to bfloat16 (7 fraction bits) or
float16 (10) is off by at most half a unit in the last place of each element, 2^-8 and 2^-11
(float16 below its normal range, 2^-24 here: 2^-25 more in absolute value).  In float32 a
result of n products summed in any order is off by about sqrt(n) 2^-24 of the terms' size
and activations by a few 2^-24: 1e-5 holds sums of up to 10^4 terms with cancellation."""
import numpy as np
import torch

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
F32_TOL = 1e-5
TOL = {torch.float32: F32_TOL, torch.bfloat16: 2.0 ** -8 + F32_TOL, torch.float16: 2.0 ** -11 + F32_TOL}


def need_gpu():
    import pytest
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__ as g
    g.build()


def to64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def close(got, ref, name, tol=None):
    tol = TOL[got.dtype] if tol is None else tol
    g = to64(got)
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    assert np.isfinite(g).all(), name
    off = np.linalg.norm(g - ref)
    slack = 2.0 ** -25 * np.sqrt(g.size) if got.dtype == torch.float16 else 0.0
    assert off <= tol * np.linalg.norm(ref) + slack, (name, off / max(np.linalg.norm(ref), 1e-300), tol)


class Inputs:
    """Seeded device tensors; `wide` gives a slice of a wider array, so that rows are strided."""

    def __init__(self, seed):
        self.rng = np.random.default_rng(seed)

    def normal(self, *shape, dtype=torch.float32, scale=1.0, shift=0.0):
        return torch.from_numpy(self.rng.standard_normal(shape) * scale + shift).to(dtype).cuda()

    def wide(self, *shape, dtype=torch.float32, scale=1.0, left=3, right=2):
        """The channels [left, left + C) of rows of left + C + right channels."""
        full = self.normal(*shape[:-1], left + shape[-1] + right, dtype=dtype, scale=scale)
        return full[..., left:left + shape[-1]]
