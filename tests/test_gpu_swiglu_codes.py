"""The SwiGLU product's codes are the nearest ones.

A value is p = (g * s) * u against the exact product: s is within (1.25 |g| + 8)
roundings of binary32 (EPS = 2^-24), the two products add one each.  The code is p
times a multiplier, relative to the stored scale: a rounding each of the multiplier,
of that product and of the scale; with the second-order terms (1.25 |g| + 14) EPS.
"""
import pytest
import torch

import tests.test_gpu_block_ops as B
from tests.fp8_bound import room

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    yield


@pytest.mark.parametrize("shape", [(1, 14336), (37, 160), (301, 1440)])
@pytest.mark.parametrize("dtype", B.TYPES)
@pytest.mark.parametrize("fp8", B.FP8)
@pytest.mark.parametrize("block", [128, 32])
@pytest.mark.parametrize("sigma", [2.0, 20.0])
def test_codes_are_the_nearest(shape, dtype, fp8, block, sigma):
    rows, cols = shape
    g, u = B.halves(500 + rows, rows, cols, B.TYPES[dtype], sigma=sigma)
    g = g.clamp(min=-80.0)  # below, a tile may be all subnormal
    u = u.clone()
    o = B.swiglu(g, u, fp8=fp8, block=block)
    f8 = B.FP8[fp8][1]
    s = o["y_scales"].double() if block == 128 else torch.exp2(o["y_scales"].double() - 127)
    s = s.repeat_interleave(block, 1)[:, :cols]
    g, u = g.double(), u.double()
    q = g * torch.special.expit(g) * u / s
    off, limit = (o["y"].view(f8).double() - q).abs(), room(q, (1.25 * g.abs() + 14) * B.EPS, f8)
    assert bool((off <= limit).all()), f"off by {float((off / limit).max()):.3f} of the bound"
