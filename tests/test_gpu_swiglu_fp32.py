"""FP32 SwiGLU: nothing of an output's error may grow with the gate.

Bounds, in roundings of binary32 (EPS = 2^-24), derived from the formulas with
the base-2 exponential within 2.5 EPS and the reciprocal within 1.7:

* s = 1 / (1 + exp(-g)): 2.5 of the exponential, 1 of the factor that makes up for
  its rounded argument, 1 of the sum, 1.7 of the reciprocal; 6.2 EPS, relative.
* dup = dp * (g * s): 6.2 + 1 + 1; 9 EPS.
* dgate = (dp * u) * f, f = s + (g * s) * (1 - s).  Errors of f: 6.2 s of s; 7.2 of
  g * s and at most 1 of 1 - s, whose own error is that of s again, in all
  8.2 |g| s; 1 |f|.  The two products: 2 |f|.  With |f| <= s * (1 + |g|) that is
  within (9.2 + 11.2 |g|) s |dp * u| EPS, of which s has its 6.2 only for a gate
  below zero, where |g| counts too: (9 + 12 |g|).  For large |g| the gradient itself
  is about g * s * dp * u, so this is a constant relative error.
* a 1x128 scale, amax of (g * s) * u over 448: 6.2 + 1 + 1 + 1; 10 EPS.
"""
import pytest
import torch

import tests.test_gpu_block_ops as B

pytestmark = pytest.mark.gpu
EPS = B.EPS


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    yield


def gates(seed, rows, cols, lo, hi):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lo + (hi - lo) * torch.rand(rows, cols, generator=g, device="cuda")


def away_from_zero(seed, rows, cols):
    """Values of both signs, none near zero: every product stays in the normal range."""
    v = B.normal(seed, rows, cols)
    return torch.where(v < 0, v - 0.25, v + 0.25)


@pytest.mark.parametrize("lo,hi", [(-85.0, -60.0), (-60.0, -20.0), (-20.0, -2.0), (-2.0, 2.0), (2.0, 85.0)])
def test_backward_error_does_not_grow_with_the_gate(lo, hi):
    rows, cols = 64, 1040
    g, u, dp = gates(1, rows, cols, lo, hi), away_from_zero(2, rows, cols), away_from_zero(3, rows, cols)
    dg, du = B.swiglu_backward(dp, gate=g, up=u)
    g, u, d = g.double(), u.double(), dp.double()
    s = torch.special.expit(g)
    off = (du.double() - d * g * s).abs() / (d * g * s).abs().clamp_min(1e-300)
    assert float(off.max()) <= 9 * EPS, f"dup off by {float(off.max()) / EPS:.1f} roundings"
    off = (dg.double() - d * u * s * (1 + g * (1 - s))).abs() / ((d * u).abs() * s)
    room = (9 + 12 * g.abs()) * EPS
    assert bool((off <= room).all()), f"dgate off by {float((off / room).max()):.2f} of the bound"


def test_backward_from_the_checkpoint():
    rows, cols = 64, 1040
    g, u, dp = gates(4, rows, cols, -80.0, 4.0), away_from_zero(5, rows, cols), away_from_zero(6, rows, cols)
    o = B.swiglu(g, u)
    g, u = B.dequantise(o["ckpt"], o["ckpt_scales"])  # binary32 products in the kernel: one more rounding of g and u
    dg, du = B.swiglu_backward(dp, ckpt=o["ckpt"], ckpt_scales=o["ckpt_scales"])
    g, u = g.float().double(), u.float().double()
    d, s = dp.double(), torch.special.expit(g)
    off = (du.double() - d * g * s).abs() - 9 * EPS * (d * g * s).abs()
    assert float(off.max()) <= 0
    off = (dg.double() - d * u * s * (1 + g * (1 - s))).abs() - (9 + 12 * g.abs()) * EPS * (d * u).abs() * s
    assert float(off.max()) <= 0


@pytest.mark.parametrize("lo,hi", [(-80.0, -70.0), (-45.0, -40.0), (-10.0, 10.0)])
def test_forward_scales(lo, hi):
    rows, cols = 32, 1024
    g, u = gates(7, rows, cols, lo, hi), away_from_zero(8, rows, cols)
    o = B.swiglu(g, u)
    p = g.double() * torch.special.expit(g.double()) * u.double()
    want = p.abs().view(rows, -1, 128).amax(2) / 448
    off = float(((o["y_scales"].double() - want) / want).abs().max())
    assert off <= 10 * EPS, f"scales off by {off / EPS:.1f} roundings"


def test_gates_at_the_ends_of_the_range():
    """Where exp(-g) is 0 or infinite: the identity times up, and zeros; between them the subnormal results of
    elementary arithmetic, within 2^-149 of the logistic function."""
    g = torch.tensor([100.0, 3e38, -89.0, -104.0, -3e38, 0.0, -0.0, -87.0, -88.0, -88.5] + [1.0] * 6, device="cuda")[None]
    one = torch.ones_like(g)
    dg, du = (t[0].double().cpu() for t in B.swiglu_backward(one, gate=g, up=one))
    x = g[0].double().cpu()
    s = torch.special.expit(x)
    s[2:5] = 0.0
    assert bool(((du - x * s).abs() <= 9 * EPS * (x * s).abs() + 2.0**-149 * (1 + x.abs())).all())
    assert bool(((dg - s * (1 + x * (1 - s))).abs() <= (9 + 12 * x.abs()) * EPS * s + 2.0**-149 * (2 + x.abs())).all())
    assert float(du[0]) == 100.0 and float(dg[1]) == 1.0 and not bool(du[2:5].any()) and not bool(dg[2:5].any())
