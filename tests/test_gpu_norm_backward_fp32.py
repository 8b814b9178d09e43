"""FP32 norm backward next to a large stream gradient: dh is rounded into dx once.

dx = rstd * (g - xh * c) + dh with g = dy * w, xh = v * rstd, c = mean(g * xh).
Where |dh| is far above the rest, what counts is the last addition, half a step
of dx.  In roundings of binary32 (EPS = 2^-24) the other terms are: g and its
product, 3 * |rstd * g|; of xh * rstd * c two factors of rstd, a scale and a
code's product, the factor 1 / cols and four products, 9 on top of the row's sum
(ROW_CHAIN) of magnitudes; the sum of both, 1 of each.
"""
import pytest
import torch

import tests.test_gpu_block_ops as B

pytestmark = pytest.mark.gpu
EPS = B.EPS


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    yield


# rows in lanes of a warp, two rows a team, two units a thread, one stage, dh read directly (from h)
@pytest.mark.parametrize("cols", [96, 512, 1040, 2064, 9216, 16384])
@pytest.mark.parametrize("saved", [True, False])
def test_the_stream_gradient_is_rounded_once(cols, saved):
    rows = 305
    h, dy, dh = B.normal(1, rows, cols, sigma=2.0), B.normal(2, rows, cols, sigma=1e-3), B.normal(3, rows, cols)
    w = 1.0 + B.normal(4, cols, sigma=0.2)
    o = B.norm(h, w)
    if saved:
        v = B.dequantise(o["ckpt"], o["ckpt_scales"])
        dx, _ = B.norm_backward(dy, w, o["rstd"], ckpt=o["ckpt"], scales=o["ckpt_scales"], dh=dh)
    else:
        v = h.double()
        dx, _ = B.norm_backward(dy, w, o["rstd"], h=h, dh=dh)
    r, g = o["rstd"].double()[:, None], dy.double() * w.double()
    xh = v * r
    c, c_abs = (g * xh).mean(1, keepdim=True), (g * xh).abs().mean(1, keepdim=True)
    want = r * (g - xh * c) + dh.double()
    room = EPS * (want.abs() + 5 * (r * g).abs() + (B.ROW_CHAIN + 12) * (r * xh).abs() * c_abs) + 2.0**-140
    off = (dx.double() - want).abs()
    assert bool((off <= room).all()), f"dx off by {float((off / room).max()):.2f} of the bound"
