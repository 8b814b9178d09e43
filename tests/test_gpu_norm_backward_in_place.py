"""dx over dy, over dh and over h, in every layout of the backward norm, from the stream and from its checkpoint,
with enough rows that a team's rings wrap while earlier rows are overwritten."""
import pytest
import torch

import tests.test_gpu_block_ops as B

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    yield


@pytest.mark.parametrize("saved", [True, False])
@pytest.mark.parametrize("dtype,cols", [
    ("bf16", 208),    # rows in lanes of a warp
    ("f16", 640),     # rows in whole tiles of a team
    ("bf16", 2048), ("f32", 1040),  # two rows a team
    ("bf16", 5120), ("f32", 2064),  # two units a thread
    ("bf16", 16384),  # from h with dh: room for one stage
    ("f32", 9216), ("f32", 12288),  # the same, from h and from either
    ("f32", 16384),   # from h: dh read directly
])
def test_in_place(dtype, cols, saved):
    rows = min(20_000, (1 << 24) // cols)
    h, dy, dh = (B.normal(600 + i, rows, cols, dtype=B.TYPES[dtype]) for i in range(3))
    w = 1.0 + B.normal(603, cols, sigma=0.2)
    o = B.norm(h, w)
    kw = dict(ckpt=o["ckpt"], scales=o["ckpt_scales"]) if saved else dict(h=h)
    dx, dw = B.norm_backward(dy, w, o["rstd"], dh=dh, **kw)
    dx, dw = dx.clone(), dw.clone()
    for over in ("dy", "dh") if saved else ("dy", "dh", "h"):
        t = dict(dy=dy.clone(), dh=dh.clone(), h=h.clone())
        kw = dict(ckpt=o["ckpt"], scales=o["ckpt_scales"]) if saved else dict(h=t["h"])
        got, gw = B.norm_backward(t["dy"], w, o["rstd"], dh=t["dh"], in_place=t[over], **kw)
        B.assert_bits(got, dx, f"dx over {over}")
        B.assert_bits(gw, dw, f"dweight with dx over {over}")
    kw = dict(ckpt=o["ckpt"], scales=o["ckpt_scales"]) if saved else dict(h=h)
    dx, dw = B.norm_backward(dy, w, o["rstd"], **kw)  # without dh the rings hold less
    t = dy.clone()
    got, gw = B.norm_backward(t, w, o["rstd"], in_place=t, **kw)
    B.assert_bits(got, dx, "dx over dy without dh")
    B.assert_bits(gw, dw, "dweight with dx over dy without dh")
    assert B.M.mp_wait_failures() == 0
