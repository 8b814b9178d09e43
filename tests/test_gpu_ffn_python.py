"""The feed-forward products and the gradient norm through the Python marshalling alone: the same results; and
what either marshalling refuses, before anything is launched."""
import pytest
import torch

import tests.test_gpu_ffn as T
import tests.test_gpu_grads as G

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture
def M(cuda_ok):
    import mixed_precision_numerics_gb300

    return mixed_precision_numerics_gb300


@pytest.mark.parametrize("check", [
    lambda M: T.test_forward(M, 37, 1040, 272, F16), lambda M: T.test_forward(M, 257, 5120, 96, BF16),
    lambda M: T.test_forward_in_8_bits(M, 301, 528, 1440, 128, "e4m3", 8),
    lambda M: T.test_forward_in_8_bits(M, 37, 1040, 288, 32, "e5m2", 16),
    lambda M: T.test_backward(M, 129, 48, 400, "16", BF16), lambda M: T.test_backward(M, 64, 512, 1456, "8", F16),
    lambda M: T.test_backward(M, 301, 1040, 1456, "again", BF16), lambda M: T.test_nothing_to_do(M, 5, 32, 0),
    lambda M: T.test_captured_and_on_two_streams(M), lambda M: G.test_mixed_types(M, F16),
    lambda M: G.test_loss_scale_and_empty_lists(M), lambda M: G.test_repeats_and_leaves_its_workspace_ready(M),
])
def test_without_the_native_marshalling(M, check, monkeypatch):
    monkeypatch.setattr(M, "_mpcall", None)
    check(M)


def z(*shape, dtype=BF16):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


@pytest.mark.parametrize("native", [True, False])
def test_refusals_launch_nothing(M, native, monkeypatch):
    x, w, p, ws = z(8, 64), z(96, 64), z(8, 96), M.new_linear_swiglu_workspace(8, 64, 96)
    dw, norm = z(2, 96, 64), z(1, dtype=F32)
    M.linear_swiglu(x, w, w, p)  # binds the native marshalling
    if not native:
        monkeypatch.setattr(M, "_mpcall", None)
    gws = M.new_grad_norm_workspace([x, w])
    n0 = M.mp_launch_count()
    back = M.linear_swiglu_backward
    for call, error in [
        (lambda: M.linear_swiglu(x.float(), w.float(), w.float(), z(8, 96, dtype=F32)), M.MpError),
        (lambda: M.linear_swiglu(x, w.half(), w, p), ValueError), (lambda: M.linear_swiglu(x, w, w[:80], p), ValueError),
        (lambda: M.linear_swiglu(x, w, z(96, 48), p), ValueError), (lambda: M.linear_swiglu(x, w, w, p.half()), ValueError),
        (lambda: M.linear_swiglu(x, w, w, z(7, 96)), ValueError), (lambda: M.linear_swiglu(x, w, w, z(96, 8).t()), ValueError),
        (lambda: M.linear_swiglu(z(8, 128)[:, :64], w, w, p), ValueError),
        (lambda: M.linear_swiglu(x.cpu(), w, w, p), ValueError), (lambda: M.linear_swiglu(x, w, w, p.cpu()), ValueError),
        (lambda: M.linear_swiglu(x, w, w, p, gate=z(8, 96)), ValueError),
        (lambda: M.linear_swiglu(x, w, w, p, gate=z(8, 96), up=z(8, 200)[:, :96]), ValueError),
        (lambda: M.linear_swiglu(x, w, w, p, gate=z(8, 80), up=z(8, 80)), ValueError),
        (lambda: M.linear_swiglu(x, w, w, p, gate=z(8, 96, dtype=F16), up=z(8, 96, dtype=F16)), ValueError),
        (lambda: M.linear_swiglu(x, w, w, p, gate=z(8, 100)[:, :96], up=z(8, 100)[:, :96]), M.MpError),  # pitch % 8
        (lambda: M.linear_swiglu(x, w, w, p, ckpt=z(2, 8, 96, dtype=torch.uint8)), M.MpError),
        (lambda: M.linear_swiglu(x, w, w, p, ckpt=z(8, 96, dtype=torch.uint8), ckpt_scales=z(2, 8, 1, dtype=F32)), ValueError),
        (lambda: M.linear_swiglu(x, w, w, z(8, 96, dtype=torch.uint8), p_scales=z(7, dtype=F32)), ValueError),
        (lambda: M.linear_swiglu(x, w, w, z(8, 96, dtype=torch.uint8), p_scales=z(8, dtype=F32), fp8_dtype=M.MP_E2M1), M.MpError),
        (lambda: M.linear_swiglu(z(8, 72), z(96, 72), z(96, 72), p), M.MpError),
        (lambda: back(p, x, w, w, x, dw[0], None, ws), M.MpError), (lambda: back(p, x, w, w, x, dw[0], dw[1], None), M.MpError),
        (lambda: back(p, x, w, w, x, dw[0], dw[1], ws[:256]), M.MpError), (lambda: back(p, x, w, w, z(7, 64), None, None, ws), ValueError),
        (lambda: back(p.half(), x, w, w, x, dw[0], dw[1], ws), ValueError),
        (lambda: back(p, x, w, w, x, dw[0].float(), dw[1].float(), ws), ValueError),
        (lambda: back(p, x, w, w, x, dw[0], dw[1], ws, gate=p), ValueError),
        (lambda: M.mp_grad_norm([x], z(1), gws), ValueError), (lambda: M.mp_grad_norm([x], norm, gws[:32]), M.MpError),
        (lambda: M.mp_grad_norm([x], norm, gws, loss_scale=z(1)), ValueError), (lambda: M.mp_grad_norm([x], norm, None), M.MpError),
        (lambda: M.mp_grad_norm([w.t()], norm, gws), ValueError), (lambda: M.mp_grad_norm([ws], norm, gws), ValueError),
        (lambda: M.mp_grad_norm([x.view(-1)[1:]], norm, gws), M.MpError), (lambda: M.make_grad_array([x, x]), ValueError),
        (lambda: M.make_grad_array([x], [z(8, 63)]), ValueError), (lambda: M.mp_grad_clip([x], norm, 0.0), M.MpError),
        (lambda: M.mp_grad_clip(M.make_grad_array([x]), norm, float("nan")), M.MpError),
        (lambda: M.mp_grad_clip(M.make_grad_array([x]), norm.cpu(), 1.0), ValueError),
        (lambda: M.mp_grad_clip([x, w], norm, 1.0, out=[x]), ValueError),
    ]:
        with pytest.raises(error):
            call()
    assert M.mp_launch_count() == n0


def test_a_list_of_another_device_is_refused(M):
    arr, norm = M.make_grad_array([z(64)]), z(1, dtype=F32)
    arr.device = 5  # as if it had been made there
    for call in (lambda: M.mp_grad_clip(arr, norm, 1.0), lambda: M.mp_grad_norm(arr, norm, M.new_grad_norm_workspace([z(64)]))):
        with pytest.raises(ValueError, match="device 5"):
            call()
