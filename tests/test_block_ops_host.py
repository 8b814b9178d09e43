"""CPU tests of the block operators' host side: arguments are checked before
anything else, so every refusal shows without a GPU; host tensors are refused by
the binding; the scratch size follows from the shape."""
import pytest
import torch

import mixed_precision_numerics_gb300 as M

A = 4096  # a pointer that is aligned to everything
F, B, P, Q = (getattr(M.lib, n) for n in ("rmsnorm_residual_fp8", "rmsnorm_residual_backward", "swiglu_fp8", "swiglu_backward"))


def norm(x=A, residual=None, x_dtype=M.MP_BF16, rows=4, cols=256, weight=A, w_dtype=M.MP_F32, eps=1e-5, h=None, y=A,
         fp8=M.MP_E4M3, block=128, scales=A, rstd=None, ckpt=None, ckpt_scales=None):
    return F(x, residual, x_dtype, rows, cols, weight, w_dtype, eps, h, y, fp8, block, scales, rstd, ckpt, ckpt_scales, None)


def norm_bwd(dy=A, dh=None, x_dtype=M.MP_BF16, rows=4, cols=256, h=A, ckpt=None, ckpt_scales=None, weight=A,
             w_dtype=M.MP_F32, rstd=A, dx=A, dweight=A, dw_dtype=M.MP_F32, workspace=A, nbytes=1 << 30):
    return B(dy, dh, x_dtype, rows, cols, h, ckpt, ckpt_scales, weight, w_dtype, rstd, dx, dweight, dw_dtype, workspace,
             nbytes, None)


def swiglu(gate=A, up=A, ld=256, x_dtype=M.MP_BF16, rows=4, cols=256, y=A, fp8=M.MP_E4M3, block=128, scales=A, ckpt=None,
           ckpt_scales=None):
    return P(gate, up, ld, x_dtype, rows, cols, y, fp8, block, scales, ckpt, ckpt_scales, None)


def swiglu_bwd(dp=A, x_dtype=M.MP_BF16, rows=4, cols=256, gate=A, up=A, ld=256, ckpt=None, ckpt_scales=None, dgate=A,
               dup=A, d_ld=256):
    return Q(dp, x_dtype, rows, cols, gate, up, ld, ckpt, ckpt_scales, dgate, dup, d_ld, None)


@pytest.mark.parametrize("call,bad", [
    (norm, dict(x=None)), (norm, dict(weight=None)), (norm, dict(y=None)), (norm, dict(scales=None)),
    (norm, dict(rows=-1)), (norm, dict(cols=-16)), (norm, dict(x_dtype=M.MP_E4M3)), (norm, dict(w_dtype=9)),
    (norm, dict(fp8=M.MP_F16)), (norm, dict(block=16)), (norm, dict(eps=-1e-9)), (norm, dict(eps=float("inf"))),
    (norm, dict(eps=float("nan"))), (norm, dict(ckpt=A)), (norm, dict(ckpt_scales=A)),
    (norm_bwd, dict(dy=None)), (norm_bwd, dict(dx=None)), (norm_bwd, dict(rstd=None)), (norm_bwd, dict(weight=None)),
    (norm_bwd, dict(dweight=None)), (norm_bwd, dict(h=None)), (norm_bwd, dict(ckpt=A, ckpt_scales=A)),
    (norm_bwd, dict(h=None, ckpt=A)), (norm_bwd, dict(dw_dtype=M.MP_E5M2)), (norm_bwd, dict(rows=-4)),
    (swiglu, dict(gate=None)), (swiglu, dict(up=None)), (swiglu, dict(y=None)), (swiglu, dict(scales=None)),
    (swiglu, dict(ckpt=A)), (swiglu, dict(fp8=M.MP_E2M1)), (swiglu, dict(block=64)), (swiglu, dict(x_dtype=M.MP_E5M2)),
    (swiglu_bwd, dict(dp=None)), (swiglu_bwd, dict(gate=None)), (swiglu_bwd, dict(up=None)),
    (swiglu_bwd, dict(gate=None, up=None)), (swiglu_bwd, dict(ckpt=A, ckpt_scales=A)), (swiglu_bwd, dict(dgate=None)),
    (swiglu_bwd, dict(dup=None)), (swiglu_bwd, dict(gate=None, up=None, ckpt=A)), (swiglu_bwd, dict(rows=-1)),
])
def test_invalid_arguments(call, bad):
    assert call(**bad) == M.MP_EINVAL


@pytest.mark.parametrize("call,bad", [
    (norm, dict(cols=264)), (norm, dict(cols=272, block=32)), (norm, dict(cols=16400)), (norm, dict(rows=2**31)),
    (norm_bwd, dict(cols=8)), (norm_bwd, dict(cols=16400)), (norm_bwd, dict(rows=2**31 - 31)),
    (swiglu, dict(cols=24)), (swiglu, dict(cols=48, block=32)), (swiglu, dict(ld=255)), (swiglu, dict(ld=260)),
    (swiglu, dict(ld=258, x_dtype=M.MP_F32)), (swiglu, dict(rows=2**31)), (swiglu, dict(cols=2**31)), (swiglu, dict(rows=1, cols=2**31 - 16)),
    (swiglu, dict(rows=2**30, cols=256)), (swiglu_bwd, dict(d_ld=240)), (swiglu_bwd, dict(d_ld=257)),
    (swiglu_bwd, dict(ld=8)), (swiglu_bwd, dict(cols=40)),
])
def test_shapes_that_are_not_taken(call, bad):
    assert call(**bad) == M.MP_ESHAPE


@pytest.mark.parametrize("call,bad", [
    (norm, dict(x=A + 8)), (norm, dict(residual=A + 2)), (norm, dict(weight=A + 4)), (norm, dict(h=A + 8)),
    (norm, dict(y=A + 1)), (norm, dict(scales=A + 2)), (norm, dict(rstd=A + 1)), (norm, dict(ckpt=A + 8, ckpt_scales=A)),
    (norm, dict(ckpt=A, ckpt_scales=A + 2)), (norm_bwd, dict(dy=A + 8)), (norm_bwd, dict(dh=A + 8)),
    (norm_bwd, dict(dweight=A + 4)), (norm_bwd, dict(workspace=A + 4)), (swiglu, dict(gate=A + 4)),
    (swiglu, dict(up=A + 8)), (swiglu, dict(ckpt=A, ckpt_scales=A + 1)), (swiglu_bwd, dict(dgate=A + 8)),
    (swiglu_bwd, dict(dp=A + 8)), (swiglu_bwd, dict(gate=None, up=None, ckpt=A + 4, ckpt_scales=A)),
])
def test_misaligned_pointers(call, bad):
    assert call(**bad) == M.MP_EALIGN


def test_workspace():
    need = M.rmsnorm_workspace_size(4, 256)
    assert need >= 4 * 256 and norm_bwd(nbytes=need - 1) == M.MP_EWORKSPACE
    assert norm_bwd(workspace=None) == M.MP_EWORKSPACE
    assert M.rmsnorm_workspace_size(0, 256) == 0 == M.rmsnorm_workspace_size(4, 0)
    sizes = [M.rmsnorm_workspace_size(r, 4096) for r in (1, 2, 100, 10_000, 2**31 - 32)]
    assert sizes == sorted(sizes) and sizes[-1] <= 608 * 4096 * 4  # a workspace serves fewer rows too


def test_nothing_to_do_needs_no_pointers():
    n0 = M.mp_launch_count()
    assert norm(rows=0, x=None, weight=None, y=None, scales=None) == M.MP_OK
    assert norm(cols=0) == M.MP_OK and norm_bwd(cols=0) == M.MP_OK
    assert swiglu(rows=0, gate=None, up=None, y=None, scales=None) == M.MP_OK
    assert swiglu_bwd(cols=0, dp=None) == M.MP_OK
    assert M.mp_launch_count() == n0


def test_host_tensors_are_refused():
    x, s = torch.zeros(4, 256), torch.zeros(4, 2)
    y = torch.zeros(4, 256, dtype=torch.uint8)
    for call in (lambda: M.rmsnorm_residual_fp8(x, x[0], y, s),
                 lambda: M.rmsnorm_residual_backward(x, x[0], s[0], x, x[0], y, h=x),
                 lambda: M.swiglu_fp8(x, x, y, s), lambda: M.swiglu_backward(x, x, x, gate=x, up=x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
