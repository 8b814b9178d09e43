"""CPU tests of the gated feed-forward products' and the gradient norm's host side: every refusal comes before
anything else, so it shows without a GPU; host tensors are refused by the binding."""
import ctypes

import pytest
import torch

import mixed_precision_numerics_gb300 as M

A = 4096  # a pointer that is aligned to everything
NAN, INF = float("nan"), float("inf")


def fwd(x=A, t=M.MP_BF16, rows=4, width=64, hidden=256, wg=A, wu=A, p=A, p_t=M.MP_E4M3, block=128, scales=A, gate=None,
        up=None, ld=256, ckpt=None, ckpt_scales=None):
    return M.lib.linear_swiglu(x, t, rows, width, hidden, wg, wu, p, p_t, block, scales, gate, up, ld, ckpt, ckpt_scales, None)


def bwd(dp=A, t=M.MP_BF16, rows=4, width=64, hidden=256, x=A, wg=A, wu=A, gate=A, up=A, ld=256, ckpt=None,
        ckpt_scales=None, dx=A, dwg=A, dwu=A, ws=A, nbytes=1 << 30):
    return M.lib.linear_swiglu_backward(dp, t, rows, width, hidden, x, wg, wu, gate, up, ld, ckpt, ckpt_scales, dx, dwg,
                                        dwu, ws, nbytes, None)


def lists(grad=A, out=A, numel=100, gt=M.MP_F32, ot=M.MP_F32, n=2):
    arr = (M.MpGrad * 2)()
    arr[0] = M.MpGrad(2 * A, 2 * A, 8, M.MP_BF16, M.MP_BF16)
    arr[1] = M.MpGrad(grad, out, numel, gt, ot)
    return arr, n


def norm(ls=None, scale=None, to=A, ws=A, nbytes=1 << 30, **kw):
    arr, n = lists(**kw)
    return M.lib.mp_grad_norm(arr, n, scale, to, ws, nbytes, None)


def clip(to=A, most=1.0, **kw):
    arr, n = lists(**kw)
    return M.lib.mp_grad_clip(arr, n, to, most, None)


@pytest.mark.parametrize("call,bad", [
    (fwd, dict(x=None)), (fwd, dict(wg=None)), (fwd, dict(wu=None)), (fwd, dict(p=None)), (fwd, dict(scales=None)),
    (fwd, dict(t=M.MP_F32)), (fwd, dict(p_t=M.MP_F16)), (fwd, dict(p_t=M.MP_BF16)), (fwd, dict(p_t=M.MP_E2M1)),
    (fwd, dict(block=64)), (fwd, dict(rows=-1)), (fwd, dict(width=-16)), (fwd, dict(hidden=-16)), (fwd, dict(gate=A)),
    (fwd, dict(up=A)), (fwd, dict(ckpt=A)), (fwd, dict(ckpt_scales=A)),
    (fwd, dict(gate=A, up=A, ckpt=A, ckpt_scales=A)),
    (bwd, dict(dp=None)), (bwd, dict(x=None)), (bwd, dict(wg=None)), (bwd, dict(wu=None)), (bwd, dict(gate=None)),
    (bwd, dict(up=None)), (bwd, dict(ckpt=A)), (bwd, dict(ckpt=A, ckpt_scales=A)), (bwd, dict(dwg=None)),
    (bwd, dict(dwu=None)), (bwd, dict(t=M.MP_F32)), (bwd, dict(rows=-1)),
    (norm, dict(to=None)), (norm, dict(grad=None)), (norm, dict(numel=-1)), (norm, dict(gt=M.MP_E4M3)), (norm, dict(n=-1)),
    (clip, dict(to=None)), (clip, dict(grad=None)), (clip, dict(out=None)), (clip, dict(ot=M.MP_F16)),
    (clip, dict(out=2 * A, ot=7)), (clip, dict(most=0.0)), (clip, dict(most=-1.0)), (clip, dict(most=NAN)),
    (clip, dict(most=INF)),
])
def test_invalid_arguments(call, bad):
    n0 = M.mp_launch_count()
    assert call(**bad) == M.MP_EINVAL and M.mp_launch_count() == n0


@pytest.mark.parametrize("call,bad", [
    (fwd, dict(width=24)), (fwd, dict(hidden=24)), (fwd, dict(hidden=48, block=32)), (fwd, dict(width=0)),
    (fwd, dict(rows=2**31 - 256)), (fwd, dict(width=2**20 + 16)), (fwd, dict(hidden=2**20 + 16)),
    (fwd, dict(gate=A, up=A, ld=248)), (fwd, dict(gate=A, up=A, ld=260)), (bwd, dict(width=8)), (bwd, dict(hidden=8)),
    (bwd, dict(ld=248)), (bwd, dict(ld=257)), (bwd, dict(width=0)), (bwd, dict(rows=2**31 - 256)),
    (fwd, dict(rows=2**30, hidden=2**20)),
])
def test_shapes_that_are_not_taken(call, bad):
    assert call(**bad) == M.MP_ESHAPE


@pytest.mark.parametrize("call,bad", [
    (fwd, dict(x=A + 8)), (fwd, dict(wg=A + 8)), (fwd, dict(wu=A + 2)), (fwd, dict(p=A + 1)), (fwd, dict(scales=A + 2)),
    (fwd, dict(gate=A + 8, up=A)), (fwd, dict(gate=A, up=A + 8)), (fwd, dict(ckpt=A + 4, ckpt_scales=A)),
    (fwd, dict(ckpt=A, ckpt_scales=A + 1)), (bwd, dict(dp=A + 8)), (bwd, dict(x=A + 8)), (bwd, dict(wg=A + 8)),
    (bwd, dict(dx=A + 8)), (bwd, dict(dwg=A + 8)), (bwd, dict(dwu=A + 8)), (bwd, dict(ws=A + 8)), (bwd, dict(up=A + 8)),
    (norm, dict(grad=A + 8)), (norm, dict(to=A + 2)), (norm, dict(scale=A + 2)), (norm, dict(ws=A + 8)),
    (clip, dict(grad=A + 4)), (clip, dict(out=A + 8)), (clip, dict(to=A + 1)),
])
def test_misaligned_pointers(call, bad):
    assert call(**bad) == M.MP_EALIGN


def test_workspaces():
    need = M.linear_swiglu_workspace_size(4, 64, 256)
    assert need >= 4 * 256 * 4 and bwd(nbytes=need - 1) == M.MP_EWORKSPACE and bwd(ws=None) == M.MP_EWORKSPACE
    for size in ((0, 64, 256), (4, 0, 256), (4, 64, 0), (4, 24, 256), (-1, 64, 256)):
        assert M.linear_swiglu_workspace_size(*size) == 0
    arr, n = lists()
    need = M.lib.mp_grad_norm_workspace_size(arr, n)
    assert need > 0 and norm(nbytes=need - 1) == M.MP_EWORKSPACE and norm(ws=None) == M.MP_EWORKSPACE


def test_nothing_to_do_needs_no_pointers():
    n0 = M.mp_launch_count()
    assert fwd(rows=0, x=None, wg=None, wu=None, p=None, scales=None) == M.MP_OK
    assert fwd(hidden=0, x=None, p=None) == M.MP_OK
    assert bwd(dx=None, dwg=None, dwu=None, dp=None) == M.MP_OK
    assert bwd(rows=0, hidden=0, gate=None, up=None) == M.MP_OK and bwd(rows=0, dwg=None, dwu=None) == M.MP_OK
    assert M.lib.mp_grad_clip(None, 0, A, 1.0, None) == M.MP_OK
    assert M.mp_launch_count() == n0


def test_host_tensors_are_refused():
    x, w, p = torch.zeros(4, 64).half(), torch.zeros(256, 64).half(), torch.zeros(4, 256).half()
    ws, n = torch.zeros(1 << 16, dtype=torch.uint8), torch.zeros(1)
    for call in (lambda: M.linear_swiglu(x, w, w, p), lambda: M.linear_swiglu_backward(p, x, w, w, x, w, w, ws),
                 lambda: M.mp_grad_norm([x], n, ws), lambda: M.mp_grad_clip([x], n, 1.0), lambda: M.make_grad_array([w])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="w_up"):
        M.linear_swiglu(x, w, w[:16], p)
    with pytest.raises(ValueError, match="out: 2 tensors"):
        M.make_grad_array([x], [x, w])
    with pytest.raises(ValueError, match="prebuilt"):
        M.mp_grad_clip((M.MpGrad * 1)(), n, 1.0, out=[x])


def test_struct_layout():
    assert ctypes.sizeof(M.MpGrad) == 32 and M.MpGrad.numel.offset == 16 and M.MpGrad.out_dtype.offset == 28


def test_a_plain_c_program_calls_them(tmp_path):
    import os
    import shutil
    import subprocess

    from tests.conftest import ROOT

    pkg, exe, cc = os.path.join(ROOT, "mixed_precision_numerics_gb300"), str(tmp_path / "check"), shutil.which("gcc")
    if cc is None:
        pytest.skip("no C compiler")
    p = subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"),
                        os.path.join(ROOT, "tests", "products_abi_check.c"), "-L", pkg, "-lmpnum", f"-Wl,-rpath,{pkg}",
                        "-o", exe], capture_output=True, text=True)
    assert p.returncode == 0, p.stderr
    p = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert p.returncode == 0 and "products abi ok" in p.stdout, p.stderr
