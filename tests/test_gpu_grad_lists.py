"""Clipping: empty gradients in a list, the clipped bits, norms beyond binary32."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture
def M(cuda_ok):
    import mixed_precision_numerics_gb300

    return mixed_precision_numerics_gb300


def norm_of(M, grads):
    norm = torch.full((1,), -7.0, device="cuda")
    M.mp_grad_norm(grads, norm, M.new_grad_norm_workspace(grads))
    return norm


@pytest.mark.parametrize("out", [F32, F16, BF16])
@pytest.mark.parametrize("sizes", [[0, 1000, 0], [0, 0], [7] * 40 + [0] + [9] * 600])
def test_empty_gradients_into_another_type(M, sizes, out):
    gen = torch.Generator(device="cuda").manual_seed(3)
    grads = [torch.randn(n, generator=gen, device="cuda") for n in sizes]
    outs = [torch.full((n,), 9.0, dtype=out, device="cuda") for n in sizes]
    norm = norm_of(M, grads)
    M.mp_grad_clip(grads, norm, 0.5, out=outs)
    c = torch.tensor(min(1.0, 0.5 / (float(norm) + 1e-6)), dtype=F32, device="cuda")
    assert all(torch.equal(o, (g * c).to(out)) for g, o in zip(grads, outs))


@pytest.mark.parametrize("out", [F32, F16, BF16])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_clipped_bits(M, dtype, out):
    """The binary32 product of the gradient and the factor, then that rounded to the type written."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    grads = [(torch.randn(n, generator=gen, device="cuda") * 2.0**-6).to(dtype) for n in (1 << 20, 16391, 3)]
    outs = [torch.empty(g.numel(), dtype=out, device="cuda") for g in grads]
    norm = norm_of(M, grads)
    M.mp_grad_clip(grads, norm, 0.7, out=outs)
    most = float(torch.tensor(0.7))  # a C float
    c = torch.tensor(min(1.0, most / (float(norm) + 1e-6)), dtype=F32, device="cuda")
    assert all(torch.equal(o, (g.float() * c).to(out)) for g, o in zip(grads, outs))


def test_a_norm_beyond_binary32(M):
    """Finite FP32 gradients whose norm is not: infinity, and NaN for every clipped gradient."""
    grads = [torch.full((5000,), 1e38, device="cuda"), torch.ones(3, dtype=BF16, device="cuda")]
    norm = norm_of(M, grads)
    assert float(norm) == math.inf
    M.mp_grad_clip(grads, norm, 1.0)
    assert all(g.isnan().all() for g in grads)
