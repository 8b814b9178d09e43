"""Rows of gate and up, and of their gradients, 2^31 and more elements apart."""
import pytest
import torch

import tests.test_gpu_block_ops as B

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    yield


@pytest.mark.parametrize("pitch", [2**31 - 8, 2**31, 2**31 + 8, 2**32 + 64])
def test_rows_far_apart(pitch):
    rows, cols = 2, 272
    wide = torch.empty(pitch + 4 * cols, dtype=torch.float16, device="cuda")

    def matrix(at):
        return wide.as_strided((rows, cols), (pitch, 1), at)

    g, u = matrix(0), matrix(cols)
    dense = [B.normal(1 + k, rows, cols, dtype=torch.float16) for k in range(3)]
    g.copy_(dense[0])
    u.copy_(dense[1])
    want, got = B.swiglu(*dense[:2]), B.swiglu(g, u)
    for k in want:
        B.assert_bits(got[k], want[k], k)
    dg, du = matrix(2 * cols), matrix(3 * cols)
    want = B.swiglu_backward(dense[2], gate=dense[0], up=dense[1])
    B.M.swiglu_backward(dense[2], dg, du, gate=g, up=u)
    B.assert_bits(dg, want[0], "dgate")
    B.assert_bits(du, want[1], "dup")
    B.assert_bits(g, dense[0], "gate")
    B.assert_bits(u, dense[1], "up")
