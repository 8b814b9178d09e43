"""The row distances that the SwiGLU calls take, shown without a GPU by what a call refuses next."""
import pytest

import mixed_precision_numerics_gb300 as M
from tests.test_block_ops_host import A, swiglu, swiglu_bwd


@pytest.mark.parametrize("ld", [2**62, 2**63 - 8])
def test_distances_whose_offsets_pass_64_bits_are_refused(ld):
    assert swiglu(ld=ld) == M.MP_ESHAPE
    assert swiglu_bwd(ld=ld) == M.MP_ESHAPE
    assert swiglu_bwd(d_ld=ld) == M.MP_ESHAPE


@pytest.mark.parametrize("ld", [2**31, 2**31 + 8, 2**40])
def test_distances_above_32_bits_are_taken(ld):
    """A misaligned output is refused after the distance has passed."""
    assert swiglu(ld=ld, y=A + 8) == M.MP_EALIGN
    assert swiglu_bwd(ld=ld, dp=A + 8) == M.MP_EALIGN
    assert swiglu_bwd(d_ld=ld, dp=A + 8) == M.MP_EALIGN
    assert swiglu_bwd(gate=None, up=None, ckpt=A, ckpt_scales=A, d_ld=ld, dp=A + 8) == M.MP_EALIGN
