"""Lists with empty gradients: nothing of them is read or written, so their pointers have no part in the checks."""
import pytest

import mixed_precision_numerics_gb300 as M

A = 4096


def clip(*entries):
    arr = (M.MpGrad * len(entries))(*(M.MpGrad(*e) for e in entries))
    return M.lib.mp_grad_clip(arr, len(entries), A, 1.0, None)


@pytest.mark.parametrize("grad,out", [(None, None), (A, A), (A, 2 * A), (A + 2, A + 6), (None, A + 2)])
@pytest.mark.parametrize("types", [(M.MP_F32, M.MP_F16), (M.MP_F32, M.MP_F32), (M.MP_BF16, M.MP_F32)])
def test_an_empty_gradient_is_taken_with_any_pointers(grad, out, types):
    n0 = M.mp_launch_count()
    assert clip((grad, out, 0, *types)) == M.MP_OK
    assert clip((None, None, 0, M.MP_F32, M.MP_BF16), (grad, out, 0, *types)) == M.MP_OK
    assert M.mp_launch_count() == n0


@pytest.mark.parametrize("entry,status", [
    ((None, None, 0, M.MP_E4M3, M.MP_F32), M.MP_EINVAL), ((None, None, 0, M.MP_F32, 7), M.MP_EINVAL),
    ((None, None, -1, M.MP_F32, M.MP_F32), M.MP_EINVAL), ((A, A, 1, M.MP_F32, M.MP_F16), M.MP_EINVAL),
    ((None, A, 1, M.MP_F32, M.MP_F32), M.MP_EINVAL), ((A, None, 1, M.MP_F32, M.MP_F32), M.MP_EINVAL),
    ((A + 8, A, 1, M.MP_F32, M.MP_F32), M.MP_EALIGN), ((A, A + 8, 1, M.MP_F32, M.MP_F32), M.MP_EALIGN),
])
def test_refusals_beside_an_empty_gradient(entry, status):
    n0 = M.mp_launch_count()
    assert clip((None, None, 0, M.MP_F32, M.MP_F16), entry) == status and M.mp_launch_count() == n0
