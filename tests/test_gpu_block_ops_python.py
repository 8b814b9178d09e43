"""The block operators' calls through the Python marshalling alone: the same checks and refusals, the same results."""
import os

import pytest

import __graft_entry__
import tests.test_gpu_block_ops as B

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    yield


def test_the_native_marshalling_is_the_one_in_use():
    build = __graft_entry__._package_builder()
    assert os.path.exists(build.PYTHON_H) == (B.M._mpcall is not None)


@pytest.mark.parametrize("check", [
    lambda: B.test_refusals_launch_nothing(),
    lambda: B.test_norm_forward((33, 128), "bf16", 128),
    lambda: B.test_norm_forward((5, 160), "f32", 32),
    lambda: B.test_norm_weight_types_and_optional_outputs("f16", "bf16"),
    lambda: B.test_norm_writes_the_stream_over_its_input(),
    lambda: B.test_norm_backward((40, 1040), "f16", True),
    lambda: B.test_norm_backward((40, 1040), "f32", False),
    lambda: B.test_norm_backward_of_no_rows_and_of_nonfinite_rows(),
    lambda: B.test_swiglu_forward((37, 160), "bf16", 32),
    lambda: B.test_swiglu_backward((37, 160), "bf16", True),
    lambda: B.test_swiglu_backward((37, 160), "f32", False),
    lambda: B.test_swiglu_backward_in_place(),
    lambda: B.test_calls_on_another_stream_and_in_a_graph(),
    lambda: B.test_pointers_aligned_to_16_bytes_only((9, 48)),
])
def test_without_the_native_marshalling(check, monkeypatch):
    monkeypatch.setattr(B.M, "_mpcall", None)
    check()
