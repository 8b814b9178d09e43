"""The feed-forward training example runs on the library's calls and learns."""
import importlib.util
import os

import pytest

from tests.conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    yield


def test_fp8_mlp_blocks_learn():
    spec = importlib.util.spec_from_file_location("fp8_mlp_blocks", os.path.join(ROOT, "examples", "fp8_mlp_blocks.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    losses = ex.train(steps=60, tokens=1000, blocks=2, log=None)
    assert all(v == v for v in losses)
    assert sum(losses[-5:]) < 0.5 * sum(losses[:5])
