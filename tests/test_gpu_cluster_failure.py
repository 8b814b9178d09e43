"""A wait that gives up in one CTA of a cluster is seen in the sums of all of them: nothing finite comes of
sums which are not complete.  The probe kernel (tests/cluster_probe.cu) uses the library's own routines."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import mixed_precision_numerics_gb300 as M

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def library(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    out = tmp_path_factory.mktemp("probe") / "libclusterprobe.so"
    r = subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-O2", "-std=c++17", "-shared",
                        "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "mixed_precision_numerics_gb300", "csrc"),
                        os.path.join(ROOT, "tests", "cluster_probe.cu"), "-o", str(out)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return str(out)


def test_the_probe_builds(library):
    assert os.path.exists(library)


@pytest.mark.gpu
@pytest.mark.parametrize("silent", [-1, 0, 3])
def test_every_sum_shows_it(library, cuda_ok, silent):
    L = ctypes.CDLL(library)
    L.cluster_probe.argtypes = [ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]
    sums = torch.full((4,), 7.0, device="cuda")
    assert L.cluster_probe(silent, sums.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert (sums == 10.0).all() if silent < 0 else sums.isnan().all()
    # the context runs library work as before
    x = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda")
    w, p = torch.ones(32, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(4, 32, dtype=torch.bfloat16, device="cuda")
    M.linear_swiglu(x, w, w, p)
    assert (p == 4096.0).all()
    assert M.mp_wait_failures() == 0  # the probe is not one of the library's kernels
