"""bind_device against a runtime of two devices that exists only in the test
(tests/host/bind_device_check.cu; nvcc is needed, no GPU)."""
import os
import shutil
import subprocess
import tempfile

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")


@pytest.mark.skipif(not (os.path.exists(NVCC) or shutil.which("nvcc")), reason="nvcc not found")
def test_calls_run_on_their_streams_device():
    nvcc = NVCC if os.path.exists(NVCC) else shutil.which("nvcc")
    with tempfile.TemporaryDirectory() as d:
        exe = os.path.join(d, "bind_check")
        subprocess.check_call([nvcc, "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17",
                               "--expt-relaxed-constexpr", "-w", "-I", os.path.join(ROOT, "include"),
                               "-I", os.path.join(ROOT, "nested_bit_weight_b200", "csrc"),
                               os.path.join(ROOT, "tests", "host", "bind_device_check.cu"), "-o", exe], timeout=600)
        out = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0 and "bad=0" in out.stdout, out.stdout + out.stderr
