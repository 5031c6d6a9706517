"""Kernels whose CTAs hold tensor memory while they wait for another CTA must not
share an SM (nvcc is needed; no GPU)."""
import ctypes
import os
import shutil
import subprocess
import tempfile

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
SM_SHARED, RESERVED = 228 * 1024, 1024              # of an SM; of each CTA beside what it asks for


@pytest.mark.skipif(not (os.path.exists(NVCC) or shutil.which("nvcc")), reason="nvcc not found")
def test_no_cluster_of_the_nested_gemv_fits_beside_a_pair():
    from tests.test_gpu_timeout import _hooks_lib
    L = _hooks_lib()
    L.mq_test_mx4_pair_smem.restype = ctypes.c_size_t
    nvcc = NVCC if os.path.exists(NVCC) else shutil.which("nvcc")
    with tempfile.TemporaryDirectory() as d:
        exe = os.path.join(d, "least")
        subprocess.check_call([nvcc, "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17",
                               "--expt-relaxed-constexpr", "-w", "-I", os.path.join(ROOT, "include"),
                               "-I", os.path.join(ROOT, "nested_bit_weight_b200", "csrc"),
                               os.path.join(ROOT, "tests", "host", "gemv_least_smem.cu"), "-o", exe], timeout=600)
        out = subprocess.run([exe], capture_output=True, text=True, timeout=300).stdout
    least = int(out.split("least=")[1])
    pair = L.mq_test_mx4_pair_smem()
    assert least < 1 << 20 and pair + RESERVED + least + RESERVED > SM_SHARED, (pair, least)
    assert pair <= 227 * 1024
