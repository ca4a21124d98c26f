"""A kernel's shared-memory limit only grows, whichever of two host threads comes
last (tests/smem_limit.cu; no GPU)."""
import os
import subprocess

import pytest

from block_quantized_matmul_gguf_gb300 import build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_threads_leave_the_larger_limit(tmp_path):
    try:
        nvcc = build.nvcc_path()
    except RuntimeError:
        pytest.skip("nvcc not available")
    exe = str(tmp_path / "smem_limit")
    subprocess.run([nvcc, "-std=c++17", "--expt-relaxed-constexpr", "-I", build.INCLUDE, "-I", build.CSRC, "-o", exe,
                    os.path.join(HERE, "smem_limit.cu"), "-lpthread"], check=True, capture_output=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
