"""The shared-memory limit of the kernels that need more than 48 KB, without a GPU: a small C++ program
over csrc/fp8q_internal.h with stand-ins for the CUDA runtime."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_launch_asks_for_its_limit(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("g++ not found")
    from dequantisation_fp8q_token_b200 import build
    cuda = os.path.join(os.path.dirname(os.path.dirname(build.nvcc())), "include")
    exe = str(tmp_path / "smem_limit_check")
    r = subprocess.run([cxx, "-std=c++17", "-O1", "-isystem", cuda, "-I", build.INCLUDE, "-I", build.CSRC,
                        os.path.join(ROOT, "tests", "smem_limit_check.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    assert r.stdout.startswith("ok: ")
