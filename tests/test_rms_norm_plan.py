"""Host arithmetic of the norm's backward launches, without a GPU: small C++ programs over the
header that the kernel's host side takes its launches from (csrc/rms_norm_plan.h)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "dequantisation_fp8q_token_b200", "csrc")


def run_program(name, tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("g++ not found")
    exe = str(tmp_path / name)
    r = subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-I", CSRC,
                        os.path.join(ROOT, "tests", name + ".cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout


def test_every_backward_launch_has_room_for_a_row(tmp_path):
    assert run_program("rms_norm_plan_check", tmp_path).startswith("ok: ")


def test_no_copy_of_the_backward_pass_leaves_its_tensor(tmp_path):
    assert run_program("rms_norm_copy_check", tmp_path).startswith("ok: ")
