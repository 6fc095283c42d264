"""Kernels whose waves share LDS, run on the host with their waves in both orders (CPU only).

tests/native/blocks/hip/hip_runtime.h stands in for the runtime's header: the kernels'
sources as they are, every thread a context of its own.  What is read behind the last
barrier and written by another wave before the next one gives other results in one of
the orders, or threads that wait at different barriers."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gather_lora_matmul_amd", "csrc")
NATIVE = os.path.join(ROOT, "tests", "native")
CXX = "/opt/rocm/llvm/bin/clang++"     # (vector types of the kernels' sources)


def run(tmp_path, name):
    if not os.path.exists(CXX):
        pytest.skip("no clang++")
    exe = str(tmp_path / name)
    subprocess.run([CXX, "-std=c++17", "-O2", "-w", "-I" + os.path.join(NATIVE, "blocks"), "-I" + CSRC, "-x", "c++",
                    os.path.join(NATIVE, name + ".cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    print(r.stdout)


def test_selection_does_not_depend_on_the_order_of_waves(tmp_path):
    run(tmp_path, "select_check")
