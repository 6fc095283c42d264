"""Settings that each device needs once (host code, compiled with the host compiler)."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gather_lora_matmul_amd", "csrc")
PROGRAM = r"""
#include <cstdio>
#include "per_device.h"
int main() {
  lora::PerDevice a, b;
  int calls = 0, result = 0;
  auto set = [&] { ++calls; return result; };
  auto expect = [&](lora::PerDevice& p, int device, int more) {
    const int before = calls, got = p.done(device, set);
    if (calls - before != more || got != (more ? result : 0)) {
      std::printf("device %d: %d calls, result %d\n", device, calls - before, got);
      return 1;
    }
    return 0;
  };
  int bad = 0;
  bad += expect(a, 0, 1) + expect(a, 0, 0);      // once on the first device
  bad += expect(a, 1, 1) + expect(a, 1, 0) + expect(a, 0, 0);   // and once on another
  bad += expect(b, 0, 1);                        // each setting for itself
  result = 7;                                    // what failed is tried again
  bad += expect(a, 63, 1) + expect(a, 63, 1);
  result = 0;
  bad += expect(a, 63, 1) + expect(a, 63, 0);
  bad += expect(a, 64, 1) + expect(a, 64, 1) + expect(a, -1, 1) + expect(a, -1, 1) + expect(a, 0, 0);
  return bad;
}
"""


def test_a_setting_is_made_once_on_each_device(tmp_path):
    gxx = shutil.which("g++") or shutil.which("c++")
    if gxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-Wall", "-Werror", "-I" + CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
