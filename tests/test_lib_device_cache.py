"""CPU-only: the numbers that the launches ask of a device are kept per device, and a query that failed
is asked again (csrc/device_cache.h, compiled with the host's compiler)."""
import os
import shutil
import subprocess

import pytest

from grouped_gemm_device_gb300 import build as gbuild

PROGRAM = r"""
#include <cstdio>
#include <initializer_list>
#include "device_cache.h"
#define CHECK(x) if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; }
int main() {
  static moe::DeviceCache cache;
  int asked = 0;
  auto answer = [&](int n) { return [&asked, n] { ++asked; return n; }; };
  CHECK(cache.get(0, answer(0)) == 0 && asked == 1);   // failed
  CHECK(cache.get(0, answer(19)) == 19 && asked == 2); // asked again
  CHECK(cache.get(0, answer(7)) == 19 && asked == 2);  // kept
  CHECK(cache.get(1, answer(7)) == 7 && asked == 3);   // another device
  CHECK(cache.get(0, answer(5)) == 19 && cache.get(1, answer(5)) == 7 && asked == 3);
  for (int dev : {-1, 64, 1000}) {                     // not kept, but answered
    CHECK(cache.get(dev, answer(3)) == 3 && cache.get(dev, answer(4)) == 4);
  }
  return 0;
}
"""


def test_kept_for_each_device_and_asked_again_after_a_failure(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    src, exe = tmp_path / "cache.cpp", tmp_path / "cache"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Werror", "-I" + gbuild.CSRC, str(src), "-o",
                    str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_launches_ask_through_it():
    """No function-static answer to an occupancy query outside the shared ones of api.cu."""
    for name in ("layernorm.cu", "grad_clip.cu", "gemm_fp8.cu"):
        with open(os.path.join(gbuild.CSRC, name)) as f:
            text = f.read()
        assert "DeviceCache" in text and "static const int" not in text, name
