"""What a launcher finds out once per device, on the host: kept by device, asked
again after a failure, and the same for threads that come together."""

import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "unpermute_moe_permute_gb300", "csrc")

PROGRAM = r"""
#include <stdio.h>
#include <thread>
#include <vector>
#include "per_device.h"
#define CHECK(x) do { if (!(x)) { printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)
int main() {
  static moe::PerDevice p;
  int calls = 0;
  auto make = [&](int v) { return [&calls, v] { ++calls; return v; }; };
  CHECK(p.get(0, make(10)) == 10 && calls == 1);
  CHECK(p.get(0, make(99)) == 10 && calls == 1);
  CHECK(p.get(1, make(11)) == 11 && calls == 2);   // another device finds out for itself
  CHECK(p.get(2, make(-1)) == -1 && p.get(2, make(0)) == 0 && calls == 4);
  CHECK(p.get(2, make(12)) == 12 && p.get(2, make(99)) == 12 && calls == 5);
  CHECK(p.get(64, make(7)) == 7 && p.get(64, make(8)) == 8 && p.get(-1, make(9)) == 9);
  std::vector<std::thread> t;
  std::atomic<int> wrong{0};
  for (int i = 0; i < 8; ++i)
    t.emplace_back([&] {
      for (int k = 0; k < 10000; ++k) wrong += p.get(3 + k % 50, [k] { return 100 + k % 50; }) != 100 + k % 50;
    });
  for (auto& x : t) x.join();
  CHECK(wrong == 0);
  return 0;
}
"""


def test_per_device(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    (tmp_path / "t.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-pthread", "-I", CSRC, "t.cpp", "-o", "t"], cwd=tmp_path, check=True)
    res = subprocess.run([str(tmp_path / "t")], capture_output=True, text=True, timeout=60)
    assert res.returncode == 0, res.stdout


@pytest.mark.parametrize("name", ["gmm_i8.cu", "few_tokens.cu"])
def test_launchers_set_up_each_device(name):
    """A kernel's shared-memory limit belongs to a device: no flag of the process guards it."""
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    assert "cudaFuncSetAttribute" in text and "once_flag" not in text and "static int resident" not in text
