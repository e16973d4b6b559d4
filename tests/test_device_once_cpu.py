"""Kernel attributes are set once for every device, not once a process. The
bookkeeping is plain C++ and runs here without a GPU."""
import glob
import os
import re
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "speculative_verify_paged_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "device_once.cuh"
int main() {
  sv::DeviceOnce once;
  int calls[100] = {};
  auto set = [&](int dev, int err) { return once.run<int>(dev, [&] { ++calls[dev]; return err; }); };
  if (set(0, 7) != 7 || calls[0] != 1) return 1;          // a failure is returned and tried again
  if (set(0, 0) != 0 || calls[0] != 2) return 2;
  if (set(0, 9) != 0 || calls[0] != 2) return 3;          // done: not run again
  if (set(1, 0) != 0 || calls[1] != 1) return 4;          // another device has its own
  if (set(63, 0) != 0 || set(63, 0) != 0 || calls[63] != 1) return 5;
  if (set(64, 0) != 0 || calls[64] != 1) return 6;        // not taken for device 0
  if (set(64, 3) != 3 || calls[64] != 2) return 7;
  std::vector<std::thread> ts;
  std::atomic<int> runs{0};
  for (int t = 0; t < 8; ++t)
    ts.emplace_back([&] { for (int d = 2; d < 60; ++d) once.run<int>(d, [&] { ++runs; return 0; }); });
  for (auto &t : ts) t.join();
  if (runs < 58) return 8;
  const int before = runs;
  for (int d = 2; d < 60; ++d) once.run<int>(d, [&] { ++runs; return 0; });
  return runs == before ? 0 : 9;
}
"""


def test_once_a_device(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-pthread", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.cu"))), ids=os.path.basename)
def test_attributes_are_set_a_device_at_a_time(path):
    with open(path) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    for m in re.finditer(r"call_once\(", text):
        lambda_end = text.index("});", m.start())
        assert "cudaFuncSetAttribute" not in text[m.start():lambda_end]
