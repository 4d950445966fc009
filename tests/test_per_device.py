"""A kernel's set-up is done on each device that it is launched on, not once for
the process: the attributes of a kernel are a device's own.  Plain C++, no GPU."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "rns_emulated_fp64_gb300", "csrc")

MAIN = r"""
#include <cassert>
#include <thread>
#include <vector>
#include "per_device.h"
enum Status { ok = 0, no = 7 };
int main() {
  static PerDevice ready;
  int calls = 0;
  auto set_up = [&] { calls++; return ok; };
  for (int turn = 0; turn < 3; turn++)
    for (int dev = 0; dev < 8; dev++) assert(ready(dev, set_up) == ok);
  assert(calls == 8);                       // each device once
  PerDevice other;                          // a failure is told, and tried again
  assert(other(1, [&] { calls++; return no; }) == no && calls == 9);
  assert(other(1, set_up) == ok && other(1, set_up) == ok && calls == 10);
  assert(other(99, set_up) == ok && other(99, set_up) == ok && calls == 12);  // past the table: each time
  PerDevice shared;
  std::atomic<int> seen{0};
  std::vector<std::thread> ts;
  for (int i = 0; i < 16; i++)
    ts.emplace_back([&, i] { for (int j = 0; j < 1000; j++) shared(i % 4, [&] { seen++; return ok; }); });
  for (auto &t : ts) t.join();
  assert(seen == 4);
}
"""


@pytest.mark.skipif(not shutil.which(os.environ.get("CXX") or "g++"), reason="no C++ compiler")
def test_each_device_is_set_up_once(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(MAIN)
    subprocess.run([os.environ.get("CXX") or "g++", "-std=c++17", "-pthread", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    subprocess.run([str(exe)], check=True)


def test_no_kernel_is_set_up_once_for_the_process():
    """cudaFuncSetAttribute is called by the function that keeps count by device, or at every launch."""
    for name in sorted(os.listdir(CSRC)):
        text = open(os.path.join(CSRC, name)).read()
        for m in re.finditer(r"cudaFuncSetAttribute\(", text):
            before = text[max(0, m.start() - 200):m.start()]
            assert "static" not in before.split("{")[-1] and "call_once" not in before, name
