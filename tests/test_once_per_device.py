"""Kernel attributes belong to a device: they are set on each device that a process uses, and again after a failure."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_weight_quantized_matmul_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "wq_once.h"
int main() {
  std::atomic<uint64_t> done{0};
  int runs = 0;
  bool works = true;
  auto set = [&] { ++runs; return works; };
  auto step = [&](int device) { const bool ok = wq::once_per_device(done, device, set); std::printf("%d%d ", ok, runs); };
  step(0); step(0); step(1); step(0); step(1);       // each device once
  works = false;
  step(0); step(2); step(2);                         // a device that worked before still does; a failure is tried again
  works = true;
  step(2); step(2); step(63); step(63); step(64); step(64);
}
"""


def test_each_device_once_and_failures_again(tmp_path):
    cc = shutil.which("g++") or pytest.skip("no C++ compiler")
    (tmp_path / "main.cpp").write_text(PROGRAM)
    exe = str(tmp_path / "main")
    subprocess.run([cc, "-std=c++17", "-I", CSRC, str(tmp_path / "main.cpp"), "-o", exe], check=True)
    out = subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split()
    assert out == ["11", "11", "12", "12", "12", "12", "03", "04", "15", "15", "16", "16", "17", "18"]


def test_attention_sets_no_attribute_once_for_all_devices():
    """Every cudaFuncSetAttribute of the attention kernels, and of the helper they share, stands inside a once_per_device."""
    for name in ("wq_attend.cu", "wq_attend_tc.cu", "wq_internal.h"):
        text = open(os.path.join(CSRC, name)).read()
        for m in re.finditer(r"cudaFuncSetAttribute\(", text):
            assert "once_per_device(" in text[max(0, m.start() - 250):m.start()], (name, text[m.start():m.start() + 80])
    assert "cudaFuncSetAttribute" in text
