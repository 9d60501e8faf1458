"""What the library does once per device (a kernel's shared-memory limit): once for each, again
after a failure, and never one flag for the whole process."""
import os
import re
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "post_weight_quantization_gb300", "csrc")

MAIN = r"""
#include <cstdio>
#include "per_device.h"
int main() {
  static gptq::PerDevice d;
  int calls[64] = {0};
  bool fail = true;
  auto go = [&](int dev) { return d.once(dev, [&] { ++calls[dev]; return !fail; }); };
  const bool first = go(0);
  fail = false;
  const bool rest = go(0) && go(0) && go(1) && go(63) && go(1) && go(63) && go(0);
  std::printf("%d %d %d %d %d\n", first, rest, calls[0], calls[1], calls[63]);
}
"""


def test_once_per_device(tmp_path):
    cxx = os.environ.get("CXX") or shutil.which("g++")
    if not cxx:
        pytest.skip("no C++ compiler")
    (tmp_path / "main.cpp").write_text(MAIN)
    subprocess.run([cxx, "-std=c++17", "-I", CSRC, str(tmp_path / "main.cpp"), "-o", str(tmp_path / "main")], check=True)
    assert subprocess.run([str(tmp_path / "main")], capture_output=True, text=True).stdout.split() == ["0", "1", "2", "1", "1"]


def test_shared_memory_limits_are_set_per_device():
    """Every remembered cudaFuncSetAttribute goes through the helper."""
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        assert not re.search(r"static\s+(std::atomic<bool>|bool)\s+\w*(attr|done|set)\w*", text), name
