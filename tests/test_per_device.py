"""The table of numbers asked for once a device (csrc/per_device.h), compiled for the host."""
import os
import shutil
import subprocess

import pytest

import nvfp4_weight_only_top_b200 as moe

_PROGRAM = """
#include <cstdio>
#include "per_device.h"
int main() {
  static moe::PerDevice t;
  int asked = 0, answer = 0;
  const auto ask = [&](int dev) { return t.get(dev, [&] { ++asked; return answer; }); };
  if (ask(0) != 0 || ask(0) != 0 || asked != 2) return 1;          // a failure is not kept
  answer = 66;
  if (ask(0) != 66 || asked != 3) return 2;
  answer = 60;
  if (ask(0) != 66 || asked != 3) return 3;                        // an answer is
  if (ask(1) != 60 || ask(1) != 60 || asked != 4) return 4;        // another device has its own
  if (ask(63) != 60 || ask(64) != 60 || ask(64) != 60 || ask(-1) != 60 || asked != 8) return 5;
  answer = 5;
  if (ask(0) != 66 || ask(1) != 60 || ask(64) != 5) return 6;
  std::puts("same");
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_answers_are_kept_by_device_and_failures_are_not(tmp_path):
    csrc = os.path.join(os.path.dirname(moe.__file__), "csrc")
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(_PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", csrc, "-o", str(exe), str(src)], check=True)
    p = subprocess.run([str(exe)], capture_output=True, text=True)
    assert p.returncode == 0 and p.stdout == "same\n"
