"""What a launch sets up once, it sets up once on every device of the process (csrc/per_device.h, plain
C++: no GPU; a fake of the call counts)."""
import os
import subprocess

from _util import ROOT

SRC = r"""
#include "per_device.h"
#include <cstdio>
int main() {
  ql::OncePerDevice once, other;
  int calls = 0;
  auto act = [&] { ++calls; return 0; };
  auto fail = [&] { ++calls; return 7; };
  if (once.run(0, 0, fail) != 7 || calls != 1) return 1;             // a failure is told, and tried again
  if (once.run(0, 0, act) != 0 || calls != 2) return 2;
  if (once.run(0, 0, fail) != 0 || calls != 2) return 3;             // done on device 0
  if (once.run(1, 0, act) != 0 || calls != 3) return 4;              // not yet on device 1
  if (once.run(1, 0, fail) != 0 || calls != 3) return 5;
  if (once.run(63, 0, act) != 0 || once.run(63, 0, fail) != 0 || calls != 4) return 6;
  if (other.run(0, 0, act) != 0 || calls != 5) return 7;             // another kernel's state
  for (int i = 0; i < 2; ++i)
    if (once.run(64, 0, act) != 0 || calls != 6 + i) return 8;       // past the 64th: at every call
  if (once.run(-1, 0, act) != 0 || calls != 8) return 9;
  return 0;
}
"""


def test_once_on_every_device(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(SRC)
    inc = os.path.join(ROOT, "skinny_gemm_dequant_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", inc, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0


def test_every_kernel_asks_per_device():
    """No launch keeps a flag of its own for the whole process."""
    csrc = os.path.join(ROOT, "skinny_gemm_dequant_gb300", "csrc")
    for name in os.listdir(csrc):
        if name.endswith(".cu"):
            for line in open(os.path.join(csrc, name)):
                if "raise_smem_limit(" in line:
                    assert "once" in line, (name, line)
