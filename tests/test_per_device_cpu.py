"""The opt-in of kernels to more shared memory is made on every device that is
used, and again where it failed (no GPU: the header alone, with a fake call)."""
import os
import re
import subprocess

import pytest

from tests.conftest import ROOT

CSRC = os.path.join(ROOT, "exact_top_sparse_gb300", "csrc")

PROGRAM = r"""
#include "per_device.h"
#include <cstdio>
int main() {
  OncePerDevice once;
  int calls[80] = {0};
  bool fail = true;
  auto on = [&](int d) { return once.ensure(d, [&] { ++calls[d]; return !fail; }); };
  std::printf("%d%d ", on(3), on(3));          // failures are not kept
  fail = false;
  std::printf("%d%d%d ", on(3), on(3), on(0)); // once per device
  std::printf("%d%d ", on(63), on(0));
  std::printf("%d%d ", on(70), on(70));        // beyond the mask: every time
  std::printf("%d %d %d %d\n", calls[0], calls[3], calls[63], calls[70]);
}
"""


def test_once_per_device(tmp_path):
    src, exe = str(tmp_path / "once.cpp"), str(tmp_path / "once")
    with open(src, "w") as f:
        f.write(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, src, "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout
    assert out.split() == ["00", "111", "11", "11", "1", "3", "1", "2"]


@pytest.mark.parametrize("name", ["sparse_attend.cu", "sparse_attend_grad.cu", "index_scores.cu"])
def test_launches_opt_in_per_device(name):
    """A function's attribute belongs to one device: not behind a flag of the process."""
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    assert "cudaFuncSetAttribute" in text
    for m in re.finditer("cudaFuncSetAttribute", text):
        before = text[:m.start()]
        assert before.rfind("opted_in.ensure(dev") > max(before.rfind("call_once"), before.rfind("\n}\n"))
