"""What the gated linear recurrence reports: the forward that its backward runs again, where it is given no saved
states, has the caller's status word (host side, CPU), and waits that run out are reported (GPU, no fault)."""
import os
import shutil
import subprocess

import pytest

from chunked_gated_delta_gdn_gb300 import build

AGAIN = r"""
#include <stdio.h>
#include "gdn_recurrence.h"
int main() {
  int status = 0, room = 0;
  float carries[4], state[4], y[4];
  gdn::RecurrenceArgs a{};
  a.dev_status = &status;
  a.initial_state = state;
  a.y = y;
  a.T = 7;
  const gdn::RecurrenceArgs f = gdn::carries_again(a, carries, &room);
  if (f.dev_status != &status) { puts("the status word is lost"); return 1; }
  if (f.carries != carries || f.workspace != &room || f.y || f.initial_state != state || f.T != 7 || f.final_state)
    { puts("not the call that the carries need"); return 1; }
  return 0;
}
"""


def test_the_forward_run_again_reports_to_the_caller(tmp_path):
    cxx = shutil.which("g++")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc_path()))), "include")
    if cxx is None or not os.path.exists(os.path.join(cuda, "cuda_runtime.h")):
        pytest.skip("no host compiler or no CUDA headers")
    src, exe = tmp_path / "again.cc", tmp_path / "again"
    src.write_text(AGAIN)
    subprocess.run([cxx, "-std=c++17", "-I", build.INCLUDE, "-I", build.CSRC, "-I", cuda, str(src), "-o", str(exe)],
                   check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True)
    assert got.returncode == 0, got.stdout
