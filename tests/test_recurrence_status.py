"""What the gated linear recurrence reports: the forward that its backward runs again, where it is given no saved
states, has the caller's status word (host side, CPU), and waits that run out are reported (GPU, no fault)."""
import os
import shutil
import subprocess

import pytest

from chunked_gated_delta_gdn_gb300 import _lib, build

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


def test_waits_selftest_validates_on_the_host():
    L = _lib.load()
    assert L.gdn_selftest_recurrence_wait(None, 10, 0, None, None) == _lib.GDN_ERR_NULL
    assert L.gdn_selftest_recurrence_wait(1 << 20, 10, 0, None, None) == _lib.GDN_ERR_NULL
    for tries in (0, -1, 10001):
        assert L.gdn_selftest_recurrence_wait(1 << 20, tries, 0, 1 << 20, None) == _lib.GDN_ERR_SHAPE


def waits(tries, arrive_first):
    """(status bits, nanoseconds of the four waits and the tries of the kernels' own)."""
    torch = pytest.importorskip("torch")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    waited = torch.zeros(5, dtype=torch.int64, device="cuda")
    rc = _lib.load().gdn_selftest_recurrence_wait(status.data_ptr(), tries, arrive_first, waited.data_ptr(),
                                                  torch.cuda.current_stream().cuda_stream)
    assert rc == _lib.GDN_OK, _lib.status_string(rc)
    torch.cuda.synchronize()
    return status.item(), waited.tolist()


@pytest.mark.gpu
def test_waits_that_run_out_are_reported_once():
    """The time goes with the tries; the second wait of a kind does not wait, and the copies' one gives those under
    way their time as well."""
    few, many = waits(10, 0), waits(1000, 0)
    print("10 tries %s ns, 1000 tries %s ns" % (few[1], many[1]))
    for bits, waited in (few, many):
        assert bits == _lib.GDN_DEV_TIMEOUT
    first, again, copies, none, _ = many[1]
    assert 0 < first < 1e9 and again < first / 10 and none < first / 10 and copies > 1.5 * first
    assert many[1][0] > 5 * few[1][0]


@pytest.mark.gpu
def test_waits_for_what_has_come_report_nothing():
    bits, waited = waits(1000, 1)
    assert bits == 0 and max(waited[:4]) < 1e6


@pytest.mark.gpu
def test_the_kernels_waits_end_within_seconds():
    _, waited = waits(1000, 0)
    limit = waited[0] / 1000 * waited[4] * 1e-9
    print("a wait of the kernels ends after %.2f s" % limit)
    assert 0.2 < limit < 5
