"""The row that an acceptance draws from (csrc/gdn_accept_row.hpp), built for
the host with loads that count: a draft's row is read only where something was
rejected, since behind a node without children there need be none."""

import shutil
import subprocess

import pytest

from gated_delta_rule_79_amd import build

SOURCE = r"""
#define __device__
#include "gdn_accept_row.hpp"
#include <stdio.h>

static float target[3] = {0.5f, 0.25f, 0.25f}, draft[3] = {0.25f, 0.5f, 0.25f};
static int reads;

struct watched {
  static float load(const void* p, int64_t i) {
    if (p == draft) ++reads;
    return static_cast<const float*>(p)[i];
  }
};

int main() {
  const double scale[2] = {1.0, 4.0};
  const int tried[2] = {1, 0};
  for (int with = 0; with < 2; ++with)
    for (int m = 0; m < 3; ++m) {
      const gdn::AcceptRow<watched> r{target, with ? draft : nullptr, m, scale, tried};
      reads = 0;
      printf("%d %d:", with, m);
      double w[4];
      r.take(0, 3, w);
      for (int x = 0; x < 4; ++x) printf(" %.17g", w[x]);
      printf(" reads %d two %d\n", reads, static_cast<int>(r.two()));
    }
}
"""


def test_a_draft_row_is_read_behind_a_rejection_only(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("g++ not found")
    src, exe = tmp_path / "row.cpp", tmp_path / "row"
    src.write_text(SOURCE)
    subprocess.run([cxx, "-O1", "-std=c++17", "-I", build.CSRC, str(src), "-o", str(exe)],
                   check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split("\n")
    # the target's row; less the draft's (or a one at the token), then that
    # times 4 less it again
    assert out[:6] == [
        "0 0: 0.5 0.25 0.25 0 reads 0 two 0",
        "0 1: 0.5 0 0.25 0 reads 0 two 0",
        "0 2: 1 0 1 0 reads 0 two 0",
        "1 0: 0.5 0.25 0.25 0 reads 0 two 0",
        "1 1: 0.25 0 0 0 reads 3 two 1",
        "1 2: 0.75 0 0 0 reads 3 two 1"]

