"""Integer arithmetic that the attention kernels share with the host (csrc/awq_attn.cuh), compiled into a
small host program: no GPU is needed."""
import os
import subprocess

import pytest

from w4a16_weight_only_gb300 import build

PROGRAM = r"""
#include <stdio.h>
#include "awq_attn.cuh"
using namespace awq::attn;
int failures = 0;
void check(bool ok, const char* what, long long got) {
  if (!ok) printf("%s: got %lld\n", what, got), ++failures;
}
BODY
int main() {
  test();
  return failures != 0;
}
"""


@pytest.fixture
def run(tmp_path):
    def run(body):
        src, exe = tmp_path / "t.cu", tmp_path / "t"
        src.write_text(PROGRAM.replace("BODY", body))
        subprocess.run([build.nvcc_path(), *build.NVCC_FLAGS, "-I" + build.CSRC, str(src), "-o", str(exe)], check=True)
        r = subprocess.run([str(exe)], capture_output=True, text=True)
        assert r.returncode == 0, r.stdout
    return run


def test_blocks_beyond_the_last_group_have_no_steps(run):
    # own keys outweigh a long prefix: one group takes all of its steps, and blocks stand by for 152
    run(r"""
void test() {
  const int total = 1 << 27, groups = 152;
  for (int per : {2, 883012, 14 << 20, total / 2, total}) {
    long long covered = 0;
    for (int g = 0; g < groups; ++g) {
      const int begin = tc_first_step(g, per, total), end = begin + per < total ? begin + per : total;
      check(begin >= 0 && begin <= total, "first step", begin);
      check(begin == total || begin == static_cast<long long>(g) * per, "steps of a group in front", begin);
      covered += end - begin;
    }
    const long long most = static_cast<long long>(groups) * per;
    check(covered == (most < total ? most : total), "steps of all groups", covered);
  }
}""")
