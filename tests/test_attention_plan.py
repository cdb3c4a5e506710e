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


def test_the_join_stays_within_a_rows_slots(run):
    # what an old workspace holds in place of a number of parts: an fp32 sum, a negative one, NaN, noise
    run(r"""
void test() {
  const int found[] = {0, 1, 5, 6, 7, 1 << 20, 0x4f3a1200, 0x7fffffff, -1, -7, static_cast<int>(0x80000000u),
                       static_cast<int>(0xc1200000u), 0x7fc00000};
  for (int most : {0, 1, 6, 4096})
    for (int count : found) {
      const int got = parts_within(count, most);
      check(got >= 0 && got <= most, "parts", got);
      if (count >= 0 && count <= most) check(got == count, "parts that were written", got);
    }
}""")
