"""The dense products' plans (csrc/dense_plan.h) at the largest sizes that the entry points take: no integer
overflows on the way, and each shape has a slot to be kept in."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROBE = r"""
#include <stdio.h>
#include "dense_plan.h"
using namespace moe;
int main() {
  const DenseDevice d = {152, 76, {{0, 152, 152, 138, 144, 140, 138, 105, 120}, {0, 304, 304, 276, 288, 280, 276, 210, 240}}};
  const long long T = 1 << 24, M = 1 << 20;
  long used[kPlanSlots] = {}, shapes = 0;
  for (long long I : {1LL, 513LL, M, T - 1, T})
    for (long long J : {1LL, 4097LL, M - 1, M})
      for (long long K : {8LL, 2048LL, M, T})
        for (int form = 0; form < 16; ++form) {
          const DenseShape s = {I, J, K, (form & 1) != 0, false, (form & 2) != 0, (form & 4) != 0, (form & 8) != 0};
          const int slot = plan_slot(s);
          if (slot < 0 || slot >= kPlanSlots || !same_shape(s, s)) return 1;
          ++used[slot], ++shapes;
          if (form % 5 == 0) dense_plan(s, d);
          const DenseShape b[2] = {{I, K, J, false, false, false, false, true}, {J, K, I, false, true, false, false, true}};
          DensePlan p[2];
          if (form == 0) dense_plan_both(b, d, p);
        }
  int filled = 0;
  for (long n : used) filled += n > 0;
  printf("%ld %d\n", shapes, filled);
  return filled < kPlanSlots / 2;
}
"""


def test_the_largest_sizes(tmp_path):
    src, exe = tmp_path / "probe.cpp", tmp_path / "probe"
    src.write_text(PROBE)
    # an overflow of a signed integer ends the program
    subprocess.run(["g++", "-O1", "-std=c++17", "-fsanitize=signed-integer-overflow", "-fsanitize-undefined-trap-on-error",
                    "-I", os.path.join(ROOT, "combine_counting_sort_gb300", "csrc"), str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stdout)
