"""The decoding kernels' divisions of shared memory and registers (csrc/few_plan.h)."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROBE = r"""
#include <stdio.h>
#include "few_plan.h"
using namespace moe;
// every batch, number of pairs, form and fullest segment: one line for each that has fewer than two
// stages or leaves the block's shared memory, and the counts
int main() {
  long calls = 0, fewer = 0, two_slices = 0;
  int fewer_least = 1 << 30;
  const int groups[4] = {0, 32, 64, 128};
  for (int g : groups)
    for (int rt2 = 1; rt2 <= 3; ++rt2)
      for (int T = 1; T <= 64; ++T)
        for (int k = 1; k <= 32 && T * k <= 1024; ++k) {
          const bool direct = T <= 8;
          const int P = T * k, cols = layer_cols(g, rt2, direct, T, P, kFewMinSmem);
          if (cols < kLayerCols) {
            ++fewer;
            if (P < fewer_least) fewer_least = P;
            if (cols < 15 || g != 0 || rt2 != 3) printf("narrow %d %d %d %d: %d\n", g, rt2, T, k, cols);
          }
          for (int cap = 1; cap <= (T < cols ? T : cols); ++cap) {
            const int sp = layer_slices(g, rt2, direct, T, P, cap, kFewMinSmem);
            const LayerRoom r = layer_room(g, sp, rt2, direct, T, P, cap, kFewMinSmem);
            const int gate_up = 2 * layer_pairs(g, sp, direct), rt = rt2 > gate_up ? rt2 : gate_up;
            const uint32_t weights = rt * 8 * sp * (g ? 1024 + 4096 / g : 2048), records = cap * (8 * sp * kTokenRecord + 64);
            const uint32_t ring = (few_tables_end(P) + r.sums + r.out + 1023) / 1024 * 1024;
            const bool fits = r.stage >= weights + records + (g ? 0 : 32 * rt) && ring + r.stages * r.stage <= kFewMinSmem &&
                              r.sums >= r.bufs * r.buf && r.buf >= (uint32_t)(8 * (direct ? 2 : rt2) * cap * kFewColPitch * 4) &&
                              (!direct || r.sums >= (uint32_t)(8 * rt2 * T * kFewColPitch * 4)) && few_tables_end(P) >= kTablesAt + 21 * P;
            if (r.stages < 2 || !fits) printf("call %d %d %d %d cap %d: %d stages, fits %d\n", g, rt2, T, k, cap, r.stages, (int)fits);
            ++calls;
            two_slices += sp == 2;
          }
        }
  printf("counts %ld %ld %d %ld\n", calls, fewer, fewer_least, two_slices);
  return 0;
}
"""


def run(tmp_path, text):
    src, exe = tmp_path / "probe.cpp", tmp_path / "probe"
    src.write_text(text)
    csrc = os.path.join(ROOT, "combine_counting_sort_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", csrc, str(src), "-o", str(exe)], check=True)
    return subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines()


def test_every_call_leaves_the_ring_two_stages(tmp_path):
    lines = run(tmp_path, PROBE)
    assert len(lines) == 1, lines[:20]
    calls, fewer, least, two_slices = (int(v) for v in lines[0].split()[1:])
    assert calls > 100000 and two_slices > 10000
    # segments of 15 tokens for FP8 with three row tiles and many pairs alone
    assert fewer > 0 and least > 800


def test_a_kernel_with_too_few_registers_for_the_split_is_refused(tmp_path):
    # 16 x 56 + 8 x 120 + 4 x 40 warps x registers = 28 x 72
    text = """
#include <stdio.h>
#include "few_plan.h"
int main() { for (int r = 24; r <= 72; ++r) if (moe::tensor_split_fits(r)) printf("%d\\n", r); }
"""
    assert run(tmp_path, text) == ["72"]
    # and the launch asks before it launches
    launch = open(os.path.join(ROOT, "combine_counting_sort_gb300", "csrc", "few_tensor.cuh")).read()
    assert launch.count("few_launch(matvec_tensor_kernel") == 1 and launch.index("if (!split_ok) return") < launch.index("few_launch(matvec_tensor_kernel")


def test_the_tensor_kernels_ring_has_the_stages_that_its_waits_need(tmp_path):
    # a model of the widening warps' waits: a wait by parity is safe only if the slot's fill before
    # the one waited for is known to be complete, and what a set knows is that slices up to i - 4
    # are done (its A buffer's last use) and its own i - 2 and before
    text = """
#include <stdio.h>
#include "few_plan.h"
int main() {
  for (int g = 32; g <= 128; g *= 2)
    for (int n = 16; n <= 64; n += 16) printf("%d\\n", moe::tensor_stages(g, n, moe::kFewMinSmem));
  printf("%d\\n", moe::kTensorMinStages);
}
"""
    *stages, least = (int(v) for v in run(tmp_path, text))

    def safe(count):
        known = lambda i: {j for j in range(i) if j <= i - 4 or (i - j) % 2 == 0}   # noqa: E731
        return all(i - count < 0 or i - count in known(i) for i in range(40))

    assert all(safe(s) for s in range(least, 13)) and not safe(3)
    assert len(stages) == 12 and min(stages) >= least and any(s % 2 for s in stages)
    kernel = open(os.path.join(ROOT, "combine_counting_sort_gb300", "csrc", "few_tensor.cuh")).read()
    assert "static_assert(tensor_stages(GROUP, kN, kFewMinSmem) >= kTensorMinStages" in kernel
