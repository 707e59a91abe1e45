"""The dense operators' host code on several devices, and after a call of the runtime failed: against a
fake CUDA runtime (fake_cudart.h) that keeps what belongs to a device by device, without a GPU."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# calls: every operator in sizes that take each of its kernels, none of which reads its addresses
CALLS = r"""
#include "fake_cudart.h"
#include "moe.h"
static void* const A = (void*)(1 << 20);
static int32_t* const S = (int32_t*)A;
static float* const FA = (float*)A;
static size_t big = (size_t)1 << 40;
static int few_linear() { return moe_linear(A, 1, 2048, A, 7168, MOE_BF16, 0, 0, 0, A, 0, S, 0); }
static int pair_linear() { return moe_linear(A, 4096, 2048, A, 7168, MOE_F16, 0, 0, 0, A, 0, S, 0); }
static int pair_slope() { return moe_linear(A, 4096, 2048, A, 7168, MOE_BF16, 0, 0, 2, A, A, S, 0); }
static int few_gated() { return moe_gated(A, 8, 2048, A, 1024, MOE_F16, 2, A, 0, S, 0); }
static int pair_gated() { return moe_gated(A, 4096, 2048, A, 1024, MOE_BF16, 2, A, A, S, 0); }
static int both_backward() { return moe_linear_bwd(A, A, 300, 512, A, 256, MOE_BF16, 0, A, A, A, A, big, S, 0); }
static int pair_backward() { return moe_gated_bwd(A, A, 4096, 2048, A, 1024, MOE_BF16, A, A, A, A, big, S, 0); }
static int norm() { return moe_layernorm(A, 8192, 7168, MOE_BF16, A, A, MOE_BF16, 1e-5f, A, 0, 0, 0); }
static int odd_norm() { return moe_layernorm(A, 8192, 7167, MOE_F16, A, A, MOE_F32, 1e-5f, A, 0, 0, 0); }
static int norm_backward() { return moe_layernorm_bwd(A, A, 8192, 7168, MOE_BF16, A, MOE_BF16, FA, FA, A, A, A, A, big, 0); }
static int few_norm_backward() { return moe_layernorm_bwd(A, A, 8, 7168, MOE_BF16, A, MOE_BF16, FA, FA, (char*)A + 4096, A, A, A, big, 0); }
static int (*const calls[])() = {few_linear, pair_linear, pair_slope, few_gated, pair_gated, both_backward, pair_backward, norm, odd_norm, norm_backward,
                                 few_norm_backward};
"""

DEVICES = CALLS + r"""
int main() {
  for (auto call : calls)
    for (int dev : {0, 1, 0, 2}) {
      fake().device = dev;
      fake().launches.clear();
      EXPECT(call() == MOE_OK);
      EXPECT(!fake().launches.empty());
      // a grid that is as large as the device: its own SMs
      if (call == norm) EXPECT((int)fake().launches[0].grid.x == fake().sms[dev] / 8 * 8 * 2);
      if (call == pair_linear) EXPECT((int)fake().launches[0].grid.x <= fake().sms[dev]);
    }
  // one shape on two devices: each has the plan for its own SMs, whichever was asked first
  unsigned grid[2][2];
  for (int turn = 0; turn < 2; ++turn)
    for (int dev : {1, 0}) {
      fake().device = dev;
      fake().launches.clear();
      EXPECT(moe_linear(A, 64, 1024, A, 4096, MOE_BF16, 0, 0, 0, A, 0, S, 0) == MOE_OK);
      grid[turn][dev] = fake().launches[0].grid.x;
    }
  EXPECT(grid[0][0] == grid[1][0] && grid[0][1] == grid[1][1] && grid[0][0] != grid[0][1]);
  printf("ok\n");
}
"""

FAILURES = CALLS + r"""
int main() {
  // the first call on a device meets a failure of the runtime, in each place; the next one does not
  int dev = 0;
  for (int which = 0; which < 2; ++which, ++dev) {
    fake().device = dev;
    for (auto call : calls)
      for (int n = 1; n <= 2; ++n) {
        (which ? fake().fail_occupancy : fake().fail_attribute) = n;
        const int rc = call();
        EXPECT(rc == MOE_OK || rc == MOE_ERR_CUDA);
        fake().fail_attribute = fake().fail_occupancy = 0;
        EXPECT(call() == MOE_OK);
      }
  }
  printf("ok\n");
}
"""

LEFT_BEHIND = CALLS + r"""
int main() {
  // after a call that failed, wherever it did, a later cudaGetLastError finds nothing
  int dev = 0;
  for (int which = 0; which < 3; ++which, ++dev) {
    fake().device = dev;
    for (auto call : calls) {
      int& fail = which == 0 ? fake().fail_attribute : which == 1 ? fake().fail_occupancy : fake().fail_launch;
      fail = 1;
      const int rc = call();
      EXPECT(rc == MOE_ERR_CUDA || (rc == MOE_OK && fail == 1));   // (a limit that is set already is not set again)
      fail = 0;
      EXPECT(fake().last == cudaSuccess);
      EXPECT(call() == MOE_OK);
    }
  }
  printf("ok\n");
}
"""

GRIDS = CALLS + r"""
static int blocks(int (*call)(int rows), int rows, int dev) {
  fake().device = dev;
  fake().launches.clear();
  EXPECT(call(rows) == MOE_OK);
  const dim3 g = fake().launches[0].grid;
  return (int)(g.x * g.y);
}
static int sums(int T) { return moe_linear_bwd(A, A, T, 512, A, 4096, MOE_BF16, A, 0, 0, A, A, big, S, 0); }
static int slopes(int T) { return moe_linear_bwd(A, A, T, 512, A, 4096, MOE_BF16, A, A, 0, 0, A, big, S, 0); }
static int factors(int T) { return moe_gated_bwd(A, A, T, 512, A, 4096, MOE_BF16, A, A, 0, A, big, S, 0); }
int main() {
  // the elementwise kernels in front of the backward products, with more rows than any device takes at once:
  // as many blocks as the device runs, whichever it is (32 strips of 128 columns; the gated one's of 2048)
  fake().sms[1] = 76;
  for (int dev : {0, 1}) {
    const int sms = fake().sms[dev];
    EXPECT(blocks(slopes, 1 << 20, dev) > 2 * sms - 32 && blocks(slopes, 1 << 20, dev) <= 2 * sms);
    EXPECT(blocks(sums, 1 << 20, dev) > sms && blocks(sums, 1 << 20, dev) <= 2 * sms);
    EXPECT(blocks(factors, 1 << 20, dev) == 16 * sms);
  }
  EXPECT(blocks(slopes, 1, 0) == 32 && blocks(factors, 1, 0) == 2);
  printf("ok\n");
}
"""


def run(source, tmp_path):
    from combine_counting_sort_gb300 import _build
    _build.build()
    objects = [os.path.join(_build.BUILD, o + ".o") for o in ("dense", "dense_bf16", "dense_f16", "norm", "norm_bwd", "norm_bwd_few")]
    if not all(os.path.exists(o) for o in objects):   # a library that was built elsewhere
        _build.build(force=True)
    nvcc = _build.nvcc()
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    if not os.path.isdir(include):
        pytest.skip("the toolkit's headers are not where its compiler is")
    src, exe = tmp_path / "main.cpp", tmp_path / "main"
    src.write_text(source)
    subprocess.run([shutil.which("g++") or "g++", "-std=c++17", "-isystem", include, "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "tests"),
                    str(src), *objects, "-o", str(exe), "-lpthread"], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.endswith("ok\n"), r.stdout[-2000:]


def test_every_device_has_its_own(tmp_path):
    run(DEVICES, tmp_path)


def test_grids_are_the_devices(tmp_path):
    run(GRIDS, tmp_path)


def test_a_failure_leaves_no_error_behind(tmp_path):
    run(LEFT_BEHIND, tmp_path)


def test_a_failure_is_not_kept(tmp_path):
    run(FAILURES, tmp_path)
