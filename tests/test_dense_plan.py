"""The dense products' choice of kernel and shape (csrc/dense_plan.h): every plan keeps within
shared memory, its contraction and the device, over sizes far apart and at the tiles' edges."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROBE = r"""
#include <stdio.h>
#include "dense_plan.h"
using namespace moe;
static long plans = 0, bad = 0, pairs = 0, merged = 0;
static bool check(const DenseShape& s, const DensePlan& p) {
  ++plans;
  if (p.pair) { ++pairs; return true; }
  const long long KB = (s.K + 63) / 64;
  const long stage = 16384 + p.nt * 128, ring = p.stages * stage;
  bool ok = p.nt >= (s.p_mn ? 64 : 16) && p.nt <= 256 && (p.nt & (p.nt - 1)) == 0;
  ok = ok && p.split >= 1 && p.split <= kDFewMaxSplit && p.split <= KB;   // every CTA has a share
  ok = ok && p.stages >= 1 && p.stages <= kDFewMaxStages;
  ok = ok && ring + 1024 + 512 <= 227 * 1024;      // the ring, its alignment and the barriers
  ok = ok && ring >= p.nt * 512L;                  // the tile's sums lie over the ring
  if (!ok) { ++bad; printf("bad: %lld %lld %lld nt %d split %d stages %d\n", s.I, s.J, s.K, p.nt, p.split, p.stages); }
  return ok;
}
int main() {
  const DenseDevice devices[2] = {{152, 76, {{0, 152, 152, 138, 144, 140, 138, 105, 120}, {0, 304, 304, 276, 288, 280, 276, 210, 240}}},
                                  {20, 9, {{0, 20, 18, 15, 12, 5, 0, 0, 0}, {0, 40, 36, 30, 24, 10, 0, 0, 0}}}};   // one that holds no large clusters
  const long long n[] = {1, 7, 8, 15, 16, 17, 33, 64, 65, 127, 128, 129, 255, 256, 257, 511, 1000, 4096, 33000, 1 << 20}, ks[] = {8, 64, 72, 1056, 7168, 1 << 20};
  for (const DenseDevice& d : devices)
    for (long long I : n)
      for (long long J : n)
        for (long long K : ks)
          for (int form = 0; form < 8; ++form) {
            const bool gated = form & 1, mn = !gated && (form & 2), extra = form & 4;
            const DenseShape s = {I, J, K, gated, mn, extra, extra && !gated, !(form & 4)};
            check(s, dense_plan(s, d));
            if (form) continue;
            // a backward pass: d [T, n] with T = I, n = J
            const DenseShape b[2] = {{I, K, J, false, false, false, false, true}, {J, K, I, false, true, false, false, true}};
            DensePlan p[2];
            if (dense_plan_both(b, d, p)) {
              ++merged;
              const int big = p[0].split > p[1].split ? p[0].split : p[1].split, small = p[0].split + p[1].split - big;
              if (!check(b[0], p[0]) || !check(b[1], p[1]) || p[0].pair || p[1].pair || big % small || d.cta[0][big] < big) ++bad;
            } else if (!check(b[0], p[0]) || !check(b[1], p[1])) {
              ++bad;
            }
          }
  printf("%ld %ld %ld %ld\n", plans, bad, pairs, merged);
  return bad != 0;
}
"""


def test_plans(tmp_path):
    src, exe = tmp_path / "probe.cpp", tmp_path / "probe"
    src.write_text(PROBE)
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", os.path.join(ROOT, "combine_counting_sort_gb300", "csrc"), str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout[-2000:]
    plans, bad, pairs, merged = (int(v) for v in r.stdout.split()[-4:])
    assert bad == 0 and plans > 30000
    assert pairs > 1000 and merged > 1000   # both kernels and both forms of a backward pass are reached
