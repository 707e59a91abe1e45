"""What the layer norm's vectors read of a tensor (csrc/norm.cuh), on the CPU: for every small number of rows
and row length, around the tensor's end and at its start, no vector reads outside the tensor, each one's part of its
row is read, and the rows' parts cover the row once."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROBE = r"""
#include <stdio.h>
#include "norm.cuh"
using namespace moe;
static long vectors = 0, bad = 0, short_reads = 0;
template <typename T, int TPR, int NV, bool MASK>
void check(int H) {
  constexpr int V = kVec16<T>;
  if ((H % V != 0) != MASK) return;
  for (int rows = 1; rows <= 40; ++rows) {
    const long long total = (long long)rows * H;
    for (long long row = 0; row < rows; ++row) {
      long covered = 0;
      for (int tid = 0; tid < TPR; ++tid) {
        const RowPart<T, TPR, NV, MASK> part(H, row, tid);
        const bool tail = row >= norm_tail(rows, H, V == 4 ? MOE_F32 : MOE_F16);
        for (int i = 0; i < NV; ++i) {
          if (!part.any(i)) continue;
          ++vectors;
          const long long at = row * H + part.col(i);
          const int n = part.readable(i, tail);
          covered += part.hi(i) - part.lo(i);
          short_reads += n < V;
          if (at < 0 || at % V || n < part.hi(i) || n > V || at + n > total) ++bad;
        }
      }
      if (covered != H) ++bad;
    }
  }
}
int main() {
  for (int H = 1; H <= 130; ++H) {
    check<__half, 32, 1, true>(H), check<__half, 32, 1, false>(H), check<__half, 32, 4, true>(H), check<__half, 64, 4, true>(H);
    check<float, 64, 1, true>(H), check<float, 64, 1, false>(H), check<float, 64, 4, true>(H);
  }
  printf("%ld %ld %ld\n", vectors, bad, short_reads);
  return bad != 0;
}
"""


def test_no_vector_reads_outside_the_tensor(tmp_path):
    from combine_counting_sort_gb300 import _build
    src, exe = tmp_path / "probe.cu", tmp_path / "probe"
    src.write_text(PROBE)
    subprocess.run([_build.nvcc(), "-std=c++17", "--expt-relaxed-constexpr", *_build.ARCH, "-I", _build.CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
    vectors, bad, short = (int(v) for v in r.stdout.split())
    assert bad == 0 and vectors > 100000 and short > 1000
