"""Every shape of the few-row dense kernel that the plan chooses (csrc/dense_plan.h): rows a tile x CTAs to a
contraction, for each product, and for each pair of products in one launch.  Which sizes take which shape is asked of
the plan itself, over sizes far apart, and the least of those runs: small whole numbers, so that every product and sum
is exact in fp32 and the outputs are the exact values rounded once, bit for bit."""
import os
import subprocess

import pytest
import torch

import combine_counting_sort_gb300 as moe
from tests import gpu_util
from tests.test_gpu_dense import gen, ints, nan_like

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HALF = (torch.bfloat16, torch.float16)

SCAN = r"""
#include <stdio.h>
#include <map>
#include <string>
#include <vector>
#include "dense_plan.h"
using namespace moe;
struct Size { long long T, N, K; int aux, res; double work; };
static std::map<std::string, Size> least;
static void offer(const char* kind, const DensePlan& p, const DensePlan* q, Size s) {
  char key[80];
  snprintf(key, sizeof key, "%s %d %d %d %d", kind, p.nt, p.split, q ? q->nt : 0, q ? q->split : 0);
  s.work = (double)s.T * s.N * s.K + 1e3 * (s.T * s.N + s.T * s.K + s.N * s.K);
  auto it = least.find(key);
  if (it == least.end() || s.work < it->second.work) least[key] = s;
}
int main() {
  const DenseDevice d = {152, 76, {{0, 152, 152, 138, 144, 140, 138, 105, 120}, {0, 304, 304, 276, 288, 280, 276, 210, 240}}};
  std::vector<long long> Ts, Ns, Ks;
  for (double v = 1; v < 8300; v *= 1.19) Ts.push_back((long long)(v + .5));
  for (double v = 64; v < 33000; v *= 1.25) Ns.push_back((long long)(v + .5)), Ns.push_back((long long)(v / 8 + .5) * 8);
  for (double v = 1; v < 1025; v *= 1.35) Ks.push_back((long long)(v + .5) * 8);
  for (long long T : Ts)
    for (long long N : Ns)
      for (long long K : Ks) {
        for (int form = 0; form < 4; ++form) {
          const bool aux = form & 1, res = form & 2;
          const DensePlan p = dense_plan({T, N, K, false, false, aux, res, N % 8 == 0}, d), q = dense_plan({T, N, K, true, false, aux, false, N % 8 == 0}, d);
          if (!p.pair) offer("linear", p, nullptr, {T, N, K, aux, res});
          if (!q.pair && !res) offer("gated", q, nullptr, {T, N, K, aux, 0});
        }
        const DenseShape b[2] = {{T, K, N, false, false, false, false, true}, {N, K, T, false, true, false, false, true}};
        DensePlan p[2] = {dense_plan(b[0], d), dense_plan(b[1], d)};
        if (!p[0].pair) offer("dx", p[0], nullptr, {T, N, K});
        if (!p[1].pair) offer("dW", p[1], nullptr, {T, N, K});
        if (T * N * K < 4000000000LL && dense_plan_both(b, d, p)) offer("both", p[0], &p[1], {T, N, K});
      }
  for (auto& e : least) printf("%s %lld %lld %lld %d %d\n", e.first.c_str(), e.second.T, e.second.N, e.second.K, e.second.aux, e.second.res);
}
"""


@pytest.fixture(scope="module")
def shapes(tmp_path_factory):
    """{product: [(shape, T, N, K, aux, residual)]}"""
    path = tmp_path_factory.mktemp("scan")
    (path / "scan.cpp").write_text(SCAN)
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", os.path.join(ROOT, "combine_counting_sort_gb300", "csrc"), str(path / "scan.cpp"), "-o",
                    str(path / "scan")], check=True)
    found = {}
    for line in subprocess.run([str(path / "scan")], capture_output=True, text=True, check=True).stdout.splitlines():
        kind, *v = line.split()
        v = [int(n) for n in v]
        found.setdefault(kind, []).append((tuple(v[:4]), *v[4:]))
    return found


def test_the_plan_takes_many_shapes(shapes):
    """What the tests below run: each number of rows a tile and of CTAs, by itself and beside another product."""
    for kind in ("linear", "gated", "dx"):
        assert {s[0][0] for s in shapes[kind]} >= {16, 32, 64, 128} and {s[0][1] for s in shapes[kind]} == set(range(1, 9))
    assert {s[0][0] for s in shapes["dW"]} >= {64, 128} and len(shapes["both"]) > 50


@pytest.fixture
def status():
    gpu_util.build()
    s = torch.zeros(1, dtype=torch.int32, device="cuda")
    yield s
    torch.cuda.synchronize()
    assert s.item() == 0, moe.status_string(s.item())


@pytest.mark.gpu
def test_linear(shapes, status):
    for i, (shape, T, N, K, aux, res) in enumerate(shapes["linear"]):
        dtype, g = HALF[i % 2], gen(i)
        x, W, bias = ints(g, T, K, dtype=dtype), ints(g, N, K, dtype=dtype), ints(g, N, lim=9, dtype=dtype)
        residual, slope, y = ints(g, T, N, lim=9, dtype=dtype) if res else None, nan_like(T, N, dtype=dtype) if aux else None, nan_like(T, N, dtype=dtype)
        moe.moe_linear(x, W, y, status, bias=bias, residual=residual, act=moe.MOE_ACT_RELU, slope=slope)
        a = x.double() @ W.double().t() + bias.double()
        assert torch.equal(y, (a.clamp_min(0) + (residual.double() if res else 0)).to(dtype)), (shape, T, N, K)
        assert not aux or torch.equal(slope, (a > 0).to(dtype)), (shape, T, N, K)


@pytest.mark.gpu
def test_gated(shapes, status):
    for i, (shape, T, F, H, aux, _) in enumerate(shapes["gated"]):
        dtype, g = HALF[i % 2], gen(i)
        # (sums of about 20 ones: the factors and their products stay exact)
        x, W1 = ints(g, T, H, dtype=dtype), ints(g, 2 * F, H, keep=min(1.0, 40.0 / H), dtype=dtype)
        h, factors = nan_like(T, F, dtype=dtype), nan_like(T, 2 * F, dtype=dtype) if aux else None
        moe.moe_gated(x, W1, h, status, act=moe.MOE_ACT_RELU, factors=factors)
        gate, up = (x.double() @ W1.double().t()).split(F, 1)
        assert torch.equal(h, (gate.clamp_min(0) * up).to(dtype)), (shape, T, F, H)
        assert not aux or torch.equal(factors, torch.cat((up * (gate > 0), gate.clamp_min(0)), 1).to(dtype)), (shape, T, F, H)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["dx", "dW", "both"])
def test_backward(kind, shapes, status):
    for i, (shape, T, N, K, _, _) in enumerate(shapes[kind]):
        dtype, g = HALF[i % 2], gen(i)
        x, W, dy = ints(g, T, K, dtype=dtype), ints(g, N, K, dtype=dtype), ints(g, T, N, dtype=dtype)
        ws = torch.full((moe.moe_linear_bwd_ws_bytes(T, N, K),), 0xFF, dtype=torch.uint8, device="cuda")
        dx, dW = nan_like(T, K, dtype=dtype) if kind != "dW" else None, nan_like(N, K, dtype=dtype) if kind != "dx" else None
        moe.moe_linear_bwd(dy, x, W, dx, dW, ws, status)
        assert dx is None or torch.equal(dx, (dy.double() @ W.double()).to(dtype)), (shape, T, N, K)
        assert dW is None or torch.equal(dW, (dy.double().t() @ x.double()).to(dtype)), (shape, T, N, K)
