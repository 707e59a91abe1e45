"""moe_layernorm and its backward pass against their formulas in 64 bits.

Bounds, with H values a row and e = 2^-23 (fp32): a mean is off by at most
(H / 64 + 12) e of the mean magnitude (each thread adds at most 32 values, the rest
is a tree), a deviation by that and one rounding; a variance, a mean of squares,
by twice a deviation's error.  u = finfo.eps / 2 of the type is the last
rounding; below the type's smallest normal value m its steps stay at finfo.eps * m
(f16: 2^-24 below 2^-14), so half a step is u * m there: `rounding` has both."""
import pytest
import torch

import combine_counting_sort_gb300 as moe
from tests import gpu_util

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]
E = 2.0 ** -23
# rows and their length: every number of threads a row, at its edges, with and without 16-byte vectors
SIZES = [(1, 1), (3, 7), (5, 8), (2, 255), (1, 256), (4, 257), (300, 512), (9, 520), (31, 1000), (700, 1024), (5, 1025), (6, 1111), (17, 2048),
         (350, 2056), (3, 4097), (1, 7168), (400, 7168), (2, 8192), (3, 8193), (4, 8200), (2, 16383), (3, 16384), (20000, 64), (1700, 130)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gpu_util.build()


def data(T, H, dtype, seed, wdtype=None):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(*s, dt=dtype):
        return torch.randn(*s, generator=g, device="cuda").to(dt)

    wd = wdtype or dtype
    x = (torch.randn(T, H, generator=g, device="cuda") * 2 + torch.randn(T, 1, generator=g, device="cuda") * 3).to(dtype)
    return x, r(T, H), (r(H, dt=torch.float32) * 0.2 + 1).to(wd), r(H, dt=wd)


def stats64(x, eps):
    x = x.double()
    mean = x.mean(1, keepdim=True)
    var = (x - mean).square().mean(1, keepdim=True)
    return mean, var, (var + eps).rsqrt()


def dev_error(x, H):
    """Bound of a computed deviation x - mean."""
    return (H / 64 + 14) * E * x.double().abs().mean(1, keepdim=True) + E * x.double().abs()


def rounding(want, dtype):
    f = torch.finfo(dtype)
    return f.eps / 2 * (want.abs() * 1.01 + f.smallest_normal)


def within(got, want, bound, what):
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / bound.clamp_min(1e-300)).max()):.3f} of its bound"


def forward_bounds(x, H, eps):
    mean, var, rstd = stats64(x, eps)
    ed = dev_error(x, H)
    d = x.double() - mean
    # variance: sum of squares of deviations each off by ed, and its own sum's error; rstd half of that relatively
    ev = (2 * d.abs() * ed + ed.square()).mean(1, keepdim=True) + (H / 64 + 14) * E * var
    er = rstd * (0.5 * ev / (var + eps) * 1.1 + 4 * E)
    n = d * rstd
    en = ed * rstd + (d.abs() + ed) * er + 2 * E * n.abs()
    return mean, rstd, n, en, er


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,H", SIZES)
def test_values(T, H, dtype):
    eps = 1e-2 if H < 8 else 1e-5   # a row of few values may lie close together
    x, dy, w, b = data(T, H, dtype, T + H)
    y, mean, rstd = torch.full_like(x, float("nan")), torch.full((T,), float("nan"), device="cuda"), torch.full((T,), float("nan"), device="cuda")
    moe.moe_layernorm(x, w, b, eps, y, mean=mean, rstd=rstd)
    m64, r64, n, en, er = forward_bounds(x, H, eps)
    want = n * w.double() + b.double()
    within(y, want, rounding(want, dtype) + (en * w.double().abs() + 2 * E * (n * w.double()).abs() + E * want.abs()) * 1.01, "y")
    within(mean[:, None], m64, (H / 64 + 14) * E * x.double().abs().mean(1, keepdim=True), "mean")
    within(rstd[:, None], r64, er, "rstd")

    dx, dw, db = torch.full_like(x, float("nan")), torch.full_like(w, float("nan")), torch.full_like(b, float("nan"))
    ws = torch.full((moe.moe_layernorm_bwd_ws_bytes(T, H),), 0xFF, dtype=torch.uint8, device="cuda")
    moe.moe_layernorm_bwd(dy, x, w, mean, rstd, dx, dw, db, ws)
    dy64, g = dy.double(), dy.double() * w.double()
    m1, m2 = g.mean(1, keepdim=True), (g * n).mean(1, keepdim=True)
    want = r64 * (g - m1 - n * m2)
    s = H / 64 + 16
    e1, e2 = s * E * g.abs().mean(1, keepdim=True), s * E * (g * n).abs().mean(1, keepdim=True) + (g.abs() * en).mean(1, keepdim=True)
    size = g.abs() + m1.abs() + (n * m2).abs()
    e = r64 * (e1 + en * m2.abs() + n.abs() * e2 + en * e2 + 5 * E * size) + er * (size + e1 + n.abs() * e2)
    within(dx, want, rounding(want, dtype) + e * 1.05, "dx")
    # sums over T rows: fp32, at most T terms
    within(dw, (dy64 * n).sum(0), rounding((dy64 * n).sum(0), dtype) + (T + 8) * E * (dy64 * n).abs().sum(0) + (dy64.abs() * en).sum(0) * 1.01, "dweight")
    within(db, dy64.sum(0), rounding(dy64.sum(0), dtype) + (T + 8) * E * dy64.abs().sum(0), "dbias")
