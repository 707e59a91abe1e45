"""Layer norm on rows where it can go wrong: shorter than a vector beside what is not the tensor's, of
equal values, and far from zero.  Bounds as in test_gpu_norm.py where nothing else is said."""
import pytest
import torch

import combine_counting_sort_gb300 as moe
from tests import gpu_util
from tests.test_gpu_norm import E, TYPES, data, forward_bounds, rounding, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gpu_util.build()


def framed(t, by):
    """t's values between NaN, `by` of them in front: a whole number of vectors, or none."""
    n = t.numel()
    buf = torch.full((by + n + 16,), float("nan"), dtype=t.dtype, device="cuda")
    v = buf[by:by + n].view(t.shape)
    v.copy_(t)
    return v, buf, by


def frame_kept(buf, by, n):
    return bool(buf[:by].isnan().all() and buf[by + n:].isnan().all())


def check_against_formula(x, dy, w, b, eps, y, mean, rstd, dx, dw, db):
    """Every output of a forward and a backward call against 64 bits, by test_gpu_norm.py's bounds."""
    T, H = x.shape
    dtype = x.dtype
    _, r64, n, en, er = forward_bounds(x, H, eps)
    w64, dy64 = w.double(), dy.double()
    want = n * w64 + b.double()
    within(y, want, rounding(want, dtype) + (en * w64.abs() + 2 * E * (n * w64).abs() + E * want.abs()) * 1.01, "y")
    within(rstd[:, None], r64, er, "rstd")
    g = dy64 * w64
    m1, m2 = g.mean(1, keepdim=True), (g * n).mean(1, keepdim=True)
    want = r64 * (g - m1 - n * m2)
    s = H / 64 + 16
    e1, e2 = s * E * g.abs().mean(1, keepdim=True), s * E * (g * n).abs().mean(1, keepdim=True) + (g.abs() * en).mean(1, keepdim=True)
    size = g.abs() + m1.abs() + (n * m2).abs()
    e = r64 * (e1 + en * m2.abs() + n.abs() * e2 + en * e2 + 5 * E * size) + er * (size + e1 + n.abs() * e2)
    within(dx, want, rounding(want, dtype) + e * 1.05, "dx")
    want = (dy64 * n).sum(0)
    within(dw, want, rounding(want, dtype) + (T + 8) * E * (dy64 * n).abs().sum(0) + (dy64.abs() * en).sum(0) * 1.01, "dweight")
    within(db, dy64.sum(0), rounding(dy64.sum(0), dtype) + (T + 8) * E * dy64.abs().sum(0), "dbias")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H", [1, 2, 3, 4, 5, 6, 7, 8, 9, 15])
def test_short_rows_beside_other_values(H, dtype):
    """Rows shorter than a vector, whose loads meet several rows and the tensor's ends: what lies around the
    tensor stays out of the results and as it was, for few rows and for many."""
    for T in (1, 2, 3, 5, 8, 9, 70001):
        x, dy, w, b = data(T, H, dtype, 100 * T + H)
        for by in (8, 3):
            (xv, _, _), (dv, _, _), (wv, _, _), (bv, _, _) = (framed(t, by) for t in (x, dy, w, b))
            (yv, yb, _), (gv, gb, _) = framed(torch.zeros_like(x), by), framed(torch.zeros_like(x), by)
            (sv, sb, _), (tv, tb, _) = framed(torch.zeros_like(w), by), framed(torch.zeros_like(w), by)
            mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
            moe.moe_layernorm(xv, wv, bv, 1e-2, yv, mean=mean, rstd=rstd)
            ws = torch.empty(moe.moe_layernorm_bwd_ws_bytes(T, H), dtype=torch.uint8, device="cuda")
            moe.moe_layernorm_bwd(dv, xv, wv, mean, rstd, gv, sv, tv, ws)
            check_against_formula(x, dy, w, b, 1e-2, yv, mean, rstd, gv, sv, tv)
            assert all(frame_kept(*f) for f in ((yb, by, T * H), (gb, by, T * H), (sb, by, H), (tb, by, H)))


def forms(H, dtype):
    """Rows and the alignment of x that take each of the forward kernels: few rows, many rows, rows that start anywhere."""
    many = 1 + 8_000_000 // max(H, 256)
    return ((3, 0), (many, 0), (5, 1))


def at_offset(x, by):
    buf = torch.empty(x.numel() + by, dtype=x.dtype, device="cuda")
    v = buf[by:].view(x.shape)
    v.copy_(x)
    return v


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H", [1, 2, 7, 33, 64, 100, 777, 1000, 1111, 4096, 7168, 8191, 12288, 16383, 16384])
def test_rows_of_equal_values(H, dtype):
    """Their mean is the value, n is 0 and y the bias, bit for bit, however far from zero and at every alignment; so
    is dweight 0.  (f16 rows of more than 8192 values: 2^13 times 11 bits fill fp32.)"""
    values = torch.tensor([0.0, 1.0, 100.0, -3.25, 50000.0, 0.1, 1000.123, -7.7e-3, 12345.678], device="cuda")
    g = torch.Generator(device="cuda").manual_seed(H)
    w, b = (torch.randn(H, generator=g, device="cuda").to(dtype) for _ in range(2))
    for T, by in forms(H, dtype):
        c = values.repeat(T // 9 + 1)[:T].to(dtype)
        x = at_offset(c[:, None].expand(T, H), by)
        y, mean, rstd = torch.full_like(x, float("nan")), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        moe.moe_layernorm(x, w, b, 1e-5, y, mean=mean, rstd=rstd)
        assert torch.equal(mean, c.float()), (T, by)
        assert torch.equal(y, b[None].expand(T, H)), (T, by, float((y.double() - b.double()).abs().max()))
        dy, dx, dw, db = torch.randn(T, H, generator=g, device="cuda").to(dtype), torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
        ws = torch.empty(moe.moe_layernorm_bwd_ws_bytes(T, H), dtype=torch.uint8, device="cuda")
        moe.moe_layernorm_bwd(dy, x, w, mean, rstd, dx, dw, db, ws)
        assert torch.equal(dw, torch.zeros_like(dw)), (T, by)


@pytest.mark.parametrize("far", [1e3, -1e5])
@pytest.mark.parametrize("H", [33, 100, 1000, 1111, 4096, 7168, 12288, 16384])
def test_f32_rows_far_from_zero(H, far):
    """Rows whose mean is 10^3 and 10^5 times their deviation.  A warp's mean and the row's are each rounded once, by
    half a step of |mean|, the deviations from the first are exact, and their sum is off by (H / 64 + 14) e of their
    size: no rounding of a sum of H such values is left, which would be (H / 64 + 12) e |mean|."""
    eps = 1e-5
    for T, by in forms(H, torch.float32):
        g = torch.Generator(device="cuda").manual_seed(T + H)
        x = at_offset(torch.randn(T, H, generator=g, device="cuda") + far, by)
        y, mean, rstd = torch.full_like(x, float("nan")), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        moe.moe_layernorm(x, None, None, eps, y, mean=mean, rstd=rstd)
        x64 = x.double()
        m64 = x64.mean(1, keepdim=True)
        d = x64 - m64
        var = d.square().mean(1, keepdim=True)
        r64 = (var + eps).rsqrt()
        em = 1.05 * E * m64.abs() + (H / 64 + 14) * E * d.abs().mean(1, keepdim=True)
        ed = em + E * d.abs()
        er = r64 * (0.55 * ((2 * d.abs() * ed + ed.square()).mean(1, keepdim=True) + (H / 64 + 14) * E * var) / (var + eps) + 4 * E)
        within(mean[:, None], m64, em, "mean")
        within(rstd[:, None], r64, er, "rstd")
        within(y, d * r64, ed * r64 + (d.abs() + ed) * er + 3 * E * (d * r64).abs(), "y")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,H", [(1, 33), (7, 1000), (400, 1111), (900, 4096), (5000, 200), (40, 8200), (700, 7168), (2500, 1112), (1200, 1999), (6, 16383)])
def test_in_place_and_on_views_against_the_formula(T, H, dtype):
    """y over x, dx over dy, dx over x, and tensors that start anywhere: each within the bounds of test_gpu_norm.py
    of the formula, as separate aligned tensors are."""
    x, dy, w, b = data(T, H, dtype, 7 * T + H)
    eps = 1e-5
    ws = torch.empty(moe.moe_layernorm_bwd_ws_bytes(T, H), dtype=torch.uint8, device="cuda")

    def run(xf, y, dyb, xb, dx, w, b, new):
        mean, rstd, dw, db = torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), new(w), new(b)
        moe.moe_layernorm(xf, w, b, eps, y, mean=mean, rstd=rstd)
        out = y.clone()   # (y may be what the backward call writes into)
        ws.fill_(0xFF)
        moe.moe_layernorm_bwd(dyb, xb, w, mean, rstd, dx, dw, db, ws)
        check_against_formula(x, dy, w, b, eps, out, mean, rstd, dx, dw, db)

    def copy(t):
        return t.clone()

    def view(t):
        return at_offset(t, 1)

    xi, di = copy(x), copy(dy)
    run(xi, xi, di, x, di, w, b, copy)            # y over x, dx over dy
    xb = copy(x)
    run(x, copy(x), dy, xb, xb, w, b, copy)       # dx over x
    wv, bv = view(w), view(b)
    run(view(x), view(x), view(dy), view(x), view(x), wv, bv, view)
    xi, di = view(x), view(dy)
    run(xi, xi, di, view(x), di, wv, bv, view)    # the same on views
    xb = view(x)
    run(view(x), view(x), view(dy), xb, xb, wv, bv, view)
    run(x, copy(x), view(dy), x, copy(x), w, bv, copy)   # one tensor alone starts anywhere
