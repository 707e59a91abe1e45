"""moe_linear and moe_gated with their backward passes, against their formulas
in 64 bits.

Two kinds of checks.  Small whole numbers as inputs: every product and sum is
exact in fp32, so the outputs are the exact values rounded once, bit for bit, at
every size, head, tail and memory order.  Random inputs: each output is within a
bound derived from the roundings on its way, element by element:

  * a sum of n terms in fp32, in any order and with truncating adders, is off by
    at most n 2^-22 sum|terms|;
  * a rounding to the type is off by u = finfo.eps / 2 of the value;
  * an activation or its slope is off by ACT of its size (|a| included): exp
    within (|a| + 2) 2^-22 for |a| < 60, the quotient and products a few 2^-23 more.
"""
import math

import pytest
import torch

import combine_counting_sort_gb300 as moe
from tests import gpu_util

pytestmark = pytest.mark.gpu

HALF = [torch.bfloat16, torch.float16]
ACTS = {"none": moe.MOE_ACT_NONE, "relu": moe.MOE_ACT_RELU, "silu": moe.MOE_ACT_SILU, "gelu": moe.MOE_ACT_GELU,
        "gelu_tanh": moe.MOE_ACT_GELU_TANH}
ACT = 2.0 ** -15

# rows, columns, contraction: one of each, one row, the tiles' edges on either side, several tiles, long contractions
SIZES = [(1, 1, 8), (1, 7168, 2048), (2, 129, 72), (15, 64, 64), (16, 127, 200), (17, 513, 1024), (33, 256, 520), (64, 4096, 512),
         (65, 1111, 1056), (129, 257, 136), (255, 128, 64), (256, 256, 256), (257, 300, 4096), (515, 711, 1032), (1000, 2048, 264),
         (2049, 2305, 328), (5000, 64, 8), (3, 20000, 16)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gpu_util.build()


@pytest.fixture
def status():
    s = torch.zeros(1, dtype=torch.int32, device="cuda")
    yield s
    torch.cuda.synchronize()
    assert s.item() == 0, moe.status_string(s.item())


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def ints(g, *shape, lim=1, keep=1.0, dtype=torch.bfloat16):
    """Whole numbers in [-lim, lim], a share `keep` of them not zero."""
    v = torch.randint(-lim, lim + 1, shape, generator=g, device="cuda").double()
    if keep < 1:
        v *= torch.rand(shape, generator=g, device="cuda") < keep
    return v.to(dtype)


def nan_like(*shape, dtype):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def act64(a, name):
    if name == "none":
        return a, torch.ones_like(a)
    if name == "relu":
        return a.clamp_min(0), (a > 0).double()
    if name == "silu":
        s = torch.sigmoid(a)
        return a * s, s * (1 + a * (1 - s))
    if name == "gelu":
        c = 0.5 * torch.erfc(-a * math.sqrt(0.5))
        return a * c, c + a * torch.exp(-0.5 * a * a) / math.sqrt(2 * math.pi)
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (a + 0.044715 * a ** 3))
    return 0.5 * a * (1 + t), 0.5 * (1 + t) + 0.5 * a * (1 - t * t) * k * (1 + 3 * 0.044715 * a * a)


def half(dtype):
    return torch.finfo(dtype).eps / 2


def within(got, want, bound, what):
    err = (got.double() - want).abs()
    assert torch.isfinite(got.double()).all(), f"{what}: not finite"
    bad = err > bound
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / bound.clamp_min(1e-300)).max()):.3f} of its bound"


# ---------------------------------------------------------------- exact: whole numbers

@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("T,N,K", SIZES)
def test_linear_exact(T, N, K, dtype, status):
    g = gen(T + N + K)
    x, W = ints(g, T, K, dtype=dtype), ints(g, N, K, dtype=dtype)
    bias, res = ints(g, N, lim=9, dtype=dtype), ints(g, T, N, lim=9, dtype=dtype)
    want = x.double() @ W.double().t()
    y = nan_like(T, N, dtype=dtype)
    moe.moe_linear(x, W, y, status)
    assert torch.equal(y, want.to(dtype))
    moe.moe_linear(x, W, y, status, bias=bias)
    assert torch.equal(y, (want + bias.double()).to(dtype))
    slope = nan_like(T, N, dtype=dtype)
    y.copy_(res)   # the residual in place
    moe.moe_linear(x, W, y, status, bias=bias, residual=y, act=moe.MOE_ACT_RELU, slope=slope)
    a = want + bias.double()
    assert torch.equal(y, (a.clamp_min(0) + res.double()).to(dtype))
    assert torch.equal(slope, (a > 0).to(dtype))


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("T,N,K", SIZES)
def test_linear_bwd_exact(T, N, K, dtype, status):
    g = gen(T + N + K + 1)
    x, W, dy = ints(g, T, K, dtype=dtype), ints(g, N, K, dtype=dtype), ints(g, T, N, lim=3, dtype=dtype)
    slope = ints(g, T, N, lim=2, dtype=dtype)
    ws = torch.full((moe.moe_linear_bwd_ws_bytes(T, N, K),), 0xFF, dtype=torch.uint8, device="cuda")   # NaN wherever it is read unwritten
    for s in (None, slope):
        d = dy.double() if s is None else dy.double() * s.double()
        dx, dW, db = nan_like(T, K, dtype=dtype), nan_like(N, K, dtype=dtype), nan_like(N, dtype=dtype)
        moe.moe_linear_bwd(dy, x, W, dx, dW, ws, status, dbias=db, slope=s)
        assert torch.equal(dx, (d @ W.double()).to(dtype))
        assert torch.equal(dW, (d.t() @ x.double()).to(dtype))
        assert torch.equal(db, d.sum(0).to(dtype))


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("T,F,H", SIZES)
def test_gated_exact(T, F, H, dtype, status):
    g = gen(T + F + H + 2)
    keep = min(1.0, 40.0 / H)   # sums of about 20 ones: the factors and their products stay exact
    x, W1 = ints(g, T, H, dtype=dtype), ints(g, 2 * F, H, keep=keep, dtype=dtype)
    gate, up = (x.double() @ W1.double().t()).split(F, 1)
    h, factors = nan_like(T, F, dtype=dtype), nan_like(T, 2 * F, dtype=dtype)
    moe.moe_gated(x, W1, h, status, act=moe.MOE_ACT_NONE)
    assert torch.equal(h, (gate * up).to(dtype))
    h.fill_(float("nan"))
    moe.moe_gated(x, W1, h, status, act=moe.MOE_ACT_RELU, factors=factors)
    want = torch.cat((up * (gate > 0), gate.clamp_min(0)), 1)
    assert torch.equal(h, (gate.clamp_min(0) * up).to(dtype)) and torch.equal(factors, want.to(dtype))


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("T,F,H", SIZES)
def test_gated_bwd_exact(T, F, H, dtype, status):
    g = gen(T + F + H + 3)
    x, W1, dh = ints(g, T, H, dtype=dtype), ints(g, 2 * F, H, dtype=dtype), ints(g, T, F, lim=2, dtype=dtype)
    factors = ints(g, T, 2 * F, lim=2, dtype=dtype)
    d = factors.double() * torch.cat((dh, dh), 1).double()
    ws = torch.full((moe.moe_gated_bwd_ws_bytes(T, F, H),), 0xFF, dtype=torch.uint8, device="cuda")
    dx, dW1 = nan_like(T, H, dtype=dtype), nan_like(2 * F, H, dtype=dtype)
    moe.moe_gated_bwd(dh, x, W1, factors, dx, dW1, ws, status)
    assert torch.equal(dx, (d @ W1.double()).to(dtype))
    assert torch.equal(dW1, (d.t() @ x.double()).to(dtype))


# ---------------------------------------------------------------- random values

def rand(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def sums(a, b, extra=0.0):
    """a @ b.T in 64 bits and the bound of its fp32 sum."""
    a, b = a.double(), b.double()
    return a @ b.t(), (a.shape[1] + 2) * 2.0 ** -22 * (a.abs() @ b.abs().t() + extra)


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("T,N,K,dtype", [(1, 700, 256, torch.bfloat16), (37, 1111, 1056, torch.float16), (300, 264, 72, torch.bfloat16),
                                         (2600, 2000, 512, torch.bfloat16)])
def test_linear_values(T, N, K, dtype, act, status):
    g = gen(7 * T + N)
    u = half(dtype)
    x, W = rand(g, T, K, dtype=dtype), rand(g, N, K, scale=2 / math.sqrt(K), dtype=dtype)
    bias, res, dy = rand(g, N, dtype=dtype), rand(g, T, N, dtype=dtype), rand(g, T, N, dtype=dtype)
    y, slope = nan_like(T, N, dtype=dtype), nan_like(T, N, dtype=dtype)
    moe.moe_linear(x, W, y, status, bias=bias, residual=res, act=ACTS[act], slope=slope)
    a, ea = sums(x, W, bias.double().abs())
    a = a + bias.double()
    want, ws = act64(a, act)
    tiny = torch.finfo(dtype).smallest_normal   # below it a rounding's step does not shrink further
    # act and act' change by at most 1.13 and 1.1 times a change of a
    within(y, want + res.double(), u * (want + res.double()).abs() * 1.01 + 1.2 * ea + ACT * (want.abs() + res.double().abs()) + u * tiny, "y")
    jump = (a.abs() <= ea) if act == "relu" else torch.zeros_like(a, dtype=torch.bool)   # relu's slope where the sum's sign is in doubt
    within(slope, torch.where(jump, slope.double(), ws), u * ws.abs() * 1.01 + 1.2 * ea + ACT * (1 + a.abs()) + u * tiny, "slope")

    # backward: from the slope as it was written
    dx, dW, db = nan_like(T, K, dtype=dtype), nan_like(N, K, dtype=dtype), nan_like(N, dtype=dtype)
    wsp = torch.empty(moe.moe_linear_bwd_ws_bytes(T, N, K), dtype=torch.uint8, device="cuda")
    moe.moe_linear_bwd(dy, x, W, dx, dW, wsp, status, dbias=db, slope=slope)
    d = dy.double() * slope.double()
    tail = u * tiny * torch.ones_like(d)
    ed = u * d.abs() * 1.01 + tail
    for name, got, l, el, r in (("dx", dx, d, ed, W.double()), ("dW", dW, d.t(), ed.t(), x.double().clone())):
        want = l @ r
        bound = u * want.abs() * 1.01 + el @ r.abs() * 1.01 + (l.shape[1] + 2) * 2.0 ** -22 * (l.abs() @ r.abs()) * 1.01 + u * tiny
        within(got, want, bound, name)
    within(db, d.sum(0), u * d.sum(0).abs() * 1.01 + (T + 2) * 2.0 ** -23 * d.abs().sum(0) + u * tiny, "dbias")


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("T,F,H,dtype", [(1, 320, 256, torch.bfloat16), (50, 711, 1032, torch.float16), (2600, 1000, 512, torch.bfloat16)])
def test_gated_values(T, F, H, dtype, act, status):
    g = gen(5 * T + F)
    u, tiny = half(dtype), torch.finfo(dtype).smallest_normal
    x, W1, dh = rand(g, T, H, dtype=dtype), rand(g, 2 * F, H, scale=2 / math.sqrt(H), dtype=dtype), rand(g, T, F, dtype=dtype)
    h, factors = nan_like(T, F, dtype=dtype), nan_like(T, 2 * F, dtype=dtype)
    moe.moe_gated(x, W1, h, status, act=ACTS[act], factors=factors)
    s, es = sums(x, W1)
    (gate, up), (eg, eu) = s.split(F, 1), es.split(F, 1)
    a, sl = act64(gate, act)
    e = 1.2 * eg * (up.abs() + eu) + a.abs() * eu + ACT * (a * up).abs()
    within(h, a * up, u * (a * up).abs() * 1.01 + 1.01 * e + u * tiny, "h")
    jump = (gate.abs() <= eg) if act == "relu" else torch.zeros_like(gate, dtype=torch.bool)
    p = sl * up
    within(factors[:, :F], torch.where(jump, factors[:, :F].double(), p),
           u * p.abs() * 1.01 + 1.2 * eg * (up.abs() + eu) + 1.2 * eu + ACT * (1 + gate.abs()) * up.abs() + u * tiny, "u act'(g)")
    within(factors[:, F:], a, u * a.abs() * 1.01 + 1.2 * eg + ACT * a.abs() + u * tiny, "act(g)")

    dx, dW1 = nan_like(T, H, dtype=dtype), nan_like(2 * F, H, dtype=dtype)
    wsp = torch.empty(moe.moe_gated_bwd_ws_bytes(T, F, H), dtype=torch.uint8, device="cuda")
    moe.moe_gated_bwd(dh, x, W1, factors, dx, dW1, wsp, status)
    d = factors.double() * torch.cat((dh, dh), 1).double()
    ed = u * d.abs() * 1.01 + u * tiny
    for name, got, l, el, r in (("dx", dx, d, ed, W1.double()), ("dW1", dW1, d.t(), ed.t(), x.double())):
        want = l @ r
        bound = u * want.abs() * 1.01 + el @ r.abs() * 1.01 + (l.shape[1] + 2) * 2.0 ** -22 * (l.abs() @ r.abs()) * 1.01 + u * tiny
        within(got, want, bound, name)
