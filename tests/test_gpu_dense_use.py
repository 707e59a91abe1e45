"""The dense operators as they are used: together with their gradients, in graphs
and on side streams, in place, on views that no vector fits, without rows, with values that
are not finite, and past 2^31 elements.  Bounds as in test_gpu_dense.py and
test_gpu_norm.py: u = finfo.eps / 2 for a rounding, n 2^-22 sum|terms| for a sum of n terms."""
import math

import pytest
import torch

import combine_counting_sort_gb300 as moe
from tests import gpu_util
from tests.test_gpu_dense import ACTS, act64, ints, nan_like

pytestmark = pytest.mark.gpu
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-5


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


def ws_of(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda")


# ---------------------------------------------------------------- the sublayer, forward and backward

class Sublayer:
    """y = linear(gated(norm(x))) + x with every gradient, in the operators' own calls."""

    def __init__(self, T, H, F, dtype, seed, status):
        g = gen(seed)

        def r(*s, scale=1.0):
            return (torch.randn(*s, generator=g, device="cuda") * scale).to(dtype)
        self.T, self.H, self.F, self.status = T, H, F, status
        self.x, self.dy = r(T, H), r(T, H)
        self.w, self.b = (r(H, scale=0.1).float() + 1).to(dtype), r(H, scale=0.1)
        self.W1, self.W2, self.b2 = r(2 * F, H, scale=H ** -0.5), r(H, F, scale=F ** -0.5), r(H, scale=0.1)
        e = lambda *s, d=dtype: nan_like(*s, dtype=d)   # noqa: E731
        self.n, self.mean, self.rstd = e(T, H), e(T, d=F32), e(T, d=F32)
        self.h, self.factors, self.y = e(T, F), e(T, 2 * F), e(T, H)
        self.dh, self.dn, self.dx = e(T, F), e(T, H), e(T, H)
        self.dw, self.db, self.dW1, self.dW2, self.db2 = e(H), e(H), e(2 * F, H), e(H, F), e(H)
        self.ws = ws_of(max(moe.moe_linear_bwd_ws_bytes(T, H, F), moe.moe_gated_bwd_ws_bytes(T, F, H), moe.moe_layernorm_bwd_ws_bytes(T, H)))

    def step(self):
        moe.moe_layernorm(self.x, self.w, self.b, EPS, self.n, mean=self.mean, rstd=self.rstd)
        moe.moe_gated(self.n, self.W1, self.h, self.status, factors=self.factors)
        moe.moe_linear(self.h, self.W2, self.y, self.status, bias=self.b2, residual=self.x)
        moe.moe_linear_bwd(self.dy, self.h, self.W2, self.dh, self.dW2, self.ws, self.status, dbias=self.db2)
        moe.moe_gated_bwd(self.dh, self.n, self.W1, self.factors, self.dn, self.dW1, self.ws, self.status)
        moe.moe_layernorm_bwd(self.dn, self.x, self.w, self.mean, self.rstd, self.dx, self.dw, self.db, self.ws)
        self.dx += self.dy   # the residual's own gradient

    def outputs(self):
        return {k: getattr(self, k) for k in ("y", "dx", "dw", "db", "dW1", "dW2", "db2")}

    def loss64(self, x, w, b, W1, W2, b2):
        n = torch.nn.functional.layer_norm(x, (self.H,), w, b, EPS)
        g, u = (n @ W1.t()).split(self.F, 1)
        y = (g * torch.sigmoid(g) * u) @ W2.t() + b2 + x
        return (y * self.dy.double()).sum(), y

    def want(self):
        leaves = [t.double().requires_grad_() for t in (self.x, self.w, self.b, self.W1, self.W2, self.b2)]
        loss, y = self.loss64(*leaves)
        loss.backward()
        return dict(zip(("dx", "dw", "db", "dW1", "dW2", "db2"), (t.grad for t in leaves)), y=y.detach())


@pytest.mark.parametrize("T,H,F,dtype", [(1, 256, 128, BF), (37, 264, 104, F16), (300, 1032, 712, BF), (1500, 512, 640, BF), (3000, 640, 1000, F16)])
def test_sublayer_and_its_gradients(T, H, F, dtype, status):
    """Against 64-bit autograd.  An output passes through at most eight roundings to the type (n, factors, h,
    d, dh, dn and its own, and the residual's sum), each off by u of the value that it rounds; errors
    add up to at most 8 u of the outputs' size where nothing amplifies them, here taken twice as large and
    in the norm over all elements (the roundings' signs are independent)."""
    s = Sublayer(T, H, F, dtype, T + H, status)
    s.step()
    u, want = torch.finfo(dtype).eps / 2, s.want()
    for k, got in s.outputs().items():
        err = (got.double() - want[k]).norm() / want[k].norm()
        assert torch.isfinite(got.double()).all() and err <= 16 * u, f"{k}: {float(err):.2e} of {16 * u:.2e}"


def test_gradients_against_differences(status):
    """The step's gradients, as directional derivatives, against central differences of the 64-bit loss: with a
    step of 1e-4 their error is about 1e-8 of the third derivative, far below 16 u of each term."""
    s = Sublayer(23, 136, 72, F16, 5, status)
    s.step()
    names, leaves = ("dx", "dw", "db", "dW1", "dW2", "db2"), [t.double() for t in (s.x, s.w, s.b, s.W1, s.W2, s.b2)]
    g = gen(9)
    for i, name in enumerate(names):
        d = torch.randn(leaves[i].shape, generator=g, device="cuda", dtype=torch.float64)
        lo, hi = ([t + (sign * 1e-4 * d if j == i else 0) for j, t in enumerate(leaves)] for sign in (-1, 1))
        want = (s.loss64(*hi)[0] - s.loss64(*lo)[0]) / 2e-4
        grad = getattr(s, name).double()
        # each element off by 16 u of the gradient's mean size: the sum along d by that times |d|
        bound = 16 * torch.finfo(F16).eps / 2 * grad.norm() * d.norm() / math.sqrt(d.numel()) * 4
        assert abs((grad * d).sum() - want) <= bound, name


def test_captured_and_replayed(status):
    """Two graphs over one workspace, replayed in turn with new inputs: the eager results bit for bit."""
    a, b = Sublayer(200, 256, 136, BF, 1, status), Sublayer(33, 1032, 72, BF, 2, status)
    size = max(a.ws.numel(), b.ws.numel())
    a.ws = b.ws = ws_of(size)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a.step(), b.step()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for s in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.step()
        graphs.append(g)
    for seed in (3, 4):
        for s, g in zip((a, b), graphs):
            s.x.copy_(torch.randn(s.x.shape, generator=gen(seed), device="cuda"))
            s.dy.copy_(torch.randn(s.x.shape, generator=gen(seed + 9), device="cuda"))
            s.ws.fill_(0xFF)
        for s, g in zip((a, b), graphs):
            for v in s.outputs().values():
                v.fill_(float("nan"))
            g.replay()
        got = [{k: v.clone() for k, v in s.outputs().items()} for s in (a, b)]
        for s, have in zip((a, b), got):
            s.step()
            for k, v in s.outputs().items():
                assert torch.equal(v, have[k]), k


def test_two_streams_at_once(status):
    """Calls that overlap on two streams, each with a workspace of its own, and repeats: the same bits."""
    a, b = Sublayer(700, 1024, 520, BF, 6, status), Sublayer(5, 2048, 1032, BF, 7, status)
    want = []
    for s in (a, b):
        s.step()
        want.append({k: v.clone() for k, v in s.outputs().items()})
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        for s, st in zip((a, b), streams):
            with torch.cuda.stream(st):
                s.step()
    torch.cuda.synchronize()
    for s, w in zip((a, b), want):
        for k, v in s.outputs().items():
            assert torch.equal(v, w[k]), k


def test_stream_argument(status):
    x, W = ints(gen(1), 40, 64), ints(gen(2), 24, 64)
    y, st = nan_like(40, 24, dtype=BF), torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    moe.moe_linear(x, W, y, status, stream=st)
    st.synchronize()
    assert torch.equal(y, (x.double() @ W.double().t()).to(BF))


# ---------------------------------------------------------------- tensors that no vector fits, and in place

def shifted(t, by=1):
    """t's values `by` elements behind a 512-byte boundary, with guards around."""
    buf = torch.full((t.numel() + by + 16,), 77.0, dtype=t.dtype, device="cuda")
    v = buf[by:by + t.numel()].view(t.shape)
    v.copy_(t)
    return v, buf, by


def untouched(buf, by, n):
    return bool((buf[:by] == 77).all() and (buf[by + n:] == 77).all())


@pytest.mark.parametrize("T,N,K", [(3, 64, 72), (40, 136, 264), (300, 520, 64), (2100, 512, 64)])
@pytest.mark.parametrize("by", [1, 3, 4])
def test_linear_on_unaligned_views(T, N, K, by, status):
    g = gen(T + by)
    x, W = ints(g, T, K), ints(g, N, K)
    bias, res, dy = ints(g, N, lim=9), ints(g, T, N, lim=9), ints(g, T, N, lim=3)
    want = x.double() @ W.double().t() + bias.double()
    (bv, _, _), (rv, _, _), (dv, _, _) = shifted(bias, by), shifted(res, by), shifted(dy, by)
    (yv, yb, _), (sv, sb, _) = shifted(torch.zeros_like(res), by), shifted(torch.zeros_like(res), by)
    moe.moe_linear(x, W, yv, status, bias=bv, residual=rv, act=moe.MOE_ACT_RELU, slope=sv)
    assert torch.equal(yv, (want.clamp_min(0) + res.double()).to(BF)) and torch.equal(sv, (want > 0).to(BF))
    assert untouched(yb, by, T * N) and untouched(sb, by, T * N)
    moe.moe_linear(x, W, rv, status, bias=bv, residual=rv, act=moe.MOE_ACT_RELU)   # in place
    assert torch.equal(rv, yv)
    (dxv, dxb, _), (dWv, dWb, _), (dbv, dbb, _) = shifted(torch.zeros_like(x), by), shifted(torch.zeros_like(W), by), shifted(torch.zeros_like(bias), by)
    moe.moe_linear_bwd(dv, x, W, dxv, dWv, ws_of(moe.moe_linear_bwd_ws_bytes(T, N, K)), status, dbias=dbv, slope=sv)
    d = dy.double() * (want > 0)
    assert torch.equal(dxv, (d @ W.double()).to(BF)) and torch.equal(dWv, (d.t() @ x.double()).to(BF)) and torch.equal(dbv, d.sum(0).to(BF))
    assert untouched(dxb, by, T * K) and untouched(dWb, by, N * K) and untouched(dbb, by, N)


@pytest.mark.parametrize("T,F,H", [(5, 64, 72), (130, 136, 264), (2100, 256, 64)])
def test_gated_on_unaligned_views(T, F, H, status):
    g = gen(T)
    x, W1, dh = ints(g, T, H), ints(g, 2 * F, H, keep=min(1.0, 40 / H)), ints(g, T, F, lim=2)
    gate, up = (x.double() @ W1.double().t()).split(F, 1)
    (hv, hb, by), (fv, fb, _), (dhv, _, _) = shifted(torch.zeros_like(dh)), shifted(torch.zeros(T, 2 * F, dtype=BF, device="cuda")), shifted(dh)
    moe.moe_gated(x, W1, hv, status, act=moe.MOE_ACT_RELU, factors=fv)
    factors = torch.cat((up * (gate > 0), gate.clamp_min(0)), 1)
    assert torch.equal(hv, (gate.clamp_min(0) * up).to(BF)) and torch.equal(fv, factors.to(BF))
    assert untouched(hb, by, T * F) and untouched(fb, by, 2 * T * F)
    f2 = ints(g, T, 2 * F, lim=2)
    fv.copy_(f2)
    dx, dW1 = nan_like(T, H, dtype=BF), nan_like(2 * F, H, dtype=BF)
    moe.moe_gated_bwd(dhv, x, W1, fv, dx, dW1, ws_of(moe.moe_gated_bwd_ws_bytes(T, F, H)), status)
    d = f2.double() * torch.cat((dh, dh), 1).double()
    assert torch.equal(dx, (d @ W1.double()).to(BF)) and torch.equal(dW1, (d.t() @ x.double()).to(BF))


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("T,H", [(1, 33), (7, 1000), (400, 1111), (900, 4096), (5000, 200), (40, 8200), (700, 7168), (2500, 1112), (1200, 1999)])
def test_norm_on_unaligned_views_and_in_place(T, H, dtype):
    """The same values on a view, in place, and aligned: the results agree to the roundings of two orders
    of summation, (H / 16 + 32) 2^-22 of the terms, and one rounding to the type."""
    g = gen(T + H)
    x, dy = (torch.randn(T, H, generator=g, device="cuda") + 0.5).to(dtype), torch.randn(T, H, generator=g, device="cuda").to(dtype)
    w, b = (torch.randn(H, generator=g, device="cuda") * 0.1 + 1).to(dtype), torch.randn(H, generator=g, device="cuda").to(dtype)
    ws = ws_of(moe.moe_layernorm_bwd_ws_bytes(T, H))

    def run(x, dy, y, dx, dw, db):
        mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        keep = x.clone()
        moe.moe_layernorm(x, w, b, EPS, y, mean=mean, rstd=rstd)
        moe.moe_layernorm_bwd(dy, keep, w, mean, rstd, dx, dw, db, ws)
        return [v.double() for v in (y, dx, dw, db)]
    base = run(x, dy, torch.empty_like(x), torch.empty_like(x), torch.empty_like(w), torch.empty_like(w))
    (yv, yb, by), (dv, db_, _) = shifted(x), shifted(dy)
    views = run(shifted(x)[0], shifted(dy)[0], yv, dv, shifted(w)[0], shifted(w)[0])
    assert untouched(yb, by, T * H) and untouched(db_, by, T * H)
    xi, di = x.clone(), dy.clone()
    inplace = run(xi, di, xi, di, torch.empty_like(w), torch.empty_like(w))   # y over x, dx over dy
    u, s = torch.finfo(dtype).eps, (H / 16 + 32) * 2.0 ** -22   # (two roundings to the type, half a step each)
    scale = [6.0, 20.0, 4 * math.sqrt(T) + 8, 4 * math.sqrt(T) + 8]   # of n * w + b, of dx, of sums over rows
    for other in (views, inplace):
        for a, c, size in zip(base, other, scale):
            assert torch.isfinite(c).all()
            assert bool(((a - c).abs() <= u * a.abs() + 64 * s * size + u * torch.finfo(dtype).smallest_normal).all())


@pytest.mark.parametrize("dtype,wdtype", [(BF, F32), (F16, F32), (BF, BF)])
@pytest.mark.parametrize("T,H", [(2, 1), (30, 333), (500, 2048), (4000, 1111), (100, 16384), (6, 16383)])
def test_norm_without_and_with_f32_parameters(T, H, dtype, wdtype):
    """No weight or bias is ones and zeros, bit for bit; f32 parameters of 16-bit values are those values."""
    g = gen(H)
    x, dy = torch.randn(T, H, generator=g, device="cuda").to(dtype), torch.randn(T, H, generator=g, device="cuda").to(dtype)
    one, zero = torch.ones(H, dtype=wdtype, device="cuda"), torch.zeros(H, dtype=wdtype, device="cuda")
    ws = ws_of(moe.moe_layernorm_bwd_ws_bytes(T, H))
    outs = []
    for w, b in ((None, None), (one, zero), (None, zero), (one, None)):
        y, m, r = nan_like(T, H, dtype=dtype), nan_like(T, dtype=F32), nan_like(T, dtype=F32)
        moe.moe_layernorm(x, w, b, EPS, y, mean=m, rstd=r)
        dx, dw, db = nan_like(T, H, dtype=dtype), nan_like(H, dtype=wdtype), nan_like(H, dtype=wdtype)
        moe.moe_layernorm_bwd(dy, x, w, m, r, dx, dw, db, ws)
        only = nan_like(H, dtype=wdtype)
        moe.moe_layernorm_bwd(dy, x, w, m, r, dx, None, only, ws)
        assert torch.equal(only, db)
        moe.moe_layernorm_bwd(dy, x, w, m, r, dx, None, None, ws)
        outs.append((y, m, r, dx, dw, db))
    for o in outs[1:]:
        for a, b in zip(outs[0], o):
            assert torch.equal(a, b)


# ---------------------------------------------------------------- no rows, values that are not finite, long tensors

def test_no_rows(status):
    W, W1 = ints(gen(1), 24, 64), ints(gen(2), 48, 64)
    x, y = torch.empty(0, 64, dtype=BF, device="cuda"), torch.empty(0, 24, dtype=BF, device="cuda")
    ws = ws_of(512)
    moe.moe_linear(x, W, y, status)
    moe.moe_gated(x, W1, y, status)
    moe.moe_layernorm(x, None, None, EPS, torch.empty_like(x))
    dW, dW1, db, dw = (nan_like(*s, dtype=BF) for s in ((24, 64), (48, 64), (24,), (64,)))
    moe.moe_linear_bwd(y, x, W, torch.empty_like(x), dW, ws, status, dbias=db)
    moe.moe_gated_bwd(y, x, W1, torch.empty(0, 48, dtype=BF, device="cuda"), torch.empty_like(x), dW1, ws, status)
    moe.moe_layernorm_bwd(x, x, None, torch.empty(0, device="cuda"), torch.empty(0, device="cuda"), torch.empty_like(x), dw, None, ws)
    for v in (dW, dW1, db, dw):   # sums over no rows
        assert bool((v == 0).all())


@pytest.mark.parametrize("T", [3, 70, 600])
@pytest.mark.parametrize("act", list(ACTS))
def test_values_that_are_not_finite_stay_in_their_rows(T, act, status):
    """A NaN or an infinity in one row of x, or one column's bias, reaches its own outputs alone."""
    g = gen(T)
    x, W, bias = ints(g, T, 64), ints(g, 200, 64), torch.zeros(200, dtype=BF, device="cuda")
    clean, slope = nan_like(T, 200, dtype=BF), nan_like(T, 200, dtype=BF)
    moe.moe_linear(x, W, clean, status, bias=bias, act=ACTS[act])
    xb, bb = x.clone(), bias.clone()
    xb[1, 5], xb[2, 9], bb[7] = float("nan"), float("inf"), float("nan")
    y = nan_like(T, 200, dtype=BF)
    moe.moe_linear(xb, W, y, status, bias=bb, act=ACTS[act], slope=slope)
    rows = [t for t in range(T) if t not in (1, 2)]
    cols = [c for c in range(200) if c != 7]
    assert torch.equal(y[rows][:, cols], clean[rows][:, cols])
    assert y[1].isnan().all() and y[:, 7].isnan().all()
    norm = nan_like(T, 64, dtype=BF)
    moe.moe_layernorm(xb, None, None, EPS, norm)
    assert norm[1].isnan().all() and norm[2].isnan().all() and torch.isfinite(norm[rows].float()).all()


@pytest.mark.parametrize("act", list(ACTS))
def test_activations_far_out(act, status):
    """From -6e4 to 6e4 (and their slopes): finite, and within the activation's bound of the formula.  Far below
    zero, where values vanish, gelu's are still within 2^-15 of themselves down to the type's smallest normal."""
    a = torch.cat((torch.linspace(-30, 30, 4001), torch.tensor([-6e4, -1e3, -100.0, 100.0, 1e3, 6e4]))).to(BF).cuda()
    x, W = a[:, None].repeat(1, 8).contiguous(), torch.zeros(8, 8, dtype=BF, device="cuda")
    x[:, 1:] = 0
    W[:, 0] = 1
    y, slope = nan_like(a.numel(), 8, dtype=BF), nan_like(a.numel(), 8, dtype=BF)
    moe.moe_linear(x, W, y, status, act=ACTS[act], slope=slope)
    want, ws = act64(a.double(), act)
    if act == "gelu_tanh":   # 1 + tanh(z) cancels far below zero (it is off by 2^-53): 2 / (1 + exp(-2 z)) does not
        v = a.double()
        z, dz = 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3), 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * v * v)
        want, ws = v * torch.sigmoid(z), torch.sigmoid(z) + v * torch.sigmoid(z) * torch.sigmoid(-z) * dz
    u, tiny = torch.finfo(BF).eps / 2, 2.0 ** -120
    # exp's argument (up to 88 where the value is not 0) is off by three roundings of it, at most min(a^2, 200) 2^-22,
    # beside 2^-18 of the value
    e = 2.0 ** -18 + (a.double() ** 2).clamp_max(200) * 2.0 ** -22
    for got, w, size in ((y[:, 0], want, want.abs()), (slope[:, 0], ws, ws.abs() + (a.double().abs() + 1) * 2.0 ** -18 * (ws.abs() < 0.01))):
        assert torch.isfinite(got.float()).all()
        assert bool(((got.double() - w).abs() <= u * w.abs() * 1.01 + e * size + tiny).all())


def test_past_2_31_elements(status):
    """Rows whose elements lie beyond 2^31: their outputs and gradients are those of the same rows alone."""
    T, N, K = (1 << 18) + 3, 8328, 8
    g = gen(1)
    x, W, dy = ints(g, T, K), ints(g, N, K), None
    y = torch.empty(T, N, dtype=BF, device="cuda")
    assert y.numel() > 1 << 31
    moe.moe_linear(x, W, y, status)
    tail = slice(T - 300, T)
    assert torch.equal(y[tail], (x[tail].double() @ W.double().t()).to(BF))
    y.sign_()
    dx, ws = nan_like(T, K, dtype=BF), ws_of(256)
    with pytest.raises(moe.MoEError):
        moe.moe_linear_bwd(y, x, W, dx, None, ws, status)   # (the workspace of padded rows is short)
    del ws
    ws = ws_of(moe.moe_linear_bwd_ws_bytes(T, N, K))
    moe.moe_linear_bwd(y, x, W, dx, None, ws, status)
    assert torch.equal(dx[tail], (y[tail].double() @ W.double()).to(BF))
    del ws, dy
    out, mean, rstd = torch.empty_like(y), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    moe.moe_layernorm(y, None, None, EPS, out, mean=mean, rstd=rstd)
    small = nan_like(300, N, dtype=BF)
    moe.moe_layernorm(y[tail].clone(), None, None, EPS, small)
    # (few rows take another kernel: two orders of summation, one rounding of values up to 100)
    assert bool(((out[tail].float() - small.float()).abs() <= torch.finfo(BF).eps * small.float().abs() + 1e-4).all())


def test_repeats_bit_for_bit(status):
    s = Sublayer(1111, 1024, 336, BF, 12, status)
    s.step()
    want = {k: v.clone() for k, v in s.outputs().items()}
    for _ in range(5):
        s.ws.fill_(0xFF)
        s.step()
        for k, v in s.outputs().items():
            assert torch.equal(v, want[k]), k


# ---------------------------------------------------------------- in the decoding example, and a short workspace

def test_decoding_with_a_shared_expert_in_bf16():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, os.path.join(root, "examples", "decode_moe.py"), "--shared", "bf16", "--tokens", "3", "--steps", "4",
                        "--hidden", "256", "--ffn", "128", "--experts", "16", "--topk", "4", "--vocab", "512"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "3 sequences x 4 steps" in r.stdout


def test_refused_on_the_gpu(status):
    x, W, y = ints(gen(1), 40, 64), ints(gen(2), 24, 64), torch.empty(40, 24, dtype=BF, device="cuda")
    ws = ws_of(moe.moe_linear_bwd_ws_bytes(40, 24, 64))
    with pytest.raises(ValueError, match="contiguous"):
        moe.moe_linear(x.t().contiguous().t(), W, y, status)
    with pytest.raises(ValueError, match="status must be torch.int32"):
        moe.moe_linear(x, W, y, status.float())
    with pytest.raises(ValueError, match="bias must be torch.bfloat16"):
        moe.moe_linear(x, W, y, status, bias=torch.zeros(24, device="cuda"))
    with pytest.raises(ValueError, match="ws must be a CUDA tensor"):
        moe.moe_linear_bwd(y, x, W, None, None, torch.empty(1 << 16, dtype=torch.uint8), status)
    with pytest.raises(moe.MoEError, match="INVALID_ARG"):
        moe.moe_linear_bwd(y, x, W, torch.empty_like(x), None, ws[:-256].clone()[:256], status, slope=y)
    with pytest.raises(moe.MoEError, match="INVALID_ARG"):   # operands of a product start on 16 bytes
        moe.moe_linear(shifted(x)[0], W, y, status)
    with pytest.raises(moe.MoEError, match="INVALID_ARG"):   # and a contraction is a multiple of 8
        moe.moe_linear(x[:, :63].contiguous(), W[:, :63].contiguous(), y, status)
