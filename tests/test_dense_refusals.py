"""What the dense operators refuse, without a GPU: tensors that are not as a
call's sizes imply (ValueError), and the C entry points' own limits, types and
alignments, which are checked before anything is launched."""
import ctypes

import pytest
import torch

import combine_counting_sort_gb300 as moe

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from combine_counting_sort_gb300 import _build
    _build.build()


def t(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


STATUS = torch.zeros(1, dtype=torch.int32)
WS = torch.zeros(1 << 16, dtype=torch.uint8)


def linear(x=(3, 8), W=(5, 8), y=(3, 5), status=STATUS, **kw):
    conv = {k: (v if isinstance(v, (torch.Tensor, int)) else t(*v)) for k, v in dict(x=x, W=W, y=y, **kw).items()}
    moe.moe_linear(conv.pop("x"), conv.pop("W"), conv.pop("y"), status, **conv)


BAD_LINEAR = [
    (dict(W=(5, 16)), "W must have shape"), (dict(y=(3, 6)), "y must have shape"), (dict(y=(4, 5)), "y must have shape"),
    (dict(bias=(6,)), "bias must have shape"), (dict(bias=(1, 5)), "bias must have shape"), (dict(residual=(5, 3)), "residual must have shape"),
    (dict(slope=(3, 8)), "slope must have shape"), (dict(x=(8,)), "x must have 2 dimensions"), (dict(W=(5, 8, 1)), "W must have 2 dimensions"),
    (dict(status=torch.zeros(0, dtype=torch.int32)), "status must hold"), (dict(x=t(3, 8, dtype=F32)), "x must be one of"),
    (dict(x=t(3, 8, dtype=torch.int32)), "x must be one of"), ({}, "must be a CUDA tensor"),
]


@pytest.mark.parametrize("kw,msg", BAD_LINEAR)
def test_linear_refuses(kw, msg):
    with pytest.raises(ValueError, match=msg):
        linear(**kw)


@pytest.mark.parametrize("call", [
    lambda: moe.moe_linear(None, t(5, 8), t(3, 5), STATUS), lambda: moe.moe_linear(t(3, 8), t(5, 8), t(3, 5), None),
    lambda: moe.moe_linear(t(3, 8), [1], t(3, 5), STATUS), lambda: moe.moe_gated(t(3, 8), t(10, 8), None, STATUS),
    lambda: moe.moe_layernorm(t(3, 8), None, None, "eps", t(3, 8)), lambda: moe.moe_linear(t(3, 8), t(5, 8), t(3, 5), STATUS, act="gelu")])
def test_refuses_what_is_no_tensor(call):
    with pytest.raises(TypeError):
        call()


@pytest.mark.parametrize("call,msg", [
    (lambda: moe.moe_gated(t(3, 8), t(9, 8), t(3, 5), STATUS), "W1 must have shape"),
    (lambda: moe.moe_gated(t(3, 8), t(10, 8), t(4, 5), STATUS), "h must have shape"),
    (lambda: moe.moe_gated(t(3, 8), t(10, 8), t(3, 5), STATUS, factors=t(3, 5)), "factors must have shape"),
    (lambda: moe.moe_gated_bwd(t(3, 5), t(3, 8), t(10, 8), t(3, 10), t(3, 8), t(5, 8), WS, STATUS), "dW1 must have shape"),
    (lambda: moe.moe_gated_bwd(t(3, 5), t(3, 8), t(10, 8), t(3, 9), None, None, WS, STATUS), "factors must have shape"),
    (lambda: moe.moe_linear_bwd(t(3, 5), t(3, 8), t(5, 8), t(3, 5), None, WS, STATUS), "dx must have shape"),
    (lambda: moe.moe_linear_bwd(t(3, 6), t(3, 8), t(5, 8), None, None, WS, STATUS), "dy must have shape"),
    (lambda: moe.moe_linear_bwd(t(3, 5), t(3, 8), t(5, 8), None, None, WS, STATUS, dbias=t(8)), "dbias must have shape"),
    (lambda: moe.moe_layernorm(t(3, 8), t(7), None, 1e-5, t(3, 8)), "weight must have shape"),
    (lambda: moe.moe_layernorm(t(3, 8), t(8), t(8, 1), 1e-5, t(3, 8)), "bias must have shape"),
    (lambda: moe.moe_layernorm(t(3, 8), t(8, dtype=F16), None, 1e-5, t(3, 8)), "weight and bias must be"),
    (lambda: moe.moe_layernorm(t(3, 8, dtype=F32), t(8), None, 1e-5, t(3, 8, dtype=F32)), "weight and bias must be"),
    (lambda: moe.moe_layernorm(t(3, 8), None, None, 1e-5, t(3, 8), mean=t(4, dtype=F32)), "mean must have shape"),
    (lambda: moe.moe_layernorm(t(3, 8, dtype=torch.float64), None, None, 1e-5, t(3, 8)), "x must be one of"),
    (lambda: moe.moe_layernorm_bwd(t(3, 8), t(3, 8), None, t(3, dtype=F32), t(2, dtype=F32), t(3, 8), None, None, WS), "rstd must have shape"),
    (lambda: moe.moe_layernorm_bwd(t(3, 8), t(3, 8), t(8), t(3, dtype=F32), t(3, dtype=F32), t(8, 3), None, None, WS), "dx must have shape")])
def test_refuses_shapes_and_types(call, msg):
    with pytest.raises(ValueError, match=msg):
        call()


# ---------------------------------------------------------------- the C entry points

INVALID = moe.MOE_ERR_INVALID_ARG
A = 1 << 20   # an address that nothing reads: each call below is refused first


def test_c_linear():
    def call(x=A, T=4, K=64, W=A, N=8, dtype=moe.MOE_BF16, bias=None, res=None, act=0, y=A, slope=None):
        return moe.lib().moe_linear(x, T, K, W, N, dtype, bias, res, act, y, slope, A, None)
    for kw in (dict(T=-1), dict(T=(1 << 24) + 1), dict(K=0), dict(K=4), dict(K=12), dict(K=(1 << 20) + 8), dict(N=0), dict(N=(1 << 20) + 1),
               dict(dtype=moe.MOE_F32), dict(dtype=-1), dict(dtype=3), dict(act=-1), dict(act=5), dict(x=None), dict(W=None), dict(y=None),
               dict(x=A + 8), dict(W=A + 2), dict(y=A + 1), dict(bias=A + 1), dict(res=A + 1), dict(slope=A + 1)):
        assert call(**kw) == INVALID, kw
    assert call(T=0, x=None, W=None, y=None) == moe.MOE_OK   # no rows: nothing is read or written


def test_c_linear_bwd():
    need = moe.moe_linear_bwd_ws_bytes(4, 9, 64)
    assert need == 4 * 16 * 2

    def call(dy=A, x=A, T=4, K=64, W=A, N=9, dtype=moe.MOE_F16, slope=None, dx=A, dW=A, db=None, ws=A, n=need):
        return moe.lib().moe_linear_bwd(dy, x, T, K, W, N, dtype, slope, dx, dW, db, ws, n, A, None)
    for kw in (dict(T=-1), dict(K=12), dict(N=0), dict(dtype=moe.MOE_F32), dict(dy=None), dict(dy=A + 1), dict(slope=A + 1), dict(ws=None),
               dict(ws=A + 16), dict(n=need - 1), dict(n=0), dict(W=None), dict(x=None), dict(W=A + 8), dict(x=A + 2), dict(dx=A + 1), dict(dW=A + 1),
               dict(db=A + 1)):
        assert call(**kw) == INVALID, kw
    assert call(dx=None, dW=None) == moe.MOE_OK          # nothing wanted
    assert call(T=0, dW=None) == moe.MOE_OK
    for bad in ((-1, 8, 8), (1, 0, 8), (1, 8, 12)):
        with pytest.raises(moe.MoEError):
            moe.moe_linear_bwd_ws_bytes(*bad)


def test_c_gated():
    def call(x=A, T=4, H=64, W1=A, F=8, dtype=moe.MOE_BF16, act=2, h=A, factors=None):
        return moe.lib().moe_gated(x, T, H, W1, F, dtype, act, h, factors, A, None)
    for kw in (dict(T=-1), dict(H=60), dict(H=0), dict(F=0), dict(F=-3), dict(F=(1 << 19) + 1), dict(dtype=2), dict(act=9), dict(x=None), dict(W1=None),
               dict(h=None), dict(x=A + 4), dict(W1=A + 8), dict(h=A + 1), dict(factors=A + 1)):
        assert call(**kw) == INVALID, kw
    assert call(T=0, x=None) == moe.MOE_OK
    need = moe.moe_gated_bwd_ws_bytes(4, 9, 64)

    def back(dh=A, x=A, T=4, H=64, W1=A, F=9, dtype=moe.MOE_BF16, factors=A, dx=A, dW1=A, ws=A, n=need):
        return moe.lib().moe_gated_bwd(dh, x, T, H, W1, F, dtype, factors, dx, dW1, ws, n, A, None)
    for kw in (dict(T=-1), dict(H=60), dict(F=0), dict(dtype=2), dict(dh=None), dict(factors=None), dict(dh=A + 1), dict(ws=None), dict(ws=A + 128),
               dict(n=need - 1), dict(W1=None), dict(x=None), dict(x=A + 8), dict(dx=A + 1), dict(dW1=A + 1)):
        assert back(**kw) == INVALID, kw
    assert back(dx=None, dW1=None) == moe.MOE_OK


def test_c_layernorm():
    def call(x=A, T=4, H=64, dtype=moe.MOE_BF16, w=A, b=None, wdtype=moe.MOE_BF16, eps=1e-5, y=A, mean=None, rstd=None):
        return moe.lib().moe_layernorm(x, T, H, dtype, w, b, wdtype, eps, y, mean, rstd, None)
    for kw in (dict(T=-1), dict(H=0), dict(H=16385), dict(dtype=3), dict(wdtype=moe.MOE_F16), dict(dtype=moe.MOE_F32), dict(eps=-1e-5),
               dict(eps=float("nan")), dict(x=None), dict(y=None), dict(x=A + 1), dict(y=A + 1), dict(w=A + 1), dict(b=A + 1), dict(mean=A + 2),
               dict(rstd=A + 1), dict(dtype=moe.MOE_F32, wdtype=moe.MOE_F32, x=A + 2)):
        assert call(**kw) == INVALID, kw
    assert call(T=0, x=None, y=None) == moe.MOE_OK
    need = moe.moe_layernorm_bwd_ws_bytes(4, 64)

    def back(dy=A, x=A, T=4, H=64, dtype=moe.MOE_BF16, w=A, wdtype=moe.MOE_BF16, mean=A, rstd=A, dx=A, dw=A, db=A, ws=A, n=need):
        return moe.lib().moe_layernorm_bwd(dy, x, T, H, dtype, w, wdtype, mean, rstd, dx, dw, db, ws, n, None)
    for kw in (dict(T=-1), dict(H=0), dict(H=16385), dict(dtype=-1), dict(wdtype=moe.MOE_F16), dict(dy=None), dict(x=None), dict(mean=None),
               dict(rstd=None), dict(dx=None), dict(ws=None), dict(ws=A + 8), dict(n=need - 1), dict(dw=A + 1), dict(mean=A + 2), dict(dy=A + 1)):
        assert back(**kw) == INVALID, kw


def test_sizes_beyond_an_int():
    out = ctypes.c_size_t()
    assert moe.lib().moe_linear_bwd_ws_bytes(1 << 24, 1 << 20, 8, ctypes.byref(out)) == moe.MOE_OK
    assert out.value == (1 << 24) * (1 << 20) * 2
    assert moe.lib().moe_layernorm_bwd_ws_bytes(1 << 30, 16384, ctypes.byref(out)) == moe.MOE_OK
    with pytest.raises(ValueError, match="too large"):
        moe.moe_linear(torch.empty(1, 1 << 32, device="meta", dtype=BF), t(5, 8), t(3, 5), STATUS)
