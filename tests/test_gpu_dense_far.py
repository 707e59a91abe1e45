"""The dense operators' activations on values as large as bf16 holds, and on NaN: what an outlier in the sums
leaves of the output and of the slope."""
import pytest
import torch

import combine_counting_sort_gb300 as moe
from tests import gpu_util
from tests.test_gpu_dense import ACTS, nan_like

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gpu_util.build()


@pytest.fixture
def status():
    s = torch.zeros(1, dtype=torch.int32, device="cuda")
    yield s
    torch.cuda.synchronize()
    assert s.item() == 0, moe.status_string(s.item())


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("T,N", [(12, 8), (12, 13), (4096, 2048), (4096, 2047)])
def test_outliers(T, N, act, status):
    """From 100 on every activation is the value itself with slope 1, from -100 on 0 with slope 0 (none: the
    value and 1), up to the largest bf16 value: a^2 overflows in fp32 from 1.8e19 on, and nothing may come of that."""
    a = torch.tensor([100.0, 1e4, 1e10, 1.5e19, 2e19, 3e38], device="cuda").to(BF)
    a = torch.cat((a, -a)).repeat((T + 11) // 12)[:T]
    x, W = torch.zeros(T, 8, dtype=BF, device="cuda"), torch.zeros(N, 8, dtype=BF, device="cuda")
    x[:, 0], W[:, 0] = a, 1
    y, slope = nan_like(T, N, dtype=BF), nan_like(T, N, dtype=BF)
    moe.moe_linear(x, W, y, status, act=ACTS[act], slope=slope)
    on = torch.ones_like(a) if act == "none" else (a > 0).to(BF)
    assert torch.equal(y, (a * on)[:, None].expand(T, N))
    assert torch.equal(slope, on[:, None].expand(T, N))

    # gated: up sums of 1, so that h is the activation and the factors are its slope and itself
    x[:, 1] = 1
    W1 = torch.cat((W, torch.zeros_like(W)))
    W1[N:, 1] = 1
    h, factors = nan_like(T, N, dtype=BF), nan_like(T, 2 * N, dtype=BF)
    moe.moe_gated(x, W1, h, status, act=ACTS[act], factors=factors)
    assert torch.equal(h, (a * on)[:, None].expand(T, N))
    assert torch.equal(factors, torch.cat((on[:, None].expand(T, N), (a * on)[:, None].expand(T, N)), 1))


@pytest.mark.parametrize("act", [a for a in ACTS if a != "none"])
@pytest.mark.parametrize("T", [12, 4096])
def test_nan_is_in_the_slope_too(T, act, status):
    """The slope at a sum that is NaN is NaN, as the output is, so that the gradients say so; the rows beside it are untouched."""
    x, W = torch.ones(T, 8, dtype=BF, device="cuda"), torch.ones(2048, 8, dtype=BF, device="cuda")
    x[5, 3] = float("nan")
    rows = [t for t in range(T) if t != 5]
    y, slope = nan_like(T, 2048, dtype=BF), nan_like(T, 2048, dtype=BF)
    moe.moe_linear(x, W, y, status, act=ACTS[act], slope=slope)
    assert y[5].isnan().all() and slope[5].isnan().all()
    assert torch.isfinite(y[rows].float()).all() and torch.isfinite(slope[rows].float()).all()
    h, factors = nan_like(T, 1024, dtype=BF), nan_like(T, 2048, dtype=BF)
    moe.moe_gated(x, W, h, status, act=ACTS[act], factors=factors)
    assert h[5].isnan().all() and factors[5].isnan().all()
    assert torch.isfinite(h[rows].float()).all() and torch.isfinite(factors[rows].float()).all()
