"""The decoding operators on values and sizes where they can go wrong."""
import numpy as np
import pytest
import torch

import combine_counting_sort_gb300 as moe
import oracle
from tests.gpu_util import build
from tests.test_gpu_few import GROUPS, Experts, bf16_t, f64, rand_bits, routes, status, w4_matrix, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()


# ---------------------------------------------------------------- weights that are not finite

def spoil(ex, e, which, how):
    """NaN codes (FP8), or infinite or NaN scales, in one row block of expert e's matrix."""
    W, scale = (ex.W1, ex.W1_scale) if which == 1 else (ex.W2, ex.W2_scale)
    if ex.group == 0:
        if how == "code":
            W[e, 5, 7] = 0x7F
        else:
            scale[e, 0, 0] = float(how)
    else:
        bits = torch.tensor([float(how)], dtype=torch.bfloat16).view(torch.uint8).cuda()
        W[e, 0, 0, 1024:1026] = bits                         # the scale of row 0 and the first group


@pytest.mark.parametrize("T", [2, 5, 8, 9, 12])
@pytest.mark.parametrize("which", [1, 2])
@pytest.mark.parametrize("group,how", [(0, "code"), (0, "inf"), (0, "nan"), (32, "inf"), (64, "nan"), (128, "inf")])
def test_layer_weights_that_are_not_finite_reach_their_own_tokens_alone(group, how, which, T):
    # token 1 alone uses expert 3; the other tokens keep their bits at every batch size
    E, k, H, F = 6, 2, 256, 256
    ex = Experts(E, H, F, group, seed=T)
    ids, w = routes(T, k, 3, seed=T)
    ids[1] = 3, 4
    xb = rand_bits(T, H, seed=T + 1)
    clean, _, _ = ex.run(xb, ids, w)
    spoil(ex, 3, which, how)
    out, _, _ = ex.run(xb, ids, w)
    keep = [t for t in range(T) if t != 1]
    assert torch.equal(out[keep].view(torch.int16), clean[keep].view(torch.int16))
    assert not torch.isfinite(out[1]).all()


# ---------------------------------------------------------------- large values that meet weights of zero

def run_matvec(xb, Wp, N, group):
    y, st = torch.full((len(xb), N), float("nan"), dtype=torch.bfloat16, device="cuda"), status()
    moe.moe_matvec_w4(bf16_t(xb), Wp, group, y, st)
    torch.cuda.synchronize()
    assert st.item() == 0
    return y


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,N,K", [(1, 48, 1024), (1, 5000, 256), (2, 48, 2048), (4, 33, 512), (7, 48, 1024), (20, 48, 1024)])
def test_matvec_large_values_on_zero_weights(T, N, K, group):
    # some columns' weights are zero (code 8) and their values 2^20 of either sign: the bound is that of
    # what the other columns add up to
    b = rand_bits(1, N, K, seed=T + N, scale=K ** -0.5)
    at = np.arange(5, K, 97)
    b[..., at] = 0
    q, s = oracle.quantize_w4(b, group)
    assert np.all(q[..., at] == 8)
    x = f64(rand_bits(T, K, seed=K))
    x[:, at] = np.where(np.arange(len(at)) % 2, 1.0, -1.0) * 2.0 ** 20
    xb = oracle.f64_to_bf16(x)
    y = run_matvec(xb, torch.from_numpy(oracle.pack_w4(q, s)[0]).cuda(), N, group)
    within(y, *oracle.matvec_bound(f64(xb), oracle.w4_values(q, s)[0]), "matvec")


@pytest.mark.parametrize("T", [1, 4, 7, 20])
def test_matvec_small_results(T):
    # results near 2^-120, bf16's normal values end at 2^-126
    N, K, group = 48, 512, 32
    Wp, W = w4_matrix(N, K, group, seed=T, scale=2.0 ** -100)
    xb = rand_bits(T, K, seed=T, scale=2.0 ** -24)
    within(run_matvec(xb, Wp, N, group), *oracle.matvec_bound(f64(xb), W), "matvec")


def experts_of(b1, b2, group):
    ex = Experts.__new__(Experts)
    ex.E, ex.H, ex.F, ex.group, ex.W1_scale, ex.W2_scale = b1.shape[0], b1.shape[2], b2.shape[2], group, None, None
    (q1, s1), (q2, s2) = oracle.quantize_w4(b1, group), oracle.quantize_w4(b2, group)
    ex.W1, ex.W2 = (torch.from_numpy(oracle.pack_w4(*v)).cuda() for v in ((q1, s1), (q2, s2)))
    ex.values = {e: (oracle.w4_values(q1[e], s1[e]), oracle.w4_values(q2[e], s2[e])) for e in range(ex.E)}
    return ex


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T", [1, 6, 12, 40])
def test_layer_large_values_on_zero_weights(T, group):
    # columns of x at 2^20 whose gate and up weights are zero; features whose activations are 2^20
    # times the others' and whose down weights are zero
    E, k, H, F = 4, 2, 512, 256
    b1, b2 = rand_bits(E, 2 * F, H, seed=1, scale=H ** -0.5), rand_bits(E, H, F, seed=2, scale=F ** -0.5)
    at, feature = np.arange(3, H, 61), np.arange(7, F, 71)
    b1[..., at] = 0
    up = f64(b1)
    up[:, F + feature] *= 2.0 ** 20
    b1, b2[..., feature] = oracle.f64_to_bf16(up), 0
    ex = experts_of(b1, b2, group)
    x = f64(rand_bits(T, H, seed=T))
    x[:, at] = np.where(np.arange(len(at)) % 2, 1.0, -1.0) * 2.0 ** 20
    xb = oracle.f64_to_bf16(x)
    ids, w = routes(T, k, E, seed=T)
    out, _, _ = ex.run(xb, ids, w)
    within(out, *oracle.layer_few(f64(xb), ids, w, ex.values), "layer")


# ---------------------------------------------------------------- row tiles of a down item, fullest segments

def capped_routes(T, k, E, cap, seed):
    """Routes of which expert 0 has exactly `cap` tokens and no other more."""
    rng = np.random.default_rng(seed)
    ids, left = np.zeros((T, k), np.int32), np.full(E, cap)
    ids[:], at = -1, rng.permutation(T)
    ids[at[:cap], 0] = 0
    for t in range(T):
        free = [j for j in range(k) if ids[t, j] < 0]
        order = 1 + np.argsort(-left[1:] + rng.random(E - 1))[:len(free)]
        assert np.all(left[order] > 0)
        left[order] -= 1
        ids[t, free] = order
    assert np.bincount(ids.ravel(), minlength=E).max() == cap
    return ids, (rng.random((T, k)) + 0.1).astype(np.float32)


_experts = {}


def experts(E, H, F, group):
    if (E, H, F, group) not in _experts:
        _experts.clear()
        _experts[E, H, F, group] = Experts(E, H, F, group, seed=11)
    return _experts[E, H, F, group]


# H 2560: two row tiles to a down item on 152 SMs, 7040: three, and two in the last item.  Experts with 8
# tokens and fewer (one block of columns, two slices a warp), 9 and 16 (two blocks), 25 (two segments);
# a token's sums over several experts, one that it names twice, slots without a route.
@pytest.mark.parametrize("T,k,cap", [(3, 4, 3), (8, 3, 8), (9, 4, 8), (33, 4, 9), (33, 4, 16), (64, 2, 8), (64, 4, 25)])
@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("H", [2560, 7040])
def test_layer_row_tiles_of_a_down_item(H, group, T, k, cap):
    E, F = 17, 128
    ex = experts(E, H, F, group)
    ids, w = capped_routes(T, k, E, cap, seed=T + cap)
    ids[1, 1], ids[2, 0] = ids[1, 0], -1
    xb = rand_bits(T, H, seed=T)
    out, _, _ = ex.run(xb, ids, w)
    within(out, *oracle.layer_few(f64(xb), ids, w, ex.values), "layer")
    again, _, _ = ex.run(xb, ids, w)
    assert torch.equal(again, out)


@pytest.mark.parametrize("group", GROUPS)
def test_layer_one_buffer_of_sums(group):
    # 1024 pairs, most of them without a route: the tables leave two stages beside one buffer alone
    T, E, H, F, cap = 64, 17, 7040, 128, 8
    ex = experts(E, H, F, group)
    few, w2 = capped_routes(T, 2, E, cap, seed=5)
    ids, w = np.full((T, 16), -1, np.int32), np.full((T, 16), np.nan, np.float32)
    ids[:, [3, 15]], w[:, [3, 15]] = few, w2
    xb = rand_bits(T, H, seed=6)
    out, _, _ = ex.run(xb, ids, w)
    within(out, *oracle.layer_few(f64(xb), few, w2, ex.values), "layer")


@pytest.mark.parametrize("T,cap", [(57, 16), (64, 25)])
def test_layer_narrow_segments(T, cap):
    # FP8 weights, three row tiles and about 1000 pairs: segments of 15 tokens
    E, k, H, F = 48, 16, 7168, 128
    ex = experts(E, H, F, 0)
    ids, w = capped_routes(T, k, E, cap, seed=T) if cap == 25 else capped_routes(T, 16, 64, cap, seed=T)
    ids = np.where(ids >= E, -1, ids)
    xb = rand_bits(T, H, seed=T)
    out, _, _ = ex.run(xb, ids, w)
    within(out, *oracle.layer_few(f64(xb), ids, w, ex.values), "layer")


@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("T", [3, 21])
def test_layer_activations_keep_eleven_bits(T, group):
    # one weight in each row of W2, so that no activation's rounding is averaged out
    E, H, F = 2, 256, 256
    b1, rng = rand_bits(E, 2 * F, H, seed=T, scale=H ** -0.5), np.random.default_rng(T)
    b2 = np.zeros((E, H, F), np.uint16)
    for e in range(E):
        b2[e, np.arange(H), rng.permutation(F)] = 0x3F30
    ex = experts_of(b1, b2, group) if group else fp8_experts_of(b1, b2)
    xb = rand_bits(T, H, seed=T + 1)
    ids, w = routes(T, 1, E, seed=T)
    out, _, _ = ex.run(xb, ids, w)
    within(out, *oracle.layer_few(f64(xb), ids, w, ex.values), "layer")


def fp8_experts_of(b1, b2):
    ex = Experts.__new__(Experts)
    ex.E, ex.H, ex.F, ex.group = b1.shape[0], b1.shape[2], b2.shape[2], 0
    (q1, s1), (q2, s2) = oracle.quantize_weights(b1), oracle.quantize_weights(b2)
    ex.W1, ex.W1_scale, ex.W2, ex.W2_scale = (torch.from_numpy(v).cuda() for v in (q1, s1, q2, s2))
    ex.values = {e: (oracle.fp8_values(q1[e], s1[e]), oracle.fp8_values(q2[e], s2[e])) for e in range(ex.E)}
    return ex
