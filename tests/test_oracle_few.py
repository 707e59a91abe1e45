"""The decoding operators' oracle against its own definition, and the binding's
refusals that need no GPU."""
import ctypes

import numpy as np
import pytest
import torch

import combine_counting_sort_gb300 as moe
import oracle
from combine_counting_sort_gb300 import inputs


@pytest.fixture(scope="module")
def lib():
    from combine_counting_sort_gb300 import _build
    _build.build()
    return moe.lib()


def rand_bits(*shape, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return inputs.bf16_bits((torch.randn(*shape, generator=g) * scale).to(torch.bfloat16))


@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantize_w4_is_the_nearest_code(group):
    bits = rand_bits(9, 256, seed=group)
    bits[3, :group] = 0
    q, s = oracle.quantize_w4(bits, group)
    w, sv = oracle.bf16_to_f32(bits).astype(np.float64), oracle.bf16_to_f32(s).astype(np.float64)
    assert q.max() <= 15 and np.all(q[3, :group] == 8) and s[3, 0] == 0
    amax = np.abs(w).reshape(9, -1, group).max(-1)
    assert np.all(np.abs(sv - amax / 7) <= amax / 7 * 2.0 ** -8)
    v = oracle.w4_values(q, s)
    # no other code is nearer, and nothing within the range is further than half a step
    step = np.repeat(sv, group, -1)
    for d in (-1, 1):
        other = np.clip(q.astype(int) + d, 0, 15)
        assert np.all(np.abs(v - w) <= np.abs((other - 8) * step - w) + 1e-12)


@pytest.mark.parametrize("N,K,group", [(16, 128, 128), (17, 160, 32), (5, 192, 64), (40, 384, 128)])
def test_pack_w4_places_every_code_and_scale(N, K, group):
    rng = np.random.default_rng(N)
    codes = rng.integers(0, 16, (2, N, K), dtype=np.uint8)
    scale = rng.integers(0, 1 << 15, (2, N, K // group), dtype=np.uint16)
    packed = oracle.pack_w4(codes, scale)
    assert packed.shape == tuple(moe.w4_packed_shape(2, N, K, group))
    # read back through (word >> 4p) & 0x000F000F, the pair of columns 2p and 2p + 1
    words = packed[..., :1024].copy().view("<u4").reshape(2, packed.shape[1], packed.shape[2], 2, 8, 4, 4)
    back = np.full((2, packed.shape[1] * 16, packed.shape[2] * 128), 99, np.uint8)
    for half in range(2):
        for g in range(8):
            for t in range(4):
                for j in range(4):
                    for p in range(4):
                        pair = (words[:, :, :, half, g, t, j] >> (4 * p)) & 0x000F000F
                        c = 32 * j + 8 * t + 2 * p
                        back[:, 8 * half + g::16, c::128] = pair & 0xFFFF
                        back[:, 8 * half + g::16, c + 1::128] = pair >> 16
    assert np.array_equal(back[:, :N, :K], codes)
    assert np.all(back[:, N:] == 8) and np.all(back[:, :, K:] == 8)


def test_layer_oracle_is_the_plain_loop():
    rng = np.random.default_rng(5)
    T, H, F = 3, 8, 4
    ids = np.array([[1, 0], [0, 0], [-1, 7]])
    w = rng.random((T, 2))
    ex = {e: (rng.standard_normal((2 * F, H)), rng.standard_normal((H, F))) for e in range(2)}
    x = rng.standard_normal((T, H))
    out, bound = oracle.layer_few(x, ids, w, ex)
    want = np.zeros((T, H))
    for t in range(T):
        for j in range(2):
            if ids[t, j] in ex:
                W1, W2 = ex[ids[t, j]]
                for h in range(H):
                    for f in range(F):
                        g, u = W1[f] @ x[t], W1[F + f] @ x[t]
                        want[t, h] += w[t, j] * W2[h, f] * g / (1 + np.exp(-g)) * u
    assert np.allclose(out, want, rtol=1e-12, atol=1e-14)
    assert np.all(out[2] == 0) and np.all(bound >= 0)


def test_sizes_and_refusals_without_a_gpu(lib):
    n = ctypes.c_size_t()
    assert lib.moe_w4_packed_bytes(17, 160, 32, ctypes.byref(n)) == moe.MOE_OK
    assert n.value == 2 * 2 * (1024 + 128) == int(np.prod(moe.w4_packed_shape(1, 17, 160, 32)))
    for N, K, g in [(0, 128, 128), (16, 0, 32), (16, 100, 32), (16, 128, 16), (16, 64, 128), (16, 65536, 128), ((1 << 20) + 1, 128, 128)]:
        assert lib.moe_w4_packed_bytes(N, K, g, ctypes.byref(n)) == moe.MOE_ERR_INVALID_ARG, (N, K, g)
    assert moe.moe_layer_few_ws_bytes(64, 16, 256, 256, 128) >= 256
    for T, k, E, H, F in [(0, 1, 8, 256, 128), (65, 1, 8, 256, 128), (64, 17, 64, 256, 128), (4, 9, 8, 256, 128), (4, 33, 64, 256, 128),
                          (4, 2, 1025, 256, 128), (4, 2, 8, 200, 128), (4, 2, 8, 256, 100), (4, 2, 8, 0, 128), (4, 2, 8, 65536, 128)]:
        with pytest.raises(moe.MoEError, match="INVALID_ARG"):
            moe.moe_layer_few_ws_bytes(T, k, E, H, F)
    assert lib.moe_matvec_w4(None, 1, 128, None, 16, 128, None, None, None) == moe.MOE_ERR_INVALID_ARG
    assert lib.moe_quant_weights_w4(None, 1, 16, 128, 128, None, None) == moe.MOE_ERR_INVALID_ARG
    assert lib.moe_pack_weights_w4(None, None, 1, 16, 128, 128, None, None) == moe.MOE_ERR_INVALID_ARG
    assert lib.moe_dequant_weights_w4(None, 1, 16, 128, 128, None, None) == moe.MOE_ERR_INVALID_ARG
    assert lib.moe_layer_few(None, 1, 256, None, 8, 2, None, None, None, None, 128, 0, None, None, None, None, 0, None, None) == \
        moe.MOE_ERR_INVALID_ARG


def test_binding_refuses_wrong_shapes(lib):
    u8, f32, bf = torch.uint8, torch.float32, torch.bfloat16
    st = torch.zeros(1, dtype=torch.int32)
    T, k, E, H, F, g = 4, 2, 8, 256, 128, 128
    x, y = torch.zeros(T, H, dtype=bf), torch.zeros(T, 40, dtype=bf)
    Wp = torch.zeros(moe.w4_packed_shape(1, 40, H, g)[1:], dtype=u8)
    ids, w, out = torch.zeros(T, k, dtype=torch.int32), torch.zeros(T, k), torch.zeros(T, H, dtype=bf)
    W1, W2 = torch.zeros(E, 2 * F, H, dtype=u8), torch.zeros(E, H, F, dtype=u8)
    s1, s2 = torch.zeros(E, 2 * F // 128, H // 128), torch.zeros(E, H // 128, F // 128)
    P1, P2 = torch.zeros(moe.w4_packed_shape(E, 2 * F, H, g), dtype=u8), torch.zeros(moe.w4_packed_shape(E, H, F, g), dtype=u8)
    ws = torch.zeros(1 << 16, dtype=u8)
    bad = [
        lambda: moe.w4_packed_shape(1, 16, 128, 16),
        lambda: moe.w4_packed_shape(1, 16, 100, 32),
        lambda: moe.moe_quant_weights_w4(torch.zeros(E, 40, H, dtype=bf), g, Wp),
        lambda: moe.moe_dequant_weights_w4(P1, g, torch.zeros(E, 2 * F + 16, H)),
        lambda: moe.moe_pack_weights_w4(torch.zeros(E, 2 * F, H // 2, dtype=u8), torch.zeros(E, 2 * F, 3, dtype=bf), g, P1),
        lambda: moe.moe_matvec_w4(x, Wp[:-1], g, y, st),
        lambda: moe.moe_matvec_w4(x, Wp, g, y[:-1], st),
        lambda: moe.moe_matvec_w4(x, Wp, 64, y, st),
        lambda: moe.moe_matvec_w4(x, Wp, g, y, torch.zeros(0, dtype=torch.int32)),
        lambda: moe.moe_layer_few(x, W1, None, W2, None, ids, w, out, ws, st),
        lambda: moe.moe_layer_few(x, W1, s1, W2, s1, ids, w, out, ws, st),
        lambda: moe.moe_layer_few(x, W1, s1, W2[:, :, :-128], s2, ids, w, out, ws, st),
        lambda: moe.moe_layer_few(x, W1[:, :, :-128], s1, W2, s2, ids, w, out, ws, st),
        lambda: moe.moe_layer_few(x, P1, s1, P2, s2, ids, w, out, ws, st, group=g),
        lambda: moe.moe_layer_few(x, P1, None, P2, None, ids, w, out, ws, st, group=64),
        lambda: moe.moe_layer_few(x, P1, None, P2, None, ids[:-1], w, out, ws, st, group=g),
        lambda: moe.moe_layer_few(x, P1, None, P2, None, ids, w[:, :-1], out, ws, st, group=g),
        lambda: moe.moe_layer_few(x, P1, None, P2, None, ids, w, out[:-1], ws, st, group=g),
        lambda: moe.moe_layer_few(x, P1, None, P2, None, ids, w, out, ws, st, group=g, router=torch.zeros(E, H - 1, dtype=bf)),
        lambda: moe.moe_layer_few(x, P1, None, P2, None, ids, w, out, ws, torch.zeros(0, dtype=torch.int32), group=g),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError, match="shape|dimensions|status|group|scale"):
            call()
    with pytest.raises(ValueError, match="CUDA tensor"):
        moe.moe_layer_few(x, P1, None, P2, None, ids, w, out, ws, st, group=g)
    with pytest.raises(ValueError, match="CUDA tensor"):
        moe.moe_matvec_w4(x, Wp, g, y, st)
