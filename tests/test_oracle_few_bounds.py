"""The bounds that the decoding tests hold the layer to: a roundoff of the activations other
than the stated one, to f16's 11 bits, is outside of them."""
import numpy as np
import pytest

import oracle

U16 = lambda v: oracle.bf16_to_f32(oracle.f64_to_bf16(v)).astype(np.float64)   # noqa: E731


def as_records(a):
    """f16 behind the power of two that brings the largest of 128 values to [2^14, 2^15)."""
    b = a.reshape(*a.shape[:-1], -1, 128)
    e = np.floor(np.log2(np.abs(b).max(-1, keepdims=True))) - 14
    return ((b * 2.0 ** -e).astype(np.float16).astype(np.float64) * 2.0 ** e).reshape(a.shape)


def one_feature_weights(H, F, rng):
    """[H, F] with one weight a row, so that an activation's rounding is not averaged out."""
    W2 = np.zeros((H, F))
    W2[np.arange(H), rng.permutation(H) % F] = 0.6875
    return W2


@pytest.mark.parametrize("seed", [0, 1])
def test_the_layers_bound_is_that_of_f16_activations(seed):
    rng = np.random.default_rng(seed)
    T, H, F = 8, 256, 256
    x, W1 = U16(rng.standard_normal((T, H))), rng.integers(-7, 8, (2 * F, H)) * 2.0 ** -6
    W2, w = one_feature_weights(H, F, rng), np.full((T, 1), 0.75)
    want, bound = oracle.layer_few(x, np.zeros((T, 1), int), w, {0: (W1, W2)})
    y = x @ W1.T
    a = 0.75 * y[:, :F] / (1 + np.exp(-y[:, :F])) * y[:, F:]
    assert np.all(np.abs(U16(as_records(a) @ W2.T) - want) <= bound)
    assert np.any(np.abs(U16(U16(a) @ W2.T) - want) > bound)


def test_a_records_step_covers_what_f16_leaves_out():
    rng = np.random.default_rng(3)
    x = U16(rng.standard_normal((5, 384)) * 2.0 ** rng.integers(-45, 46, (5, 384)))
    assert np.all(np.abs(as_records(x) - x) <= oracle.few_oracle.record_step(x))
    big = np.abs(x).reshape(5, 3, 128).max(-1).repeat(128, 1)
    assert np.all((as_records(x) == x)[np.abs(x) >= big * 2.0 ** -31])


def test_a_tokens_bound_is_its_own():
    # whatever the batch: the same token's bound, alone and as the last of many
    rng = np.random.default_rng(4)
    T, H, F, k = 9, 128, 128, 2
    x, ids, w = rng.standard_normal((T, H)), np.tile([1, 0], (T, 1)), rng.random((T, k))
    ex = {e: (rng.standard_normal((2 * F, H)), rng.standard_normal((H, F))) for e in range(2)}
    for got, alone in zip(oracle.layer_few(x, ids, w, ex), oracle.layer_few(x[-1:], ids[-1:], w[-1:], ex)):
        assert np.allclose(got[-1], alone[0], rtol=1e-12, atol=0)
