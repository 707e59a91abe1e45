"""The decoding operators on values where they can go wrong."""
import pytest
import torch

from tests.gpu_util import build
from tests.test_gpu_few import Experts, rand_bits, routes

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
