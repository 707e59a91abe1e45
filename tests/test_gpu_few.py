"""The decoding operators on the GPU against the fp64 oracle: 4-bit weights bit for
bit; products and the whole layer within the rounding bounds that the oracle
derives (elementwise)."""
import ctypes

import numpy as np
import pytest
import torch

import combine_counting_sort_gb300 as moe
import oracle
from combine_counting_sort_gb300 import inputs
from tests.gpu_util import bits, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()


def bf16_t(b: np.ndarray) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(b).view(np.int16)).view(torch.bfloat16).cuda()


def rand_bits(*shape, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return inputs.bf16_bits((torch.randn(*shape, generator=g) * scale).to(torch.bfloat16))


def f64(b):
    return oracle.bf16_to_f32(b).astype(np.float64)


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def within(got: torch.Tensor, want, bound, what=""):
    g = f64(bits(got))
    assert g.shape == want.shape
    assert np.all(np.isfinite(g)), f"{what}: not finite"
    over = np.abs(g - want) - bound
    assert over.max() <= 0, f"{what}: {np.sum(over > 0)} of {over.size} over the bound, worst {np.max(np.abs(g - want) / bound):.3g}x"


# ---------------------------------------------------------------- 4-bit weights

W4_SHAPES = [(1, 16, 128, 128), (3, 1, 32, 32), (2, 17, 160, 32), (1, 515, 2080, 32), (2, 33, 192, 64), (1, 100, 1024, 128)]


@pytest.mark.parametrize("E,N,K,group", W4_SHAPES)
def test_quantise_pack_dequantise_bit_exact(E, N, K, group):
    b = rand_bits(E, N, K, seed=N + K)
    b[0, 0, :group] = 0                                     # a group of zeros
    b[0, -1, :group] = (np.arange(group) % 5).astype(np.uint16)   # subnormals
    b[-1, -1, -group:] = np.where(np.arange(group) % 2, 0x40E0, 0x3F00)   # max 7: scale 1, ties at 0.5
    q, s = oracle.quantize_w4(b, group)
    want = oracle.pack_w4(q, s)
    Wp = torch.full(moe.w4_packed_shape(E, N, K, group), 0xAB, dtype=torch.uint8, device="cuda")
    moe.moe_quant_weights_w4(bf16_t(b), group, Wp)
    assert np.array_equal(Wp.cpu().numpy(), want)
    plain = torch.from_numpy(q[..., 0::2] | (q[..., 1::2] << 4)).cuda()
    Wp2 = torch.full_like(Wp, 0xCD)
    moe.moe_pack_weights_w4(plain, bf16_t(s), group, Wp2)
    assert np.array_equal(Wp2.cpu().numpy(), want)
    v = torch.full((E, N, K), float("nan"), device="cuda")
    moe.moe_dequant_weights_w4(Wp, group, v)
    assert np.array_equal(v.cpu().numpy().astype(np.float64), oracle.w4_values(q, s))


def test_quantise_keeps_what_is_not_finite_in_its_group():
    b = rand_bits(1, 16, 256, seed=3)
    b[0, 2, 5], b[0, 4, 200] = 0x7F80, 0x7FC0
    Wp = torch.empty(moe.w4_packed_shape(1, 16, 256, 64), dtype=torch.uint8, device="cuda")
    moe.moe_quant_weights_w4(bf16_t(b), 64, Wp)
    v = torch.empty(1, 16, 256, device="cuda")
    moe.moe_dequant_weights_w4(Wp, 64, v)
    bad = (~torch.isfinite(v[0])).cpu().numpy()
    want = np.zeros((16, 256), bool)
    want[2, 0:64] = want[4, 192:256] = True
    assert np.array_equal(bad & want, bad) and bad[2].any() and bad[4].any()


# ---------------------------------------------------------------- matrix-vector products

def w4_matrix(N, K, group, seed=0, scale=None):
    b = rand_bits(1, N, K, seed=seed, scale=scale or K ** -0.5)
    q, s = oracle.quantize_w4(b, group)
    return torch.from_numpy(oracle.pack_w4(q, s)[0]).cuda(), oracle.w4_values(q, s)[0]


MATVEC = [(1, 16, 128, 128), (1, 1, 32, 32), (1, 17, 160, 32), (3, 40, 192, 64), (7, 1111, 1056, 32), (8, 256, 2048, 128),
          (9, 300, 1152, 128), (16, 64, 4096, 64), (17, 515, 2080, 32), (33, 2432, 256, 64), (64, 129, 1408, 128), (2, 7168, 2048, 32),
          (1, 4096, 7168, 128), (5, 48, 32768, 64)]


@pytest.mark.parametrize("T,N,K,group", MATVEC)
def test_matvec_w4(T, N, K, group):
    Wp, W = w4_matrix(N, K, group, seed=T + N)
    xb = rand_bits(T, K, seed=T * 7 + K)
    xb[0, K // 2] = inputs.bf16_bits(torch.tensor([300.0]).to(torch.bfloat16))[0]   # an outlier
    y = torch.full((T, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    st = status()
    moe.moe_matvec_w4(bf16_t(xb), Wp, group, y, st)
    torch.cuda.synchronize()
    assert st.item() == 0
    within(y, *oracle.matvec_bound(f64(xb), W), "matvec")


def test_matvec_writes_no_more_than_its_output_and_repeats_bit_for_bit():
    T, N, K, group = 5, 37, 416, 32
    Wp, _ = w4_matrix(N, K, group, seed=1)
    x = bf16_t(rand_bits(T, K, seed=2))
    buf = torch.full((T * N + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    y = buf[:T * N].view(T, N)
    st = status()
    moe.moe_matvec_w4(x, Wp, group, y, st)
    first = y.clone()
    y.fill_(float("nan"))
    moe.moe_matvec_w4(x, Wp, group, y, st)
    torch.cuda.synchronize()
    assert torch.equal(first, y) and torch.all(buf[T * N:] == 7.0) and st.item() == 0


def test_matvec_tokens_do_not_meet():
    # a NaN, an infinity and the largest value in one token leave the others as they were
    T, N, K, group = 11, 64, 256, 64
    Wp, W = w4_matrix(N, K, group, seed=1)
    xb = rand_bits(T, K, seed=2)
    y0, y1 = (torch.empty(T, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    moe.moe_matvec_w4(bf16_t(xb), Wp, group, y0, status())
    xb[4, 3], xb[4, 70], xb[9, 5] = 0x7FC0, 0x7F80, 0x7F7F
    moe.moe_matvec_w4(bf16_t(xb), Wp, group, y1, status())
    keep = [t for t in range(T) if t not in (4, 9)]
    assert torch.equal(y0[keep], y1[keep])
    assert torch.isnan(y1[4]).all()


def test_matvec_on_a_side_stream_and_in_a_graph():
    T, N, K, group = 4, 640, 1024, 128
    Wp, W = w4_matrix(N, K, group, seed=4)
    xb = rand_bits(T, K, seed=5)
    x, y, st = bf16_t(xb), torch.zeros(T, N, dtype=torch.bfloat16, device="cuda"), status()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    moe.moe_matvec_w4(x, Wp, group, y, st, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    want, bound = oracle.matvec_bound(f64(xb), W)
    torch.cuda.synchronize()
    within(y, want, bound, "side stream")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_matvec_w4(x, Wp, group, y, st)
    xb2 = rand_bits(T, K, seed=6)
    x.copy_(bf16_t(xb2))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    within(y, *oracle.matvec_bound(f64(xb2), W), "graph")
    assert st.item() == 0


def test_matvec_refusals():
    Wp, _ = w4_matrix(16, 128, 128)
    x, y, st = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, 16, dtype=torch.bfloat16, device="cuda"), status()
    lib, p = moe.lib(), lambda t: ctypes.c_void_p(t.data_ptr())
    ok = [p(x), 4, 128, p(Wp), 16, 128, p(y), p(st), None]
    assert lib.moe_matvec_w4(*ok) == moe.MOE_OK
    off = ctypes.c_void_p(x.data_ptr() + 2)
    for i, v in [(0, None), (0, off), (1, 0), (1, 65), (2, 0), (2, 100), (3, None), (3, ctypes.c_void_p(Wp.data_ptr() + 8)), (4, 0),
                 (5, 48), (6, None), (7, None)]:
        args = list(ok)
        args[i] = v
        assert lib.moe_matvec_w4(*args) == moe.MOE_ERR_INVALID_ARG, i
    with pytest.raises(ValueError, match="contiguous"):
        moe.moe_matvec_w4(torch.zeros(128, 4, dtype=torch.bfloat16, device="cuda").t(), Wp, 128, y, st)
    with pytest.raises(ValueError, match="bfloat16"):
        moe.moe_matvec_w4(x.float(), Wp, 128, y, st)
    torch.cuda.synchronize()
    assert st.item() == 0


# ---------------------------------------------------------------- the whole layer

class Experts:
    """E experts in either form, with their fp64 values."""

    def __init__(self, E, H, F, group, seed=0, used=None):
        self.E, self.H, self.F, self.group = E, H, F, group
        self.W1_scale = self.W2_scale = None
        b1, b2 = rand_bits(E, 2 * F, H, seed=seed, scale=H ** -0.5), rand_bits(E, H, F, seed=seed + 1, scale=F ** -0.5)
        if group:
            (q1, s1), (q2, s2) = oracle.quantize_w4(b1, group), oracle.quantize_w4(b2, group)
            self.W1, self.W2 = (torch.from_numpy(oracle.pack_w4(*v)).cuda() for v in ((q1, s1), (q2, s2)))
            self.values = {e: (oracle.w4_values(q1[e], s1[e]), oracle.w4_values(q2[e], s2[e])) for e in range(E)}
        else:
            (q1, s1), (q2, s2) = oracle.quantize_weights(b1), oracle.quantize_weights(b2)
            self.W1, self.W1_scale, self.W2, self.W2_scale = (torch.from_numpy(v).cuda() for v in (q1, s1, q2, s2))
            self.values = {e: (oracle.fp8_values(q1[e], s1[e]), oracle.fp8_values(q2[e], s2[e])) for e in range(E)}

    def workspace(self, T, k):
        return torch.zeros(moe.moe_layer_few_ws_bytes(T, k, self.E, self.H, self.F), dtype=torch.uint8, device="cuda")

    def call(self, x, ids, w, out, ws, st, router=None, stream=None):
        moe.moe_layer_few(x, self.W1, self.W1_scale, self.W2, self.W2_scale, ids, w, out, ws, st, router=router, group=self.group, stream=stream)

    def run(self, xb, ids, w, router=None, want_status=0):
        T, k = ids.shape
        out = torch.full((T, self.H), float("nan"), dtype=torch.bfloat16, device="cuda")
        ids_t, w_t, st, ws = torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), status(), self.workspace(T, k)
        if ws.numel() > 256:
            ws[256:] = 0xFF                                # NaN wherever nothing was written
        self.call(bf16_t(xb), ids_t, w_t, out, ws, st, router)
        torch.cuda.synchronize()
        assert st.item() == want_status
        assert not ws[:256].any(), "the workspace's head is left zero"
        return out, ids_t.cpu().numpy(), w_t.cpu().numpy()


def routes(T, k, E, seed=0):
    rng = np.random.default_rng(seed)
    ids = np.argsort(rng.random((T, E)), 1)[:, :k].astype(np.int32)
    return ids, (rng.random((T, k)) + 0.1).astype(np.float32)


GROUPS = [0, 32, 64, 128]
LAYERS = [(1, 1, 1, 128, 128), (1, 2, 8, 256, 256), (2, 2, 4, 384, 128), (5, 3, 9, 256, 384), (8, 2, 8, 512, 256), (9, 8, 8, 256, 128),
          (16, 2, 4, 1152, 256), (33, 4, 60, 256, 128), (64, 2, 8, 256, 256), (64, 16, 16, 128, 128), (32, 32, 32, 128, 128)]


@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("T,k,E,H,F", LAYERS)
def test_layer_with_own_routes(T, k, E, H, F, group):
    ex = Experts(E, H, F, group, seed=T)
    ids, w = routes(T, k, E, seed=T + k)
    xb = rand_bits(T, H, seed=T + 1)
    out, ids2, w2 = ex.run(xb, ids, w)
    assert np.array_equal(ids, ids2) and np.array_equal(w, w2)
    within(out, *oracle.layer_few(f64(xb), ids, w, ex.values), "layer")


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("T,k,E,H,F", [(1, 1, 1, 128, 128), (1, 8, 256, 256, 128), (7, 2, 8, 512, 128), (40, 4, 300, 256, 128), (64, 8, 1024, 128, 128)])
def test_layer_with_router(T, k, E, H, F, group):
    ex = Experts(E, H, F, group, seed=E)
    xb, rb = rand_bits(T, H, seed=T + 1), rand_bits(E, H, seed=T + 2, scale=H ** -0.5)
    out, ids, w = ex.run(xb, np.full((T, k), -7, np.int32), np.full((T, k), np.nan, np.float32), bf16_t(rb))
    # the choice is that of logits within H 2^-24 of the magnitudes; at these seeds no two
    # of the first k + 1 logits are nearer than that
    logits, mag = f64(xb) @ f64(rb).T, np.abs(f64(xb)) @ np.abs(f64(rb)).T
    order = np.argsort(-logits, 1, kind="stable")
    sorted_l = np.take_along_axis(logits, order, 1)
    slack = (H + 2) * 2.0 ** -24 * mag.max()
    clear = np.all(-np.diff(sorted_l[:, :k + 1], axis=1) > 2 * slack, 1) if E > 1 else np.ones(T, bool)
    assert clear.mean() > 0.9
    assert np.array_equal(ids[clear], order[clear, :k])
    got_l = np.take_along_axis(logits, ids.astype(np.int64), 1)
    ew = np.exp(got_l - got_l[:, :1])
    ew /= ew.sum(1, keepdims=True)
    assert np.all(np.abs(w - ew) <= ew * (4 * slack + 2.0 ** -19))
    within(out, *oracle.layer_few(f64(xb), ids, w, ex.values), "layer")


def test_router_ties_go_to_the_lowest_expert():
    T, k, E, H, F = 3, 4, 16, 128, 128
    ex = Experts(E, H, F, 0, seed=1)
    rb = np.repeat(rand_bits(2, H, seed=2), 8, 0)          # two groups of equal logits
    out, ids, w = ex.run(rand_bits(T, H, seed=3), np.zeros((T, k), np.int32), np.zeros((T, k), np.float32), bf16_t(rb))
    for row in ids:
        assert list(row) in ([0, 1, 2, 3], [8, 9, 10, 11])
    assert np.all(np.abs(w - 0.25) < 1e-6)


@pytest.mark.parametrize("group", [0, 64])
def test_layer_padding_invalid_ids_and_repeats(group):
    T, k, E, H, F = 12, 3, 6, 256, 256
    ex = Experts(E, H, F, group, seed=2)
    ids, w = routes(T, k, E, seed=3)
    xb = rand_bits(T, H, seed=4)
    ids[2], ids[11], ids[5, 1] = -1, -1, -5                 # no route at all, and one slot without
    ids[7] = 4                                              # one expert three times
    ids[8, 2] = ids[8, 0]
    w[2] = np.nan                                           # a weight without a route is not read
    xb[11] = 0x7FC0                                         # nor is a token without one
    out, _, _ = ex.run(xb, ids, w)
    xz = f64(xb)
    xz[11] = 0
    within(out, *oracle.layer_few(xz, ids, np.nan_to_num(w), ex.values), "layer")
    assert torch.all(out[[2, 11]] == 0)
    ids[0, 0], ids[3] = E, 1 << 30                          # out of range: skipped and reported
    out, _, _ = ex.run(xb, ids, w, want_status=moe.MOE_ERR_EXPERT_ID)
    within(out, *oracle.layer_few(xz, ids, np.nan_to_num(w), ex.values), "layer")
    ids[:] = -1                                             # a batch of padding
    out, _, _ = ex.run(xb, ids, w)
    assert torch.all(out == 0)


@pytest.mark.parametrize("group", [0, 32])
def test_layer_one_expert_takes_every_token(group):
    for T in (17, 64):
        ex = Experts(3, 256, 128, group, seed=T)
        xb = rand_bits(T, 256, seed=T)
        ids, w = np.full((T, 1), 1, np.int32), np.full((T, 1), 0.5, np.float32)
        out, _, _ = ex.run(xb, ids, w)
        within(out, *oracle.layer_few(f64(xb), ids, w, ex.values), "layer")


@pytest.mark.parametrize("group", [0, 128])
def test_layer_reads_no_other_expert_and_tokens_do_not_meet(group):
    T, k, E, H, F = 10, 2, 8, 256, 256
    ex = Experts(E, H, F, group, seed=9)
    ids, w = routes(T, k, 6, seed=1)                        # experts 6 and 7 are used by nobody
    xb = rand_bits(T, H, seed=2)
    ref, _, _ = ex.run(xb, ids, w)
    for e in (6, 7):                                        # NaN codes, and NaN in the scales
        ex.W1[e] = ex.W2[e] = 0x7F
        if not group:
            ex.W1_scale[e] = ex.W2_scale[e] = float("nan")
        else:
            ex.W1[e, ..., 1024:] = ex.W2[e, ..., 1024:] = 0xFF
    out, _, _ = ex.run(xb, ids, w)
    assert torch.equal(out, ref)
    xb[3, 100] = 0x7FC0                                     # one token's NaN stays its own
    out, _, _ = ex.run(xb, ids, w)
    keep = [t for t in range(T) if t != 3]
    assert torch.isnan(out[3]).all() and torch.equal(out[keep], ref[keep])


@pytest.mark.parametrize("group", [0, 128])
def test_layer_repeats_bit_for_bit_on_one_workspace(group):
    ex = Experts(16, 256, 128, group, seed=5)
    ws, st = ex.workspace(20, 4), status()
    outs = {}
    for rep in range(3):                                    # other sizes in between
        for T, k in ((20, 4), (1, 2), (7, 4)):
            ids, w = routes(T, k, 16, seed=T)
            out = torch.empty(T, 256, dtype=torch.bfloat16, device="cuda")
            ex.call(bf16_t(rand_bits(T, 256, seed=T)), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), out, ws, st)
            assert torch.equal(outs.setdefault(T, out), out)
    torch.cuda.synchronize()
    assert st.item() == 0


def test_layer_at_full_width():
    T, k, E, H, F = 3, 2, 4, 7168, 2048
    for group in (0, 128):
        ex = Experts(E, H, F, group, seed=1)
        ids, w = routes(T, k, E, seed=2)
        xb = rand_bits(T, H, seed=3)
        out, _, _ = ex.run(xb, ids, w)
        within(out, *oracle.layer_few(f64(xb), ids, w, ex.values), "layer")


def test_layer_on_a_side_stream_and_in_a_graph():
    T, k, E, H, F = 4, 2, 8, 512, 256
    ex = Experts(E, H, F, 64, seed=5)
    rb = rand_bits(E, H, seed=6, scale=H ** -0.5)
    router = bf16_t(rb)
    ids, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    out, ws, st = torch.empty(T, H, dtype=torch.bfloat16, device="cuda"), ex.workspace(T, k), status()
    xb = rand_bits(T, H, seed=7)
    x = bf16_t(xb)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ex.call(x, ids, w, out, ws, st, router, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    within(out, *oracle.layer_few(f64(xb), ids.cpu().numpy(), w.cpu().numpy(), ex.values), "side stream")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ex.call(x, ids, w, out, ws, st, router)
    for seed in (8, 9):
        xb = rand_bits(T, H, seed=seed)
        x.copy_(bf16_t(xb))
        graph.replay()
        torch.cuda.synchronize()
        within(out, *oracle.layer_few(f64(xb), ids.cpu().numpy(), w.cpu().numpy(), ex.values), "graph")
    assert st.item() == 0


def test_layer_refusals():
    T, k, E, H, F = 4, 2, 8, 256, 128
    ex = Experts(E, H, F, 0)
    ids, w = (torch.from_numpy(v).cuda() for v in routes(T, k, E))
    x, out, ws, st = bf16_t(rand_bits(T, H)), torch.zeros(T, H, dtype=torch.bfloat16, device="cuda"), ex.workspace(T, k), status()
    p = lambda t, o=0: ctypes.c_void_p(t.data_ptr() + o)   # noqa: E731
    ok = [p(x), T, H, None, E, k, p(ex.W1), p(ex.W1_scale), p(ex.W2), p(ex.W2_scale), F, 0, p(ids), p(w), p(out), p(ws), ws.numel(), p(st), None]
    lib = moe.lib()
    assert lib.moe_layer_few(*ok) == moe.MOE_OK
    for i, v in [(0, None), (0, p(x, 2)), (1, 0), (1, 65), (2, 200), (3, p(x, 2)), (4, 1), (5, 0), (5, 33), (6, None), (6, p(ex.W1, 8)), (7, None),
                 (8, None), (9, None), (10, 100), (11, 16), (11, 128), (12, None), (13, None), (14, None), (14, p(out, 2)), (15, None),
                 (15, p(ws, 16)), (16, 256), (17, None)]:
        args = list(ok)
        args[i] = v
        assert lib.moe_layer_few(*args) == moe.MOE_ERR_INVALID_ARG, i
    torch.cuda.synchronize()
    assert st.item() == 0


# ---------------------------------------------------------------- the kernels' own boundaries

# tokens around the switch between the two matvec kernels and the wide one's token blocks,
# rows around its groups, columns that end inside a stage, a slice and a half
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,N,K", [(8, 64, 4096), (8, 50, 32768), (9, 33, 384), (10, 1, 128), (24, 257, 640), (25, 512, 1152), (31, 4880, 512),
                                   (41, 31, 2176), (48, 272, 1024), (57, 1000, 896), (64, 16, 7168)])
def test_matvec_kernel_boundaries(T, N, K, group):
    Wp, W = w4_matrix(N, K, group, seed=T)
    xb = rand_bits(T, K, seed=N)
    y = torch.full((T, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    st = status()
    moe.moe_matvec_w4(bf16_t(xb), Wp, group, y, st)
    torch.cuda.synchronize()
    assert st.item() == 0
    within(y, *oracle.matvec_bound(f64(xb), W), "matvec")


@pytest.mark.parametrize("T", [1, 6, 20])
def test_matvec_tokens_of_very_different_sizes(T):
    # blocks of tiny and of huge values side by side: no token's scale is another block's
    N, K, group = 48, 512, 64
    Wp, W = w4_matrix(N, K, group, seed=T)
    x = f64(rand_bits(T, K, seed=T))
    x[:, 128:256] *= 2.0 ** -40
    x[:, 256:384] *= 2.0 ** 40
    x[0, :128] = 0
    xb = oracle.f64_to_bf16(x)
    y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    moe.moe_matvec_w4(bf16_t(xb), Wp, group, y, status())
    within(y, *oracle.matvec_bound(f64(xb), W), "matvec")


# few and many tokens per expert, few and many pairs, segments of 16, batches around the
# switches of the selection and of the sums
BOUNDARIES = [(4, 8, 16, 256, 128), (11, 3, 64, 256, 256), (8, 4, 4, 256, 128), (9, 1, 64, 384, 128), (16, 1, 1, 256, 128), (17, 1, 1, 256, 128),
              (24, 2, 64, 256, 128), (25, 2, 64, 256, 128), (33, 1, 2, 128, 256), (64, 8, 64, 256, 128), (3, 2, 5, 2176, 1152)]


@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("T,k,E,H,F", BOUNDARIES)
def test_layer_boundaries_with_router(T, k, E, H, F, group):
    ex = Experts(E, H, F, group, seed=T + E)
    xb, rb = rand_bits(T, H, seed=T + 1), rand_bits(E, H, seed=T + 2, scale=H ** -0.5)
    out, ids, w = ex.run(xb, np.zeros((T, k), np.int32), np.zeros((T, k), np.float32), bf16_t(rb))
    assert ids.min() >= 0 and ids.max() < E and all(len(set(r)) == k for r in ids)
    within(out, *oracle.layer_few(f64(xb), ids, w, ex.values), "layer")
    # the same routes given by the caller: the same output, bit for bit
    again, _, _ = ex.run(xb, ids, w)
    assert torch.equal(out, again)


@pytest.mark.parametrize("group", [0, 64])
def test_layer_small_tables_with_repeats_and_gaps(group):
    # at most 32 pairs: an expert three times, one without a route, one out of range
    ex = Experts(5, 256, 128, group, seed=3)
    ids = np.array([[4, 4, 4, 1], [0, -1, 4, 0], [-1, -1, -1, -1], [2, 9, 1, 2]], np.int32)
    w = np.random.default_rng(1).random(ids.shape).astype(np.float32)
    xb = rand_bits(4, 256, seed=5)
    out, _, _ = ex.run(xb, ids, w, want_status=moe.MOE_ERR_EXPERT_ID)
    within(out, *oracle.layer_few(f64(xb), ids, w, ex.values), "layer")
    assert torch.all(out[2] == 0)


@pytest.mark.parametrize("group", [0, 128])
def test_layer_offsets_past_32_bits(group):
    # the last of 200 experts' weights lies more than 2^31 (FP8) and 2^30 (4-bit) bytes in;
    # the others are NaN and unused
    E, H, F, e = 200, 7168, 1024, 199
    one = Experts(1, H, F, group, seed=1)
    fill = lambda t, v: torch.full((E, *t.shape[1:]), v, dtype=t.dtype, device="cuda")   # noqa: E731
    ex = Experts.__new__(Experts)
    ex.E, ex.H, ex.F, ex.group, ex.values = E, H, F, group, {e: one.values[0]}
    ex.W1, ex.W2 = fill(one.W1, 0x7F), fill(one.W2, 0x7F)
    ex.W1[e], ex.W2[e] = one.W1[0], one.W2[0]
    ex.W1_scale = ex.W2_scale = None
    if not group:
        ex.W1_scale, ex.W2_scale = fill(one.W1_scale, float("nan")), fill(one.W2_scale, float("nan"))
        ex.W1_scale[e], ex.W2_scale[e] = one.W1_scale[0], one.W2_scale[0]
    for T in (1, 10):
        ids, w = np.full((T, 1), e, np.int32), np.full((T, 1), 1.5, np.float32)
        xb = rand_bits(T, H, seed=2)
        out, _, _ = ex.run(xb, ids, w)
        within(out, *oracle.layer_few(f64(xb), ids, w, ex.values), "layer")


def test_layer_activations_far_from_one():
    # activations whose blocks differ by 2^60 and more than f16 holds
    H, F = 256, 256
    b1, b2 = rand_bits(1, 2 * F, H, seed=1, scale=H ** -0.5), rand_bits(1, H, F, seed=2, scale=F ** -0.5)
    f = f64(b1)
    f[0, F:F + 128] *= 2.0 ** 40
    f[0, F + 128:] *= 2.0 ** -40
    b1 = oracle.f64_to_bf16(f)
    (q1, s1), (q2, s2) = oracle.quantize_w4(b1, 32), oracle.quantize_w4(b2, 32)
    ex = Experts.__new__(Experts)
    ex.E, ex.H, ex.F, ex.group, ex.W1_scale, ex.W2_scale = 1, H, F, 32, None, None
    ex.W1, ex.W2 = (torch.from_numpy(oracle.pack_w4(*v)).cuda() for v in ((q1, s1), (q2, s2)))
    ex.values = {0: (oracle.w4_values(q1[0], s1[0]), oracle.w4_values(q2[0], s2[0]))}
    for T in (2, 12):
        xb = rand_bits(T, H, seed=T)
        ids, w = np.zeros((T, 1), np.int32), np.ones((T, 1), np.float32)
        out, _, _ = ex.run(xb, ids, w)
        within(out, *oracle.layer_few(f64(xb), ids, w, ex.values), "layer")


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("counter", [0, 1, 2])
def test_layer_meeting_that_cannot_be_complete_gives_up(group, counter):
    # a counter that starts short of its arrivals: the grid's wait runs out after a second,
    # the call reports it, leaves the workspace's head zero, and the next call is right
    T, k, E, H, F = 4, 2, 8, 256, 256
    ex = Experts(E, H, F, group, seed=1)
    ids, w = routes(T, k, E, seed=2)
    xb = rand_bits(T, H, seed=3)
    ws, st, out = ex.workspace(T, k), status(), torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    ws.view(torch.int32)[counter] = -1
    args = (bf16_t(xb), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), out, ws, st)
    ex.call(*args)
    torch.cuda.synchronize()
    assert st.item() == moe.MOE_ERR_TIMEOUT and not ws[:256].any()
    st.zero_()
    ex.call(*args)
    torch.cuda.synchronize()
    assert st.item() == 0
    within(out, *oracle.layer_few(f64(xb), ids, w, ex.values), "layer")


@pytest.mark.parametrize("weights", ["w4", "fp8"])
def test_decode_example_runs(weights):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, os.path.join(root, "examples", "decode_moe.py"), "--weights", weights, "--tokens", "3", "--steps", "4",
                        "--hidden", "256", "--ffn", "128", "--experts", "8", "--topk", "2", "--vocab", "1000"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "tokens/s" in r.stdout


# ---------------------------------------------------------------- matvec on many tokens or many rows

# clusters of 8, 4 and 2 blocks and single ones, uneven runs of slices, several rounds over the
# SMs, rows and tokens that end inside a block, few tokens on many rows
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,N,K", [(17, 3840, 1152), (33, 3841, 640), (64, 9216, 256), (48, 19456, 384), (20, 39000, 128),
                                   (9, 9744, 256), (16, 40000, 128), (2, 50, 24576), (8, 9731, 8192), (32, 255, 128)])
def test_matvec_many_tokens_or_rows(T, N, K, group):
    Wp, W = w4_matrix(N, K, group, seed=T)
    xb = rand_bits(T, K, seed=N)
    buf = torch.full((T * N + 64,), -7.0, dtype=torch.bfloat16, device="cuda")
    y, st = buf[:T * N].view(T, N), status()
    y.fill_(float("nan"))
    x = bf16_t(xb)
    moe.moe_matvec_w4(x, Wp, group, y, st)
    torch.cuda.synchronize()
    assert st.item() == 0
    within(y, *oracle.matvec_bound(f64(xb), W), "matvec")
    assert (buf[T * N:] == -7).all()
    again = torch.empty_like(y)
    moe.moe_matvec_w4(x, Wp, group, again, st)
    assert torch.equal(again.view(torch.int16), y.view(torch.int16))


def test_matvec_many_tokens_do_not_meet():
    # a token of infinities and NaN leaves every other token's bits as they were
    T, N, K, group = 40, 600, 384, 64
    Wp, _ = w4_matrix(N, K, group, seed=3)
    x = bf16_t(rand_bits(T, K, seed=4))
    want, got = (torch.empty(T, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    st = status()
    moe.moe_matvec_w4(x, Wp, group, want, st)
    x2 = x.clone()
    x2[7, ::3] = float("inf")
    x2[7, 1::3] = float("nan")
    moe.moe_matvec_w4(x2, Wp, group, got, st)
    keep = [t for t in range(T) if t != 7]
    assert torch.equal(got[keep].view(torch.int16), want[keep].view(torch.int16))
    assert got[7].isnan().all() and st.item() == 0


@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("T", [5, 14])
def test_layer_token_that_is_not_finite(T, group):
    # with the router: no logit of the token is a number, so no expert is its; with given
    # routes its out is NaN; the others' bits stay as they were
    E, k, H, F = 12, 3, 256, 384
    L = Experts(E, H, F, group, seed=5)
    x = bf16_t(rand_bits(T, H, seed=6))
    router = bf16_t(rand_bits(E, H, seed=7, scale=0.1))
    x2 = x.clone()
    x2[2, :] = float("nan")
    keep = [t for t in range(T) if t != 2]
    res = []
    for r in (router, None):
        for v in (x, x2):
            ids, w = routes(T, k, E, seed=8)
            ids, w = torch.as_tensor(ids, dtype=torch.int32).cuda(), torch.as_tensor(w, dtype=torch.float32).cuda()
            out, st = torch.full((T, H), -3.0, dtype=torch.bfloat16, device="cuda"), status()
            L.call(v, ids, w, out, L.workspace(T, k), st, r)
            torch.cuda.synchronize()
            res.append((out, ids, st.item()))
    for clean, spoilt in (res[:2], res[2:]):
        assert torch.equal(clean[0][keep].view(torch.int16), spoilt[0][keep].view(torch.int16)) and clean[2] == 0
    assert (res[1][1][2] == 0x7FFFFFFF).all() and (res[1][0][2] == 0).all() and res[1][2] == moe.MOE_ERR_EXPERT_ID
    assert res[3][0][2].isnan().all() and res[3][2] == 0
