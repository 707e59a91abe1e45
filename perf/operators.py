"""What is measured of the decode operators: 4-bit expert weights, their
matrix-vector products, and a whole MoE layer for a few tokens.

A 4-bit weight matrix [N, K] is held as tiles of 16 rows x 128 columns, each
tile one run of bytes: 1024 bytes of codes, then 128/group scales of 16 rows
each (bf16).  Byte (half, g, t, j, b) of the codes, 4 * (4 * (8 * 4 * half +
4 * g + t) + j) + b, holds in its low and high nibble (i = 0, 1) the codes of
row 8 * half + g and column 32 * j + 8 * t + 4 * (b % 2) + 2 * i + b // 2.  A code c
stands for (c - 8) * scale; what a matrix lacks of a whole tile has code 8 and
scale 0.

The quantiser's rule, per row and group of columns: scale = bf16(max|w| / 7),
code = 8 + rint(w / scale) within [0, 15], 8 where the scale is 0.
"""
import math

import torch

own = False

KINDS = ("quant", "matvec", "layer")


def listed():
    return [
        # Weights made ready once per model load: 16 experts' gate and up
        # projections, and a small ragged matrix with the finest groups.
        {"name": "quant 16x4096x7168 g128", "kind": "quant", "E": 16, "N": 4096, "K": 7168, "group": 128},
        {"name": "quant 1x515x2080 g32", "kind": "quant", "E": 1, "N": 515, "K": 2080, "group": 32},
        # One token through a projection beside the experts: the gate and up
        # rows of a shared expert, and its down projection with finer groups.
        {"name": "matvec T1 4096x7168 g128", "kind": "matvec", "T": 1, "N": 4096, "K": 7168, "group": 128},
        {"name": "matvec T3 7168x2048 g32", "kind": "matvec", "T": 3, "N": 7168, "K": 2048, "group": 32},
        # A small batch on odd sizes: latency, ragged rows and a ragged last tile.
        {"name": "matvec T7 1111x1056 g32", "kind": "matvec", "T": 7, "N": 1111, "K": 1056, "group": 32},
        # The largest batch through a vocabulary-sized projection.
        {"name": "matvec T48 32768x7168 g64", "kind": "matvec", "T": 48, "N": 32768, "K": 7168, "group": 64},
        # The smallest layer: one token, latency alone.
        {"name": "layer T1 E8 fp8 tiny", "kind": "layer", "T": 1, "E": 8, "k": 2, "H": 256, "F": 256, "group": 0, "router": True, "pad": 0},
        # Decoding one sequence: 8 of 256 experts, with the framework's FP8 weights and with 4-bit ones.
        {"name": "layer T1 E256 fp8", "kind": "layer", "T": 1, "E": 256, "k": 8, "H": 7168, "F": 2048, "group": 0, "router": True, "pad": 0},
        {"name": "layer T1 E256 w4 g128", "kind": "layer", "T": 1, "E": 256, "k": 8, "H": 7168, "F": 2048, "group": 128, "router": True, "pad": 0},
        # Small batches: about 57 experts of one or two tokens, then nearly every expert.
        {"name": "layer T8 E256 w4 g32", "kind": "layer", "T": 8, "E": 256, "k": 8, "H": 7168, "F": 2048, "group": 32, "router": True, "pad": 0},
        {"name": "layer T64 E256 fp8", "kind": "layer", "T": 64, "E": 256, "k": 8, "H": 7168, "F": 2048, "group": 0, "router": True, "pad": 0},
        # Few experts, many tokens each, the caller's own routes, and a padded
        # batch of an odd size: the last five tokens have no route.
        {"name": "layer T37 E32 w4 g128 own routes", "kind": "layer", "T": 37, "E": 32, "k": 8, "H": 7168, "F": 2048, "group": 128, "router": False, "pad": 5},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _times(rng, lo, hi, unit):
    n = max(1, round(_log(rng, lo, hi) / unit))
    return unit * (n + 1 if unit * n == 3 * 1024 else n)


def draw(rng):
    kind = rng.choices(KINDS, weights=(1, 2, 3))[0]
    if kind == "quant":
        group = rng.choice((32, 64, 128))
        return {"kind": kind, "E": rng.randint(1, 12), "N": _log(rng, 16, 4000) | 1, "K": _times(rng, 256, 7168, group), "group": group}
    if kind == "matvec":
        group = rng.choice((32, 64, 128))
        return {"kind": kind, "T": _log(rng, 1, 48), "N": _log(rng, 64, 30000) | 1, "K": _times(rng, 256, 7168, group), "group": group}
    E = rng.choice((8, 16, 60, 128, 256))
    router = rng.random() < 0.7
    T = _log(rng, 1, 60)
    return {"kind": kind, "T": T, "E": E, "k": rng.randint(1, 8), "H": _times(rng, 256, 7000, 128), "F": _times(rng, 128, 2040, 128),
            "group": rng.choice((0, 0, 32, 64, 128)), "router": router, "pad": 0 if router else rng.randint(0, T // 4)}


def _distinct(c):
    """Experts that are expected to be hit by uniform routes."""
    return c["E"] * (1 - (1 - c["k"] / c["E"]) ** (c["T"] - c["pad"]))


def _weight_bytes(n, k, group):
    return n * k + 4 * (n / 128) * (k / 128) if group == 0 else n * k / 2 + 2 * n * (k / group)


def work(c):
    if c["kind"] == "quant":  # bf16 in; the laid out codes written, and read back as the values they stand for
        n = c["E"] * c["N"] * c["K"]
        return {"bytes": 2 * n + 2 * c["E"] * _weight_bytes(c["N"], c["K"], c["group"]) + 4 * n, "flops": 3 * n}
    if c["kind"] == "matvec":
        return {"bytes": _weight_bytes(c["N"], c["K"], c["group"]) + 2 * c["T"] * (c["N"] + c["K"]), "flops": 2 * c["T"] * c["N"] * c["K"]}
    T, E, k, H, F, g = c["T"], c["E"], c["k"], c["H"], c["F"], c["group"]
    pairs = (T - c["pad"]) * k
    return {"bytes": _distinct(c) * (_weight_bytes(2 * F, H, g) + _weight_bytes(H, F, g)) + 4 * T * H + 8 * T * k + (2 * E * H if c["router"] else 0),
            "flops": 6 * pairs * H * F + (2 * T * E * H if c["router"] else 0)}


# ---------------------------------------------------------------- inputs

def _packed_shape(E, N, K, group):
    return (E, -(-N // 16), -(-K // 128), 1024 + 32 * (128 // group))


def _random_w4(gen, E, N, K, group, dev):
    """A quantised matrix as it is kept: codes of normal weights, scales around
    1 / sqrt(K) a standard deviation of the codes, laid out in tiles."""
    shape = _packed_shape(E, N, K, group)
    packed = torch.empty(shape, dtype=torch.uint8, device=dev)
    nt, kt = shape[1], shape[2]
    for e in range(E):
        q = torch.randn(nt * 16, kt * 128, generator=gen, device=dev, dtype=torch.float16).mul_(2.6).round_().add_(8.0).clamp_(0, 15).to(torch.uint8)
        q[N:] = 8
        q[:, K:] = 8
        # [nt, half, g, kt, j, t, bl, i, bh] -> [nt, kt, half, g, t, j, bh, bl, i]
        q = q.view(nt, 2, 8, kt, 4, 4, 2, 2, 2).permute(0, 3, 1, 2, 5, 4, 8, 6, 7)
        packed[e, :, :, :1024] = (q[..., 0] | (q[..., 1] << 4)).reshape(nt, kt, 1024)
        s = torch.rand(nt * 16, kt * (128 // group), generator=gen, device=dev).add_(0.5).mul_(1 / (2.6 * math.sqrt(K)))
        s[N:] = 0
        s[:, K // group:] = 0
        s = s.to(torch.bfloat16).view(nt, 16, kt, 128 // group).permute(0, 2, 3, 1).contiguous()
        packed[e, :, :, 1024:] = s.view(torch.uint8).reshape(nt, kt, -1)
    return packed


def _random_fp8(gen, E, N, K, dev):
    """e4m3 codes of normal weights and a scale for each 128 x 128 block."""
    codes = torch.empty(E, N, K, dtype=torch.uint8, device=dev)
    for e in range(E):
        codes[e] = torch.randn(N, K, generator=gen, device=dev, dtype=torch.float16).mul_(100.0).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    scale = torch.rand(E, N // 128, K // 128, generator=gen, device=dev).add_(0.5).mul_(1 / (100.0 * math.sqrt(K)))
    return codes, scale


def prepare(case, seed):
    c, dev = case, "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(1_000_003 * int(seed) + 17)
    s = {"case": c}
    if c["kind"] == "quant":
        s["W"] = torch.randn(c["E"], c["N"], c["K"], generator=gen, device=dev, dtype=torch.bfloat16).mul_(1 / math.sqrt(c["K"]))
        s["W"][0, 0, : c["group"]] = 0  # a group of zeros has scale 0
        s["packed"] = torch.empty(_packed_shape(c["E"], c["N"], c["K"], c["group"]), dtype=torch.uint8, device=dev)
        s["values"] = torch.empty(c["E"], c["N"], c["K"], dtype=torch.float32, device=dev)
        return s
    s["status"] = torch.zeros(1, dtype=torch.int32, device=dev)
    if c["kind"] == "matvec":
        s["x"] = torch.randn(c["T"], c["K"], generator=gen, device=dev).to(torch.bfloat16)
        s["packed"] = _random_w4(gen, 1, c["N"], c["K"], c["group"], dev)[0]
        s["y"] = torch.empty(c["T"], c["N"], dtype=torch.bfloat16, device=dev)
        return s
    T, E, k, H, F, g = c["T"], c["E"], c["k"], c["H"], c["F"], c["group"]
    s["x"] = torch.randn(T, H, generator=gen, device=dev).to(torch.bfloat16)
    if g:
        s["W1"], s["W1_scale"] = _random_w4(gen, E, 2 * F, H, g, dev), None
        s["W2"], s["W2_scale"] = _random_w4(gen, E, H, F, g, dev), None
    else:
        s["W1"], s["W1_scale"] = _random_fp8(gen, E, 2 * F, H, dev)
        s["W2"], s["W2_scale"] = _random_fp8(gen, E, H, F, dev)
    s["router"], s["ids"], s["w"] = None, torch.empty(T, k, dtype=torch.int32, device=dev), torch.empty(T, k, device=dev)
    if c["router"]:
        s["router"] = torch.randn(E, H, generator=gen, device=dev).mul_(1 / math.sqrt(H)).to(torch.bfloat16)
    else:
        s["ids"] = torch.rand(T, E, generator=gen, device=dev).argsort(1)[:, :k].to(torch.int32).contiguous()
        s["w"] = torch.rand(T, k, generator=gen, device=dev).add_(0.1)
        if c["pad"]:
            s["ids"][T - c["pad"]:] = -1
    s["out"] = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
    return s


# ---------------------------------------------------------------- the plain forms

def _values_w4(packed, N, K, group):
    """[..., N, K] in 32 bits from the tiles."""
    lead, (nt, kt) = packed.shape[:-3], packed.shape[-3:-1]
    b = packed[..., :1024].reshape(-1, nt, kt, 2, 8, 4, 4, 2, 2)
    q = torch.stack((b & 15, b >> 4), -1)  # [e, nt, kt, half, g, t, j, bh, bl, i]
    q = q.permute(0, 1, 3, 4, 2, 6, 5, 8, 9, 7).float().sub_(8.0)
    sc = packed[..., 1024:].contiguous().view(torch.bfloat16).view(-1, nt, kt, 128 // group, 16)
    sc = sc.permute(0, 1, 4, 2, 3).reshape(-1, nt * 16, kt * (128 // group), 1).float()
    v = q.reshape(-1, nt * 16, kt * (128 // group), group).mul_(sc)
    return v.view(*lead, nt * 16, kt * 128)[..., :N, :K]


def _values_fp8(codes, scale):
    n, k = codes.shape[-2:]
    v = codes.view(torch.float8_e4m3fn).float().view(-1, n // 128, 128, k // 128, 128)
    return v.mul_(scale.reshape(-1, n // 128, 1, k // 128, 1)).view(codes.shape)


def _plain_quant(s):
    c = s["case"]
    w = s["W"].float().view(c["E"], c["N"], -1, c["group"])
    scale = (w.abs().amax(-1, keepdim=True) / 7).to(torch.bfloat16).float()
    q = torch.where(scale > 0, (w / scale).round().clamp(-8, 7), 0.0)
    return (q * scale).view(c["E"], c["N"], c["K"])


def _plain_layer(s):
    c, x = s["case"], s["x"].float()
    T, E, k, H, F, g = c["T"], c["E"], c["k"], c["H"], c["F"], c["group"]
    if c["router"]:
        top, ids = (x @ s["router"].float().t()).sort(dim=1, descending=True, stable=True)  # ties to the lowest expert
        e = (top[:, :k] - top[:, :1]).exp()
        ids, w = ids[:, :k], e / e.sum(1, keepdim=True)
    else:
        ids, w = s["ids"].long(), s["w"]
    comb = torch.zeros(T, E + 1, device=x.device).scatter_add_(1, torch.where(ids < 0, E, ids), w)[:, :E]
    use = (comb != 0).any(0).nonzero()[:, 0]
    if g:
        w1, w2 = _values_w4(s["W1"][use], 2 * F, H, g), _values_w4(s["W2"][use], H, F, g)
    else:
        w1, w2 = _values_fp8(s["W1"][use], s["W1_scale"][use]), _values_fp8(s["W2"][use], s["W2_scale"][use])
    gate, up = (x @ w1.transpose(1, 2)).split(F, -1)
    h = gate / (1 + (-gate).exp()) * up * comb[:, use].t().unsqueeze(-1)
    out = (h @ w2.transpose(1, 2)).sum(0).to(torch.bfloat16)
    return {"out": out, "ids": ids.to(torch.int32), "w": w} if c["router"] else {"out": out}


def _plain(s):
    c = s["case"]
    if c["kind"] == "quant":
        return {"values": _plain_quant(s)}
    if c["kind"] == "matvec":
        return {"y": (s["x"].float() @ _values_w4(s["packed"], c["N"], c["K"], c["group"]).t()).to(torch.bfloat16)}
    return _plain_layer(s)


# ---------------------------------------------------------------- the framework's operators

def _framework(s):
    import combine_counting_sort_gb300 as moe
    c = s["case"]
    if c["kind"] == "quant":
        moe.moe_quant_weights_w4(s["W"], c["group"], s["packed"])
        moe.moe_dequant_weights_w4(s["packed"], c["group"], s["values"])
        return {"values": s["values"]}
    if c["kind"] == "matvec":
        moe.moe_matvec_w4(s["x"], s["packed"], c["group"], s["y"], s["status"])
        return {"y": s["y"]}
    if "ws" not in s:  # the workspace is the caller's, made once
        s["ws"] = torch.zeros(moe.moe_layer_few_ws_bytes(c["T"], c["k"], c["E"], c["H"], c["F"]), dtype=torch.uint8, device=s["x"].device)
    moe.moe_layer_few(s["x"], s["W1"], s["W1_scale"], s["W2"], s["W2_scale"], s["ids"], s["w"], s["out"], s["ws"], s["status"],
                      router=s["router"], group=c["group"])
    return {"out": s["out"], "ids": s["ids"], "w": s["w"]} if c["router"] else {"out": s["out"]}


def run(state):
    return _framework(state) if own else _plain(state)


# ---------------------------------------------------------------- the definition, in 64 bits

def _matrix(packed, N, K, group):
    """One matrix [N, K] in 64 bits, each code looked up at its byte and nibble."""
    n, k = torch.arange(N, device=packed.device)[:, None], torch.arange(K, device=packed.device)[None, :]
    r, col = n % 16, k % 128
    lane = 4 * (r % 8) + (col % 32) // 8
    byte = 4 * (4 * (32 * (r // 8) + lane) + col // 32) + 2 * (col % 2) + (col % 8) // 4
    code = packed[n // 16, k // 128, byte]
    code = torch.where((col % 4) // 2 == 1, code >> 4, code & 15).double() - 8
    at = 1024 + 2 * (16 * (col // group) + r)
    lo, hi = packed[n // 16, k // 128, at].int(), packed[n // 16, k // 128, at + 1].int()
    return code * ((hi << 24) | (lo << 16)).view(torch.float32).double()


def _matrix_fp8(codes, scale):
    N, K = codes.shape
    n, k = torch.arange(N, device=codes.device)[:, None], torch.arange(K, device=codes.device)[None, :]
    c = codes.long()
    man, ex, sign = c & 7, (c >> 3) & 15, 1 - 2 * (c >> 7)
    mag = torch.where(ex == 0, man * 2.0 ** -9, (8 + man).double() * torch.exp2((ex - 10).double()))
    return sign * mag.double() * scale.double()[n // 128, k // 128]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["kind"] == "quant":
        out = torch.empty(s["W"].shape, dtype=torch.float64, device=s["W"].device)
        for e in range(c["E"]):
            for k in range(0, c["K"], c["group"]):
                w = s["W"][e, :, k:k + c["group"]].double()
                m = w.abs().max(1, keepdim=True).values / 7
                step = m.float().to(torch.bfloat16).double()
                q = torch.zeros_like(w)
                live = step[:, 0] > 0
                q[live] = torch.clamp(torch.round(w[live] / step[live]), -8, 7)
                out[e, :, k:k + c["group"]] = q * step
        return {"values": out}
    if c["kind"] == "matvec":
        y = torch.empty(c["T"], c["N"], dtype=torch.float64, device=s["x"].device)
        for n in range(0, c["N"], 4096):
            m = min(4096, c["N"] - n)
            y[:, n:n + m] = torch.einsum("tk,nk->tn", s["x"].double(), _matrix(s["packed"][n // 16:], m, c["K"], c["group"]))
        return {"y": y}
    T, E, k, H, F, g = c["T"], c["E"], c["k"], c["H"], c["F"], c["group"]
    x = s["x"].double()
    if c["router"]:
        logits = torch.einsum("th,eh->te", x, s["router"].double())
        order = torch.argsort(-logits, dim=1, stable=True)[:, :k]
        w = torch.softmax(torch.gather(logits, 1, order), 1)
        ids = order
    else:
        ids, w = s["ids"], s["w"].double()
    out = torch.zeros(T, H, dtype=torch.float64, device=x.device)
    for e in sorted(set(ids.flatten().tolist()) - {-1}):
        t, j = (ids == e).nonzero(as_tuple=True)
        if g:
            w1, w2 = _matrix(s["W1"][e], 2 * F, H, g), _matrix(s["W2"][e], H, F, g)
        else:
            w1, w2 = _matrix_fp8(s["W1"][e], s["W1_scale"][e]), _matrix_fp8(s["W2"][e], s["W2_scale"][e])
        a = torch.einsum("th,nh->tn", x[t], w1)
        h = a[:, :F] * torch.sigmoid(a[:, :F]) * a[:, F:]
        out.index_add_(0, t, w[t, j][:, None] * torch.einsum("tf,nf->tn", h, w2))
    return {"out": out, "ids": ids.to(torch.int32), "w": w} if c["router"] else {"out": out}
