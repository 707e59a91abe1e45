"""What is measured of the dense operators beside the experts: layer norm, a
dense projection with its epilogue, and the gated feed-forward block, each
forward for serving and forward with backward for training.

    norm    y = (x - mean) * rstd * weight + bias over each row, with
            rstd = 1 / sqrt(var + eps); backward: dx, dweight, dbias
    linear  y = act(x W^T + bias) + residual; backward: dx, dW, dbias
    gated   h = act(x Wg^T) * (x Wu^T), Wg and Wu the rows [0, F) and [F, 2F)
            of W1 [2F, H]; backward: dx, dW1

act is none, silu, gelu (by erf) or gelu_tanh.
"""
import math

import torch

own = False

KINDS = ("norm", "linear", "gated")
ACTS = ("none", "silu", "gelu", "gelu_tanh")
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-5


def listed():
    return [
        # The norm before a layer's router for one decoded token: latency alone.
        {"name": "norm T1 H7168", "kind": "norm", "T": 1, "H": 7168, "type": "bf16", "train": False},
        # A training batch's norm, with the sums over all its rows for the weight.
        {"name": "norm train T8192 H7168", "kind": "norm", "T": 8192, "H": 7168, "type": "bf16", "train": True},
        # Odd rows that no 16-byte load fits.
        {"name": "norm train T777 H1111 f16", "kind": "norm", "T": 777, "H": 1111, "type": "f16", "train": True},
        # A shared expert's down projection added to the routed experts' output, one token.
        {"name": "linear T1 7168x2048 residual", "kind": "linear", "T": 1, "N": 7168, "K": 2048, "act": "none",
         "bias": False, "residual": True, "type": "bf16", "train": False},
        # A small batch through a vocabulary-sized projection.
        {"name": "linear T48 32768x7168", "kind": "linear", "T": 48, "N": 32768, "K": 7168, "act": "none",
         "bias": True, "residual": False, "type": "bf16", "train": False},
        # Odd sizes, each part of the epilogue at once.
        {"name": "linear T333 1111x1056 gelu f16", "kind": "linear", "T": 333, "N": 1111, "K": 1056, "act": "gelu",
         "bias": True, "residual": True, "type": "f16", "train": False},
        # A training batch through a projection with all of its epilogue.
        {"name": "linear train T4096 7168x2048 gelu_tanh", "kind": "linear", "T": 4096, "N": 7168, "K": 2048, "act": "gelu_tanh",
         "bias": True, "residual": True, "type": "bf16", "train": True},
        # A shared expert's gate and up projections: one token, a small batch, a prompt.
        {"name": "gated T1 F2048 H7168", "kind": "gated", "T": 1, "F": 2048, "H": 7168, "act": "silu", "type": "bf16", "train": False},
        {"name": "gated T64 F2048 H7168", "kind": "gated", "T": 64, "F": 2048, "H": 7168, "act": "silu", "type": "bf16", "train": False},
        {"name": "gated T8192 F2048 H7168", "kind": "gated", "T": 8192, "F": 2048, "H": 7168, "act": "silu", "type": "bf16", "train": False},
        # The same block in training, and a small ragged one of the other type and activation.
        {"name": "gated train T8192 F2048 H7168", "kind": "gated", "T": 8192, "F": 2048, "H": 7168, "act": "silu", "type": "bf16", "train": True},
        {"name": "gated train T515 F711 H1032 gelu f16", "kind": "gated", "T": 515, "F": 711, "H": 1032, "act": "gelu", "type": "f16", "train": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _odd(rng, n):
    """n, or the odd number beside it."""
    return n | 1 if rng.random() < 0.5 else n


def draw(rng):
    kind = rng.choice(KINDS)
    train = rng.random() < 0.5
    if kind == "norm":
        return {"kind": kind, "T": _log(rng, 1, 8191), "H": _odd(rng, _log(rng, 64, 8000)), "type": rng.choice(tuple(TYPES)), "train": train}
    half = rng.choice(("bf16", "bf16", "f16"))
    T = _odd(rng, _log(rng, 1, 4000))
    if kind == "linear":
        return {"kind": kind, "T": T, "N": _odd(rng, _log(rng, 64, 8000)), "K": 8 * _log(rng, 8, 890), "act": rng.choice(ACTS),
                "bias": rng.random() < 0.5, "residual": rng.random() < 0.5, "type": half, "train": train}
    return {"kind": kind, "T": T, "F": _odd(rng, _log(rng, 64, 2000)), "H": 8 * _log(rng, 8, 890), "act": rng.choice(ACTS[1:]),
            "type": half, "train": train}


def work(c):
    b = 4 if c["type"] == "f32" else 2
    T = c["T"]
    if c["kind"] == "norm":  # backward reads x and dy and writes dx
        n = T * c["H"]
        return {"bytes": b * ((5 if c["train"] else 2) * n + (4 if c["train"] else 2) * c["H"]), "flops": (20 if c["train"] else 7) * n}
    if c["kind"] == "linear":
        N, K = c["N"], c["K"]
        fwd = T * K + N * K + T * N * (2 if c["residual"] else 1) + (N if c["bias"] else 0)
        bwd = T * N + T * K + N * K + (N if c["bias"] else 0)  # dy read; dx, dW and dbias written
        return {"bytes": b * (fwd + (bwd if c["train"] else 0)), "flops": (6 if c["train"] else 2) * T * N * K}
    F, H = c["F"], c["H"]
    fwd, bwd = T * H + 2 * F * H + T * F, T * F + T * H + 2 * F * H
    return {"bytes": b * (fwd + (bwd if c["train"] else 0)), "flops": (12 if c["train"] else 4) * T * F * H}


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    c, dev, dt = case, "cuda", TYPES[case["type"]]
    gen = torch.Generator(device=dev)
    gen.manual_seed(1_000_003 * int(seed) + 29)

    def rand(*shape, scale=1.0, shift=0.0):
        return torch.randn(*shape, generator=gen, device=dev).mul_(scale).add_(shift).to(dt)

    def empty(*shape, dtype=dt):
        return torch.empty(*shape, dtype=dtype, device=dev)

    s, T = {"case": c}, c["T"]
    if c["kind"] == "norm":
        H = c["H"]
        # a residual stream: rows of different size, a few channels far above the others
        x = torch.randn(T, H, generator=gen, device=dev).add_(0.1)
        x[:, :: max(1, H // 4)] *= 8.0
        s["x"] = x.mul_(torch.rand(T, 1, generator=gen, device=dev).mul_(3.0).add_(0.3)).to(dt)
        s["weight"], s["bias"] = rand(H, scale=0.1, shift=1.0), rand(H, scale=0.1)
        s["y"] = empty(T, H)
        if c["train"]:
            s["dy"], s["dx"], s["dweight"], s["dbias"] = rand(T, H), empty(T, H), empty(H), empty(H)
            s["mean"], s["rstd"] = empty(T, dtype=torch.float32), empty(T, dtype=torch.float32)
        return s
    s["status"] = torch.zeros(1, dtype=torch.int32, device=dev)
    if c["kind"] == "linear":
        N, K = c["N"], c["K"]
        s["x"], s["W"] = rand(T, K), rand(N, K, scale=1 / math.sqrt(K))
        s["bias"] = rand(N, scale=0.1) if c["bias"] else None
        s["residual"] = rand(T, N) if c["residual"] else None
        s["y"] = empty(T, N)
        if c["train"]:
            s["dy"], s["dx"], s["dW"] = rand(T, N), empty(T, K), empty(N, K)
            s["slope"] = empty(T, N) if c["act"] != "none" else None
            s["dbias"] = empty(N) if c["bias"] else None
        return s
    F, H = c["F"], c["H"]
    s["x"], s["W1"], s["h"] = rand(T, H), rand(2 * F, H, scale=1 / math.sqrt(H)), empty(T, F)
    if c["train"]:
        s["factors"], s["dh"], s["dx"], s["dW1"] = empty(T, 2 * F), rand(T, F), empty(T, H), empty(2 * F, H)
    return s


# ---------------------------------------------------------------- the plain forms

def _act(a, name):
    """act(a) and its derivative, elementwise."""
    if name == "none":
        return a, torch.ones_like(a)
    if name == "silu":
        s = 1 / (1 + (-a).exp())
        return a * s, s * (1 + a * (1 - s))
    if name == "gelu":
        cdf = 0.5 * (1 + torch.erf(a * math.sqrt(0.5)))
        return a * cdf, cdf + a * (-0.5 * a * a).exp() * (1 / math.sqrt(2 * math.pi))
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (a + 0.044715 * a ** 3))
    return 0.5 * a * (1 + t), 0.5 * (1 + t) + 0.5 * a * (1 - t * t) * k * (1 + 3 * 0.044715 * a * a)


def _plain_norm(s):
    c, x, w = s["case"], s["x"].float(), s["weight"].float()
    d = x - x.mean(1, keepdim=True)
    rstd = 1 / ((d * d).mean(1, keepdim=True) + EPS).sqrt()
    n = d * rstd
    out = {"y": n * w + s["bias"].float()}
    if c["train"]:
        dy = s["dy"].float()
        g = dy * w
        out["dx"] = rstd * (g - g.mean(1, keepdim=True) - n * (g * n).mean(1, keepdim=True))
        out["dweight"], out["dbias"] = (dy * n).sum(0), dy.sum(0)
    return out


def _plain_linear(s):
    c, x, W = s["case"], s["x"].float(), s["W"].float()
    pre = x @ W.t()
    if c["bias"]:
        pre += s["bias"].float()
    y, slope = _act(pre, c["act"])
    out = {"y": y + s["residual"].float() if c["residual"] else y}
    if c["train"]:
        dpre = s["dy"].float() * slope
        out["dx"], out["dW"] = dpre @ W, dpre.t() @ x
        if c["bias"]:
            out["dbias"] = dpre.sum(0)
    return out


def _plain_gated(s):
    c, x, W1 = s["case"], s["x"].float(), s["W1"].float()
    gate, up = (x @ W1.t()).split(c["F"], 1)
    a, slope = _act(gate, c["act"])
    out = {"h": a * up}
    if c["train"]:
        dh = s["dh"].float()
        d = torch.cat((dh * up * slope, dh * a), 1)
        out["dx"], out["dW1"] = d @ W1, d.t() @ x
    return out


def _plain(s):
    dt = TYPES[s["case"]["type"]]
    return {k: v.to(dt) for k, v in {"norm": _plain_norm, "linear": _plain_linear, "gated": _plain_gated}[s["case"]["kind"]](s).items()}


# ---------------------------------------------------------------- the framework's operators

def _workspace(s, size):
    if "ws" not in s:  # the workspace is the caller's, made once
        s["ws"] = torch.empty(size, dtype=torch.uint8, device=s["x"].device)
    return s["ws"]


def _framework(s):
    import combine_counting_sort_gb300 as moe
    c = s["case"]
    if c["kind"] == "norm":
        if not c["train"]:
            moe.moe_layernorm(s["x"], s["weight"], s["bias"], EPS, s["y"])
            return {"y": s["y"]}
        moe.moe_layernorm(s["x"], s["weight"], s["bias"], EPS, s["y"], mean=s["mean"], rstd=s["rstd"])
        moe.moe_layernorm_bwd(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], s["dx"], s["dweight"], s["dbias"],
                              _workspace(s, moe.moe_layernorm_bwd_ws_bytes(c["T"], c["H"])))
        return {k: s[k] for k in ("y", "dx", "dweight", "dbias")}
    act = {"none": moe.MOE_ACT_NONE, "silu": moe.MOE_ACT_SILU, "gelu": moe.MOE_ACT_GELU, "gelu_tanh": moe.MOE_ACT_GELU_TANH}[c["act"]]
    if c["kind"] == "linear":
        moe.moe_linear(s["x"], s["W"], s["y"], s["status"], bias=s["bias"], residual=s["residual"], act=act,
                       slope=s["slope"] if c["train"] else None)
        if not c["train"]:
            return {"y": s["y"]}
        moe.moe_linear_bwd(s["dy"], s["x"], s["W"], s["dx"], s["dW"], _workspace(s, moe.moe_linear_bwd_ws_bytes(c["T"], c["N"], c["K"])),
                           s["status"], dbias=s["dbias"], slope=s["slope"])
        return {k: s[k] for k in (("y", "dx", "dW", "dbias") if c["bias"] else ("y", "dx", "dW"))}
    moe.moe_gated(s["x"], s["W1"], s["h"], s["status"], act=act, factors=s["factors"] if c["train"] else None)
    if not c["train"]:
        return {"h": s["h"]}
    moe.moe_gated_bwd(s["dh"], s["x"], s["W1"], s["factors"], s["dx"], s["dW1"],
                      _workspace(s, moe.moe_gated_bwd_ws_bytes(c["T"], c["F"], c["H"])), s["status"])
    return {k: s[k] for k in ("h", "dx", "dW1")}


def run(state):
    return _framework(state) if own else _plain(state)


# ---------------------------------------------------------------- the definition, in 64 bits

def _act64(a, name):
    """act and its derivative by the functions' own definitions."""
    if name == "none":
        return a, torch.ones_like(a)
    if name == "silu":
        sig = torch.sigmoid(a)
        return a * sig, sig + a * sig * torch.sigmoid(-a)
    if name == "gelu":
        phi = 0.5 * torch.erfc(-a / math.sqrt(2.0))
        return a * phi, phi + a * torch.exp(-a.square() / 2) / math.sqrt(2.0 * math.pi)
    # 0.5 (1 + tanh z) is the logistic function of 2 z
    z = 2.0 * math.sqrt(2.0 / math.pi) * (a + 0.044715 * a * a * a)
    dz = 2.0 * math.sqrt(2.0 / math.pi) * (1.0 + 0.134145 * a * a)
    sig = torch.sigmoid(z)
    return a * sig, sig + a * sig * torch.sigmoid(-z) * dz


def exact(case, seed):
    c, s = case, prepare(case, seed)
    x = s["x"].double()
    if c["kind"] == "norm":
        w, b = s["weight"].double(), s["bias"].double()
        var, mean = torch.var_mean(x, dim=1, unbiased=False, keepdim=True)
        r = torch.rsqrt(var + EPS)
        n = (x - mean) * r
        out = {"y": torch.addcmul(b, n, w)}
        if c["train"]:
            dy, H = s["dy"].double(), c["H"]
            g = dy * w
            # the Jacobian of a row: r (I - 1 1^T / H - n n^T / H)
            s1, s2 = torch.einsum("th->t", g)[:, None], torch.einsum("th,th->t", g, n)[:, None]
            out["dx"] = r * (g - (s1 + n * s2) / H)
            out["dweight"], out["dbias"] = torch.einsum("th,th->h", dy, n), torch.einsum("th->h", dy)
        return out
    if c["kind"] == "linear":
        W = s["W"].double()
        pre = torch.einsum("tk,nk->tn", x, W)
        if c["bias"]:
            pre = pre + s["bias"].double()[None, :]
        a, slope = _act64(pre, c["act"])
        out = {"y": a + s["residual"].double() if c["residual"] else a}
        if c["train"]:
            d = s["dy"].double() * slope
            out["dx"], out["dW"] = torch.einsum("tn,nk->tk", d, W), torch.einsum("tn,tk->nk", d, x)
            if c["bias"]:
                out["dbias"] = torch.einsum("tn->n", d)
        return out
    F = c["F"]
    Wg, Wu = s["W1"][:F].double(), s["W1"][F:].double()
    g, u = torch.einsum("th,fh->tf", x, Wg), torch.einsum("th,fh->tf", x, Wu)
    a, slope = _act64(g, c["act"])
    out = {"h": a * u}
    if c["train"]:
        dh = s["dh"].double()
        dg, du = dh * u * slope, dh * a
        out["dx"] = torch.einsum("tf,fh->th", dg, Wg) + torch.einsum("tf,fh->th", du, Wu)
        out["dW1"] = torch.cat((torch.einsum("tf,th->fh", dg, x), torch.einsum("tf,th->fh", du, x)), 0)
    return out
