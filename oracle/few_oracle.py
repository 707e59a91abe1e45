"""CPU oracle of the decoding operators: 4-bit weights with group scales, their
matrix-vector products, and a whole MoE layer for a few tokens.

TEST INFRASTRUCTURE ONLY (see moe_oracle.py).  Values are fp64; the 4-bit codes
and scales, which floating point decides, follow the stated rule exactly: the
scale is bf16(max|w| / 7) of the fp32 quotient, the code the nearest integer
(ties to even) of the fp32 quotient w / scale.
"""
import numpy as np

from .moe_oracle import bf16_to_f32, e4m3_decode, f64_to_bf16


def quantize_w4(w_bits: np.ndarray, group: int):
    """bf16 bits [..., N, K] -> codes u8 [..., N, K] in 0..15 and scale bits
    u16 [..., N, K/group]."""
    w = bf16_to_f32(w_bits)
    shape = w.shape
    w = w.reshape(*shape[:-1], shape[-1] // group, group)
    scale_bits = f64_to_bf16((np.abs(w).max(-1) / np.float32(7)).astype(np.float64))
    s = bf16_to_f32(scale_bits)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.clip(np.rint(w / s), -8, 7)
    q = np.where(s > 0, q, 0)
    return (q + 8).astype(np.uint8).reshape(shape), scale_bits


def w4_values(codes: np.ndarray, scale_bits: np.ndarray) -> np.ndarray:
    """fp64 values (c - 8) * scale."""
    group = codes.shape[-1] // scale_bits.shape[-1]
    return (codes.astype(np.float64) - 8) * np.repeat(bf16_to_f32(scale_bits).astype(np.float64), group, -1)


def pack_w4(codes: np.ndarray, scale_bits: np.ndarray) -> np.ndarray:
    """Codes [E, N, K] and scales [E, N, K/group] -> the laid-out bytes, one
    code and one scale at a time from the stated byte and nibble."""
    E, N, K = codes.shape
    group = K // scale_bits.shape[-1]
    nt, kt, G = -(-N // 16), -(-K // 128), 128 // group
    full = np.full((E, nt * 16, kt * 128), 8, np.uint8)
    full[:, :N, :K] = codes
    fs = np.zeros((E, nt * 16, kt * G), np.uint16)
    fs[:, :N, :K // group] = scale_bits
    out = np.zeros((E, nt, kt, 1024 + 32 * G), np.uint8)
    for r in range(16):
        half, g = r // 8, r % 8
        for c in range(128):
            j, t, i, b = c // 32, c % 32 // 8, c % 4 // 2, 2 * (c % 2) + c % 8 // 4
            byte = 4 * (4 * (32 * half + 4 * g + t) + j) + b
            out[..., byte] |= full[:, r::16, c::128] << (4 * i)
        for q in range(G):
            v = fs[:, r::16, q::G]
            out[..., 1024 + 2 * (16 * q + r)] = v & 255
            out[..., 1024 + 2 * (16 * q + r) + 1] = v >> 8
    return out


def fp8_values(codes: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """fp64 values of e4m3 codes [N, K] with scales [N/128, K/128]."""
    s = np.repeat(np.repeat(scale.astype(np.float64), 128, 0), 128, 1)
    return e4m3_decode(codes).astype(np.float64) * s


def matvec(x: np.ndarray, W: np.ndarray):
    """x [T, K], W [N, K] in fp64 -> y [T, N] and the sums of magnitudes that
    bound its rounding errors."""
    return x @ W.T, np.abs(x) @ np.abs(W).T


# Rounding: bf16 keeps 8 significant bits, so one rounding is within 2^-8 of the
# value; f16 11, fp32 24.  A product of two bf16 values (or bf16 and a 4-bit or e4m3
# code) is exact in fp32, so a sum of n products with group scales applied to
# partial sums has at most n + 2 roundings of 2^-24 of the magnitudes' sum.
U_BF16, U_F16, U_F32 = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24


def record_step(v: np.ndarray) -> np.ndarray:
    """How far a value of v [.., K] may be moved where the products take it as f16 behind a power of
    two that its 128 columns share: their largest comes to 2^14 or more, f16's values end in steps of 2^-24."""
    K = v.shape[-1]
    most = np.abs(np.pad(v, [(0, 0)] * (v.ndim - 1) + [(0, -K % 128)])).reshape(*v.shape[:-1], -1, 128).max(-1)
    return np.repeat(most, 128, -1)[..., :K] * 2.0 ** -39


def matvec_bound(x: np.ndarray, W: np.ndarray):
    """(y, how far a bf16 result of fp32 sums may be from y), elementwise."""
    y, mag = matvec(x, W)
    err = (W.shape[1] + 2) * U_F32 * mag + record_step(x) @ np.abs(W).T
    return y, U_BF16 * (np.abs(y) + err) + err + 2.0 ** -133   # half a bf16 subnormal step


def layer_few(x: np.ndarray, ids: np.ndarray, w: np.ndarray, experts: dict):
    """x [T, H] fp64, ids / w [T, k], experts[e] = (W1 [2F, H], W2 [H, F]) fp64.
    Ids outside `experts` have no route.  Returns (out, bound): the fp64
    layer and how far a bf16 result may be from it, elementwise, where sums are
    fp32, w * silu(g) * u is rounded to f16 once, behind a power of two that 128 features share,
    and expf is good to 2^-21."""
    T, H = x.shape
    out, err = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        n_terms, moved = 2, np.zeros(H)   # terms of this token's sums, and their magnitudes' sum
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if e not in experts:
                continue
            W1, W2 = experts[e]
            F = W2.shape[1]
            n_terms += F + 1
            y, mag = matvec(x[t:t + 1], W1)
            dy = (H + 2) * U_F32 * mag[0] + np.abs(W1) @ record_step(x[t])
            g, u = y[0, :F], y[0, F:]
            sig = 1 / (1 + np.exp(-g))
            silu = g * sig
            a = float(w[t, j]) * silu * u
            # |silu'| <= 1.1; exp's argument error is inside dy; sigmoid's own relative error 2^-20
            da = abs(float(w[t, j])) * (1.1 * dy[:F] * (np.abs(u) + dy[F:]) + np.abs(silu) * dy[F:] + 2.0 ** -19 * np.abs(silu * u))
            da = da + U_F16 * (np.abs(a) + da) + record_step(np.abs(a) + da)
            out[t] += W2 @ a
            err[t] += np.abs(W2) @ da
            moved += np.abs(W2) @ (np.abs(a) + da)
        err[t] += n_terms * U_F32 * moved
    return out, U_BF16 * (np.abs(out) + err) + err + 2.0 ** -133
