"""Plain definitions of the 4-bit weights' operators (numpy, CPU, 64 bits).

The quantiser is given in fp32 with the operations that include/bsp.h names,
so that codes, scales and zero points can be compared bit for bit.  Test
infrastructure only.
"""
from __future__ import annotations

import numpy as np

F = np.float32


def to_bf16(x):
    """fp32 -> the nearest bfloat16 (ties to even), as fp32."""
    u = np.asarray(x, F).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(F)
    return np.where(np.isnan(x), F(np.nan), r)


def to_f16(x):
    with np.errstate(over="ignore"):
        return np.asarray(x, F).astype(np.float16).astype(F)


ROUND = {"float16": to_f16, "bfloat16": to_bf16}


def quantise(W, dtype: str, group: int, zeros: bool):
    """(codes [M][K], scales [M][groups] fp32, zero points [M][groups]) of W [M][K] (fp32)."""
    M, K = W.shape
    groups = -(-K // group)
    codes = np.zeros((M, K), np.uint8)
    scales, zp = np.zeros((M, groups), F), np.full((M, groups), 8, np.uint8)
    with np.errstate(all="ignore"):
        for g in range(groups):
            w = W[:, g * group:(g + 1) * group].astype(F)
            fine = np.where(np.isfinite(w), w, F(0))
            lo, hi = np.minimum(fine.min(1), F(0)), np.maximum(fine.max(1), F(0))
            s = ROUND[dtype](hi / F(15) - lo / F(15) if zeros else np.maximum(hi, -lo) / F(7))
            z = np.full(M, 8, F)
            if zeros:
                z = np.where(s > 0, np.clip(np.rint(-lo / s), F(0), F(15)), F(8)).astype(F)
            q = np.clip(np.rint(w / s[:, None]) + z[:, None], F(0), F(15))
            q = np.where((s[:, None] > 0) & ~np.isnan(w), q, z[:, None])
            codes[:, g * group:(g + 1) * group] = q.astype(np.uint8)
            scales[:, g], zp[:, g] = s, z.astype(np.uint8)
    return codes, scales, zp


def pack(codes):
    """[M][K] codes -> [M][K / 2] bytes, the even column in the low half."""
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack(packed):
    out = np.empty((packed.shape[0], 2 * packed.shape[1]), np.uint8)
    out[:, 0::2], out[:, 1::2] = packed & 15, packed >> 4
    return out


def dense(codes, scales, zeros, group: int):
    """W [M][K] in 64 bits; zeros None: 8 throughout."""
    K = codes.shape[1]
    z = 8.0 if zeros is None else np.repeat(zeros.astype(np.float64), group, 1)[:, :K]
    return (codes.astype(np.float64) - z) * np.repeat(scales.astype(np.float64), group, 1)[:, :K]


def product(X, codes, scales, zeros, group: int):
    """Y [N][M] = W X."""
    return X.astype(np.float64) @ dense(codes, scales, zeros, group).T


def act(g, name: str):
    if name == "silu":
        with np.errstate(over="ignore"):
            return g / (1 + np.exp(-g))
    if name == "gelu":
        from scipy.special import erfc
        return 0.5 * g * erfc(-g / np.sqrt(2))
    if name == "gelu_tanh":
        return 0.5 * g * (1 + np.tanh(np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)))
    return np.maximum(g, 0)


def error_bound(X, codes, scales, zeros, group: int, dtype: str = None, n_parts: int = 64):
    """Bound of a product's error before its last rounding, [N][M].

    A group's products are exact in fp32 (an activation's 11 or 8 bits times
    the 5 of code - zero).  Its sums run over at most group / 16 additions to an
    fp32 sum, each of 16 products at once with an error of at most 2^-22 of
    the largest magnitude met (a tensor core may truncate the terms it
    aligns, and its sum); the largest magnitude is at most top = 15 sum |x|.
    The scaled sums of groups, and the parts of warps and of CTAs, are added in
    fp32: their number + n_parts roundings of 2^-24 of the sum of magnitudes."""
    K = codes.shape[1]
    x = np.abs(X.astype(np.float64))
    groups = -(-K // group)
    inner, outer = np.zeros((X.shape[0], codes.shape[0])), np.zeros((X.shape[0], codes.shape[0]))
    w = np.abs(dense(codes, scales, zeros, group))
    for g in range(groups):
        cols = slice(g * group, (g + 1) * group)
        top = x[:, cols].sum(1)[:, None] * 15
        inner += top * np.abs(scales[:, g].astype(np.float64))[None] * ((group / 16 + 2) * 2.0 ** -22)
        outer += x[:, cols] @ w[:, cols].T
    return inner + outer * (groups + n_parts) * 2.0 ** -24


HALF_STEP = {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}    # eps / 2
TINY = {"float16": 2.0 ** -25, "bfloat16": 2.0 ** -134}       # half of the smallest subnormal


def gated_bound(g, u, eg, eu, name: str):
    """Bound of act(g) u before its last rounding, for errors eg, eu of g and u.

    |act'| <= 1.13 for all four (silu 1.0998, gelu 1.1290); the activation
    itself is computed in fp32 with a relative error of at most 2^-18 (its
    exponential's argument is at most 2^7 where the result is not 0, off by
    2^-24 of itself: 2^-17 only where act(g) is within |g| exp(-|g|); and the
    product rounds)."""
    a = act(g, name)
    da = 1.13 * eg + 2.0 ** -18 * np.abs(a) + 2.0 ** -17 * np.abs(g) * np.exp(-np.abs(g)) + 1e-37
    return da * (np.abs(u) + eu) + np.abs(a) * eu
