"""Plain float64 definitions of microscaled FP4 (E2M1 codes with one power of
two per 32 values): the quantiser, what an operand stands for, the products,
and expert layers for a few tokens.

Test infrastructure: written from the formulas, with no code of the GPU package.
"""

from __future__ import annotations

import numpy as np

from . import dg_oracle as O
from . import moe_oracle as M

MX = 32
LEVELS = np.array([O.e2m1_value(c) for c in range(8)])      # 0, .5, 1, 1.5, 2, 3, 4, 6
NAN_SCALE = 255


def scale_codes(x) -> np.ndarray:
    """E8M0 codes [..., K/32] of float64 x [..., K]: of the smallest power of two
    not below amax / 6, at least 2^-127; 255 where a block is not finite or its
    largest value is one that float32 rounds to infinity."""
    x = np.asarray(x, np.float64)
    amax = np.abs(x).reshape(*x.shape[:-1], x.shape[-1] // MX, MX).max(-1)
    with np.errstate(over="ignore", invalid="ignore"):
        bad = ~np.isfinite(amax.astype(np.float32))
    exponent = np.full(amax.shape, -127)
    for e in range(-126, 127):
        exponent = np.where(amax > 6.0 * 2.0 ** (e - 1), e, exponent)
    return np.where(bad, NAN_SCALE, exponent + 127).astype(np.uint8)


def codes(x, scales) -> np.ndarray:
    """E2M1 codes (sign bit 3) like x, of x / scale rounded to the nearest level,
    ties to the even one; 0 under a NaN scale."""
    x = np.asarray(x, np.float64)
    s = np.repeat(scales.astype(np.int64), MX, -1)
    dead = s == NAN_SCALE
    a = np.ldexp(np.where(dead, 0.0, np.abs(x)), 127 - np.where(dead, 127, s))
    hi = np.clip(np.searchsorted(LEVELS, a), 0, 7)
    lo = np.maximum(hi - 1, 0)
    mid = (LEVELS[lo] + LEVELS[hi]) / 2
    code = np.where((a > mid) | ((a == mid) & (hi % 2 == 0)), hi, lo)
    return np.where(dead, 0, code + 8 * np.signbit(np.where(dead, 0.0, x))).astype(np.uint8)


def pack(code) -> np.ndarray:
    return code[..., 0::2] | code[..., 1::2] << 4


def words(scales) -> np.ndarray:
    """Scale codes [..., rows, K/32] as the products take them: [..., K/128, rows] uint32."""
    s = scales.astype(np.uint32).reshape(*scales.shape[:-1], scales.shape[-1] // 4, 4)
    w = s[..., 0] | s[..., 1] << 8 | s[..., 2] << 16 | s[..., 3] << 24
    return np.swapaxes(w, -1, -2)


def quantize(x):
    """(packed codes [..., K/2] uint8, scale words [..., K/128, rows] uint32)."""
    s = scale_codes(x)
    return pack(codes(x, s)), words(s)


def values(packed, sf) -> np.ndarray:
    """What packed codes [..., rows, K/2] and words [..., K/128, >= rows] stand for."""
    w = np.swapaxes(np.asarray(sf).astype(np.uint32)[..., : packed.shape[-2]], -1, -2)
    s = np.stack([(w >> (8 * i)) & 255 for i in range(4)], -1).reshape(*w.shape[:-1], -1).astype(np.int64)
    scale = np.where(s == NAN_SCALE, np.nan, np.ldexp(1.0, np.where(s == NAN_SCALE, 0, s) - 127))
    return O.e2m1_decode_table()[O.unpack_e2m1(packed)] * np.repeat(scale, MX, -1)


def gemm(a, sfa, b, sfb):
    """(products' sums, sums of their magnitudes) of one pair of operands."""
    ahat, bhat = values(a, sfa), values(b, sfb)
    return ahat @ bhat.T, np.abs(ahat) @ np.abs(bhat).T


def experts(x, ids, w, w1, w2):
    """(y, act_mag, mag, top) of y[t] = sum_j w[t, j] W2[e] (silu(g) u), [g | u] =
    W1[e] x[t], e = ids[t, j]; ids outside [0, G) add nothing. act_mag: the second sum
    with the magnitudes of its terms; mag: the same with each activation's first-order
    dependence on its two sums, their terms by magnitude (|d silu / dg| is at most
    1.1); top: the largest |g|."""
    inner, top = w1.shape[1] // 2, 0.0
    y, act_mag, mag = (np.zeros((x.shape[0], w2.shape[1])) for _ in range(3))
    for t in range(x.shape[0]):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if not 0 <= e < w1.shape[0]:
                continue
            gu, gm = w1[e] @ x[t], np.abs(w1[e]) @ np.abs(x[t])
            g, u = gu[:inner], gu[inner:]
            s = g * M.sigmoid(g)
            top = max(top, np.abs(g).max())
            y[t] += float(w[t, j]) * (w2[e] @ (s * u))
            act_mag[t] += abs(float(w[t, j])) * (np.abs(w2[e]) @ np.abs(s * u))
            mag[t] += abs(float(w[t, j])) * (np.abs(w2[e]) @ (np.abs(s) * gm[inner:] + 1.1 * gm[:inner] * np.abs(u)))
    return y, act_mag, mag, top
