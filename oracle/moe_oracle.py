"""Plain float64 definitions of the steps around the grouped GEMMs: sorting
slots into rows, moving tokens there and back, the norms around the block,
the gated activation, the FP8 quantiser, and the gradients.

Test infrastructure: written from the formulas, one statement each, with no
code of the GPU package. Where a rounding is part of the definition (a
float32 scale, a float32 quotient, an FP8 code) it is made explicitly.
Functions named *_mag return the sum of the magnitudes of the terms a result
is made of, for error bounds.
"""

from __future__ import annotations

import numpy as np

from . import dg_oracle as O

BLOCK = 128
SEGMENT = 128

_E4M3 = O.e4m3_decode_table()


def e4m3_round(v) -> np.ndarray:
    """The E4M3 value nearest to each v, ties to the even code; NaN stays NaN.
    |v| must not exceed 464, from where a conversion overflows."""
    v = np.asarray(v, np.float64)
    levels = np.array([_E4M3[c] for c in range(0x7F)])    # codes 0..0x7E, increasing
    a = np.abs(np.where(np.isnan(v), 0.0, v))
    assert a.size == 0 or a.max() <= 464.0
    hi = np.clip(np.searchsorted(levels, a), 0, 0x7E)
    lo = np.maximum(hi - 1, 0)
    mid = (levels[lo] + levels[hi]) / 2
    code = np.where((a > mid) | ((a == mid) & (hi % 2 == 0)), hi, lo)
    return np.where(np.isnan(v), np.nan, np.copysign(levels[code], v))


def sort(ids, num_groups: int, layout: str, rows: int):
    """(row_of like ids, group_rows [G], grouped_layout [rows] or None)."""
    ids = np.asarray(ids)
    members = [[] for _ in range(num_groups)]
    for i, e in enumerate(ids.reshape(-1).tolist()):
        if 0 <= e < num_groups:
            members[e].append(i)
    row_of = np.full(ids.size, -1, np.int64)
    kept = np.zeros(num_groups, np.int64)
    ids_of = np.full(rows, -1, np.int64) if layout == "contiguous" else None
    start = 0
    for g, slots in enumerate(members):
        if layout == "masked":
            start = g * rows
        for k, i in enumerate(slots):
            if (k if layout == "masked" else start + k) < rows:
                row_of[i] = start + k
                kept[g] += 1
                if layout == "contiguous":
                    ids_of[start + k] = g
        start += -(-len(slots) // SEGMENT) * SEGMENT if layout == "contiguous" else len(slots)
    return row_of.reshape(ids.shape), kept, ids_of


def scales(x32, ue8m0: bool) -> np.ndarray:
    """Scales [..., blocks] of float32 x [..., blocks * 128]: max(amax, 1e-4) / 448
    in float32, with ue8m0 the smallest power of two not below that."""
    x32 = np.asarray(x32, np.float32)
    amax = np.abs(x32).reshape(*x32.shape[:-1], -1, BLOCK).max(-1)      # NaN propagates
    s = np.maximum(amax, np.float32(1e-4)) / np.float32(448)
    if ue8m0:
        mant, exp = np.frexp(s)
        up = np.ldexp(np.float32(1), np.where(mant == 0.5, exp - 1, exp)).astype(np.float32)
        s = np.where(np.isfinite(s), up, s)
    return s.astype(np.float32)


def quantize(x32, ue8m0: bool):
    """(E4M3 values like x, scales): codes of the float32 quotient x / scale."""
    s = scales(x32, ue8m0)
    with np.errstate(invalid="ignore"):
        quotient = (np.asarray(x32, np.float32) / np.repeat(s, BLOCK, -1)).astype(np.float32)
    return e4m3_round(quotient), s


def dispatch(x, row_of, out):
    """out[row_of[t, j]] = x[t] on a copy of out."""
    out = np.array(out)
    for t, j in np.argwhere(row_of >= 0):
        out[row_of[t, j]] = x[t]
    return out


def combine(yp, row_of, w=None):
    t, k = row_of.shape
    y = np.zeros((t, yp.shape[1]))
    for i in range(t):
        for j in range(k):
            if row_of[i, j] >= 0:
                y[i] += (1.0 if w is None else float(w[i, j])) * yp[row_of[i, j]]
    return y


def combine_mag(yp, row_of, w=None):
    return combine(np.abs(yp), row_of, None if w is None else np.abs(w))


def combine_bwd(dy, yp, row_of, w, dyp_out):
    """(dyp on a copy of dyp_out, dw)."""
    dyp, dw = np.array(dyp_out, np.float64), np.zeros(row_of.shape)
    for t, j in np.argwhere(row_of >= 0):
        r = row_of[t, j]
        dyp[r] = float(w[t, j]) * dy[t]
        dw[t, j] = np.dot(dy[t], yp[r])
    return dyp, dw


def _wide(gate):
    return 1.0 if gate is None else np.asarray(gate, np.float64)


def norm(v, w, eps):
    rstd = 1.0 / np.sqrt((v * v).mean(1, keepdims=True) + eps)
    return v * rstd * w, rstd[:, 0]


def block_norm(x, y, post_weight, gate, pre_weight, residual_scale, eps):
    """(h, n, rstd_post, rstd_pre); None where not computed."""
    h, n, r1, r2 = x, None, None, None
    if y is not None:
        if post_weight is not None:
            y, r1 = norm(y, post_weight, eps)
        h = residual_scale * x + _wide(gate) * y
    if pre_weight is not None:
        n, r2 = norm(h, pre_weight, eps)
    return h, n, r1, r2


def _sum_like(v, gate):
    if gate is None:
        return None
    if gate.ndim == 1:
        return v.sum(0)
    return v.sum(1, keepdims=True) if gate.shape[1] == 1 else v


def block_norm_bwd(dh, dn, h, y, post_weight, gate, pre_weight, r1, r2, residual_scale, mag: bool = False):
    """dict of dx, dy, dpost, dgate, dpre (None where not computed). With `mag`
    every input and term is taken by magnitude and every difference as a sum."""
    m = (lambda v: None if v is None else np.abs(v)) if mag else (lambda v: v)
    dh, dn, h, y, post_weight, gate, pre_weight = (m(v) for v in (dh, dn, h, y, post_weight, gate, pre_weight))
    sign = 1.0 if mag else -1.0
    out = dict.fromkeys(("dx", "dy", "dpost", "dgate", "dpre"))
    total = 0.0 if dh is None else dh
    if dn is not None:
        hn, a = h * r2[:, None], dn * pre_weight
        total = total + r2[:, None] * (a + sign * hn * (a * hn).mean(1, keepdims=True))
        out["dpre"] = (dn * hn).sum(0)
    out["dx"] = (abs(residual_scale) if mag else residual_scale) * total
    if y is None:
        return out
    yn = y if post_weight is None else y * r1[:, None]
    pw = 1.0 if post_weight is None else post_weight
    out["dgate"] = _sum_like(total * yn * pw, gate)
    b = total * _wide(gate) * pw
    if post_weight is None:
        out["dy"] = b
        return out
    out["dpost"] = (total * _wide(gate) * yn).sum(0)
    out["dy"] = r1[:, None] * (b + sign * yn * (b * yn).mean(1, keepdims=True))
    return out


def sigmoid(g):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-np.asarray(g, np.float64)))


def swiglu(gu):
    g, u = np.split(np.asarray(gu, np.float64), 2, axis=-1)
    return g * sigmoid(g) * u


def swiglu_bwd(da, gu):
    g, u = np.split(np.asarray(gu, np.float64), 2, axis=-1)
    s = sigmoid(g)
    return np.concatenate([da * u * s * (1.0 + g * (1.0 - s)), da * g * s], -1)


def held_rows(rows, layout: str, m: int, num_groups: int = 1) -> np.ndarray:
    """Truth of each row: [m], masked [G, m]."""
    rows = None if rows is None else np.asarray(rows)
    if layout == "dense":
        return np.ones(m, bool)
    if layout == "contiguous":
        return rows >= 0
    if layout == "masked":
        return np.arange(m)[None, :] < rows[:, None]
    return np.arange(m) < np.maximum(rows, 0).sum()
