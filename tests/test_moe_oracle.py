"""Pins of the float64 definitions of the steps around the GEMMs (CPU):
hand-derived cases, torch's FP8 conversion, and every gradient formula
against central differences of the forward definition."""

import numpy as np
import pytest
import torch

from oracle import moe_oracle as M


def test_e4m3_round_matches_torch_conversion():
    v = np.concatenate([np.linspace(-448, 448, 20001), np.random.default_rng(0).normal(0, 1, 20000) * 0.05,
                        [0.0, 2.0 ** -9, 2.0 ** -10, 1.5 * 2.0 ** -9, 17.0, 19.0, 464.0, -464.0]]).astype(np.float32)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(M.e4m3_round(v), want)
    assert np.isnan(M.e4m3_round([np.nan]))[0]


def test_sort_by_hand():
    ids = np.array([[1, 0], [1, -1], [3, 1], [2, 1]])
    row_of, kept, _ = M.sort(ids, 3, "nopad", 8)          # id 3 is out of range: dropped
    assert row_of.tolist() == [[1, 0], [2, -1], [-1, 3], [5, 4]] and kept.tolist() == [1, 4, 1]
    row_of, kept, _ = M.sort(ids, 3, "nopad", 4)          # rows at or past 4 are dropped
    assert row_of.tolist() == [[1, 0], [2, -1], [-1, 3], [-1, -1]] and kept.tolist() == [1, 3, 0]
    row_of, kept, _ = M.sort(ids, 3, "masked", 3)
    assert row_of.tolist() == [[3, 0], [4, -1], [-1, 5], [6, -1]] and kept.tolist() == [1, 3, 1]
    row_of, kept, layout = M.sort(ids, 3, "contiguous", 384)
    assert row_of.tolist() == [[128, 0], [129, -1], [-1, 130], [256, 131]] and kept.tolist() == [1, 4, 1]
    assert np.flatnonzero(layout >= 0).tolist() == [0, 128, 129, 130, 131, 256]


def test_quantize_by_hand():
    x = np.zeros((1, 256), np.float32)
    x[0, :3] = [448.0, 17.0, -19.0]                       # scale 1; 17 and 19 are ties of E4M3
    q, s = M.quantize(x, False)
    assert s.tolist() == [[1.0, np.float32(np.float32(1e-4) / np.float32(448))]]
    assert q[0, :3].tolist() == [448.0, 16.0, -20.0] and not q[0, 3:].any()
    x[0, 0] = 449.0
    assert M.scales(x, True)[0, 0] == 2.0 and M.scales(x / 2, True)[0, 0] == 1.0


def _difference(f, v, i, step=1e-5):
    up, down = v.copy(), v.copy()
    up.flat[i] += step
    down.flat[i] -= step
    return (f(up) - f(down)) / (2 * step)


def test_combine_gradient_against_differences():
    r = np.random.default_rng(1)
    yp, w, dy = r.normal(size=(9, 6)), r.normal(size=(4, 3)), r.normal(size=(4, 6))
    row_of = np.array([[0, 5, -1], [8, 2, 1], [-1, -1, -1], [3, 4, 7]])
    dyp, dw = M.combine_bwd(dy, yp, row_of, w, np.zeros_like(yp))
    for i in range(yp.size):
        assert abs(_difference(lambda v: (M.combine(v, row_of, w) * dy).sum(), yp, i) - dyp.flat[i]) < 1e-7
    for i in range(w.size):
        if row_of.flat[i] >= 0:
            assert abs(_difference(lambda v: (M.combine(yp, row_of, v) * dy).sum(), w, i) - dw.flat[i]) < 1e-7
    # the dispatch's gradient is the combine with unit weights
    x, dxp = r.normal(size=(4, 6)), r.normal(size=(9, 6))
    dx = M.combine(dxp, row_of)
    for i in range(x.size):
        assert abs(_difference(lambda v: (M.dispatch(v, row_of, np.zeros((9, 6))) * dxp).sum(), x, i) - dx.flat[i]) < 1e-7


@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("post", [True, False])
def test_block_norm_gradient_against_differences(gate, post):
    r = np.random.default_rng(2)
    t, h, rs, eps = 3, 8, 0.7, 1e-3
    v = {"x": r.normal(size=(t, h)), "y": r.normal(size=(t, h)), "pre": r.normal(size=h)}
    if post:
        v["post"] = r.normal(size=h)
    if gate != "none":
        v["gate"] = r.normal(size={"channel": (h,), "token": (t, 1), "full": (t, h)}[gate])
    dh, dn = r.normal(size=(t, h)), r.normal(size=(t, h))

    def loss(**kw):
        d = {**v, **kw}
        a, b, _, _ = M.block_norm(d["x"], d["y"], d.get("post"), d.get("gate"), d["pre"], rs, eps)
        return (a * dh).sum() + (b * dn).sum()

    a, _, r1, r2 = M.block_norm(v["x"], v["y"], v.get("post"), v.get("gate"), v["pre"], rs, eps)
    g = M.block_norm_bwd(dh, dn, a, v["y"], v.get("post"), v.get("gate"), v["pre"], r1, r2, rs)
    for name, key in (("x", "dx"), ("y", "dy"), ("pre", "dpre"), ("post", "dpost"), ("gate", "dgate")):
        if name not in v:
            assert g[key] is None
            continue
        for i in range(v[name].size):
            assert abs(_difference(lambda u: loss(**{name: u}), v[name], i) - g[key].flat[i]) < 1e-6, (name, i)


def test_swiglu_gradient_against_differences():
    r = np.random.default_rng(3)
    gu, da = r.normal(size=(3, 16)) * 3, r.normal(size=(3, 8))
    d = M.swiglu_bwd(da, gu)
    for i in range(gu.size):
        assert abs(_difference(lambda v: (M.swiglu(v) * da).sum(), gu, i) - d.flat[i]) < 1e-7
    assert np.all(M.swiglu(np.array([[-800.0, 1.0]])) == 0) and M.swiglu(np.array([[50.0, 2.0]])) == 100.0


def test_held_rows():
    assert M.held_rows([2, -3, 1], "nopad", 5).tolist() == [True] * 3 + [False] * 2
    assert M.held_rows([9, -1], "masked", 2).tolist() == [[True, True], [False, False]]
    assert M.held_rows([0, -1, 4], "contiguous", 3).tolist() == [True, False, True]
