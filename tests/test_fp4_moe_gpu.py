"""GPU parity of the steps around the FP4 products: tokens quantised on the way to
their rows, and the quantised activation. Codes and scale words are compared with
the float64 definitions bit for bit."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from moe_grouped_gemm_amd import dg, moe
from oracle import fp4_oracle as F
from oracle import moe_oracle as M
from parity import bf16_ulp, element_bound
from test_moe_gpu import GLUS, LARGE_MOVES, LONG_GLUS, MOVES, _check_sorted, _f64, _glu_inputs, _moved, _randn

pytestmark = pytest.mark.gpu

WORD, BYTE = 0x5A5A5A5A, 0xA5


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()
    return torch.device("cuda:0")


def _say(msg):
    print(msg, flush=True)


def _special(x):
    """NaN, infinities, zeros, subnormals and ties in some blocks of x."""
    b = x.view(-1, 32)
    n = b.shape[0]
    b[n - 1] = 0.0
    b[n // 2, 5] = float("nan")
    b[n // 3, 7] = float("inf")
    b[n // 5] *= 2.0 ** -126
    b[0] = torch.tensor([6.0, 0.25, -0.75, 1.25, 1.75, -2.5, 3.5, 5.0] + [-0.0] * 24).to(b)
    return x


def _room(codes_shape, scale_shape, dev):
    return (torch.full(codes_shape, BYTE, dtype=torch.uint8, device=dev),
            torch.full(scale_shape, WORD, dtype=torch.int32, device=dev))


def _check(q, sf, x, held, what=""):
    """q [..., rows, K/2] and sf hold the operand of x (float64, like q's rows) where `held`,
    and what was there before elsewhere."""
    want_q, want_sf = F.quantize(x)
    got_q, got_sf = q.cpu().numpy(), sf.cpu().numpy().astype(np.uint32)
    rows = q.shape[-2]
    np.testing.assert_array_equal(got_q[held], want_q[held], what)
    assert (got_q[~held] == BYTE).all(), what
    word_held = np.zeros(got_sf.shape, bool)
    word_held[..., :rows] = held[..., None, :]
    np.testing.assert_array_equal(got_sf[word_held], want_sf[word_held[..., :rows]], what)
    assert (got_sf[~word_held] == WORD).all(), what


def _dispatch(dev, case, with_sort, special):
    layout, t, k, g, hidden, rows = case
    plan, ids, ids_d = _moved(*case, dev)
    x = _randn(t, hidden, seed=2, scale=3.0)
    if special:
        x = _special(x)
    q, sf = _room(plan.codes_shape, plan.scale_shape, dev)
    if not with_sort:
        moe.sort(plan, ids_d)
    moe.dispatch_fp4(plan, x, q, sf, topk_ids=ids_d if with_sort else None)
    row_of = _check_sorted(plan, ids)
    total = q.numel() // (hidden // 2)
    held = np.zeros(total, bool)
    held[row_of[row_of >= 0]] = True
    xp = M.dispatch(_f64(x), row_of, np.zeros((total, hidden)))
    lead = q.shape[:-1]
    _check(q, sf, xp.reshape(*lead, hidden), held.reshape(lead))


@pytest.mark.parametrize("special", [False, True])
@pytest.mark.parametrize("with_sort", [True, False])
@pytest.mark.parametrize("case", MOVES)
def test_dispatch_fp4(dev, case, with_sort, special):
    _say(f"dispatch_fp4 {case} sort={with_sort} special={special}")
    _dispatch(dev, case, with_sort, special)


@pytest.mark.parametrize("case", LARGE_MOVES)
def test_dispatch_fp4_many_slots(dev, case):
    _say(f"dispatch_fp4 {case}")
    _dispatch(dev, case, True, True)


def _glu(dev, case, gu=None):
    layout, g, r, inner = case
    rows, made, held = _glu_inputs(layout, g, r, inner, dev)
    gu = made if gu is None else gu
    m = gu.shape[-2]
    q, sf = _room((*gu.shape[:-1], inner // 2), (*gu.shape[:-2], inner // 128, dg.get_tma_aligned_size(m, 4)), dev)
    moe.swiglu_fp4(gu, q, sf, rows=rows, layout=layout)
    a = np.zeros((*gu.shape[:-1], inner))
    a[held] = M.swiglu(_f64(gu)[held])
    _check(q, sf, a, held, str(case))


@pytest.mark.parametrize("case", GLUS + LONG_GLUS)
def test_swiglu_fp4(dev, case):
    _say(f"swiglu_fp4 {case}")
    _glu(dev, case)


@pytest.mark.parametrize("scale", [0.02, 1.0, 30.0])
def test_swiglu_fp4_many_values(dev, scale):
    """Six million values, some tens of which lie within float32's error of a border."""
    _say(f"swiglu_fp4 many values, scale {scale}")
    gu = _randn(3000, 4096, seed=int(scale * 100), scale=scale)
    _glu(dev, ("dense", 1, 3000, 2048), gu)


def test_swiglu_fp4_many_values_of_low_gates(dev):
    """Gates between -87 and -20, whose exponential is off by up to 2^-16: two million values."""
    _say("swiglu_fp4 many values of low gates")
    gen = torch.Generator().manual_seed(9)
    base = -21.0 - 65.0 * torch.rand(1000, 64, 1, generator=gen)               # a block's gates are alike
    gate = (base + 2.0 * torch.rand(1000, 64, 32, generator=gen) - 1.0).reshape(1000, 2048)
    up = torch.randn(1000, 2048, generator=gen) * 2.0 ** 60
    _glu(dev, ("dense", 1, 1000, 2048), torch.cat([gate, up], 1).to(torch.bfloat16).to(dev))


def test_swiglu_fp4_on_the_borders(dev):
    """silu(g) u of chosen g and u next to borders between codes, and next to those
    between scales."""
    _say("swiglu_fp4 on the borders")
    g = torch.linspace(-6.0, 6.0, 4096).to(torch.bfloat16)
    s = M.swiglu(torch.cat([g, torch.ones_like(g)]).double().numpy())          # silu(g)
    border = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])[np.arange(4096) % 8]
    with np.errstate(divide="ignore"):
        u = torch.from_numpy(np.clip(np.where(s == 0, 0, border / s), -1e30, 1e30)).to(torch.bfloat16)
    gu = torch.cat([g, u]).view(1, -1).repeat(3, 1)
    gu[1, :4096:32], gu[1, 4096::32] = 40.0, 0.15                              # a block's largest is 6 at most
    gu[2, :4096:32], gu[2, 4096::32] = 64.0, 0.09375                           # and 6 itself, where silu(64) is 64
    _glu(dev, ("dense", 1, 3, 4096), gu.to(dev))


def test_swiglu_fp4_special_values(dev):
    _say("swiglu_fp4 special values")
    inner = 256
    gu = _randn(9, 2 * inner, seed=50)
    gu[0] = 0
    gu[1, 3] = float("nan")                        # g of block 0
    gu[2, inner + 40] = float("inf")               # u of block 1
    gu[3, :inner] = -200.0                         # the exponential is infinite in float32
    gu[3, inner:] *= 2.0 ** 120
    gu[4, :inner] = 200.0
    gu[5, :inner] = torch.linspace(-95.0, -80.0, inner)
    gu[5, inner:] = 2.0 ** 126
    gu[6] *= 2.0 ** -60                            # products of 2^-120
    gu[7, :inner], gu[7, inner:] = 2.0 ** 64, 2.0 ** 64          # 2^128: infinite in float32
    gu[8, 10] = -float("inf")                      # -inf * 0: NaN
    gu[8, 200], gu[8, inner + 200] = 2.0 ** 100, 2.0 ** 27.9
    _glu(dev, ("dense", 1, 9, inner), gu)


def test_swiglu_fp4_next_to_overflow(dev):
    """Gates and ups whose product is 2^128 (1 - 1.1e-7), the largest below float32's overflow of all BF16 pairs
    and finite, 2^128 (1 - 1.3e-14) and 2^128, which round to infinity, and 2^128 (1 + 6e-6)."""
    _say("swiglu_fp4 next to overflow")
    inner = 256
    gu = _randn(8, 2 * inner, seed=52)
    for row, (g, u) in enumerate(((16.0, 2.0 ** 124), (32.0, 2.0 ** 123), (2.0 ** 64, 2.0 ** 64), (5.96875, 1.34375 * 2.0 ** 125))):
        for i, sign in ((row, 1.0), (row + 4, -1.0)):
            gu[i, 40], gu[i, inner + 40] = g, sign * u
            gu[i, 200], gu[i, inner + 200] = g, sign * u / 2
    _glu(dev, ("dense", 1, 8, inner), gu)


def test_offsets_past_32_bits(dev):
    """Rows and values past 2^31: the last ones."""
    _say("fp4 offsets past 32 bits")
    hidden, rows = 7168, 300_032
    plan = moe.Plan(4, 2, 8, "nopad", rows, hidden, dev)
    row_of = np.array([[rows - 1, 0], [rows - 2, -1], [5, rows - 300], [1, 2]])
    plan.row_of.copy_(torch.from_numpy(row_of.astype(np.int32)))
    x = _randn(4, hidden, seed=60)
    q, sf = torch.zeros(plan.codes_shape, dtype=torch.uint8, device=dev), torch.zeros(plan.scale_shape, dtype=torch.int32, device=dev)
    moe.dispatch_fp4(plan, x, q, sf)
    want_q, want_sf = F.quantize(_f64(x))
    for i, j in np.argwhere(row_of >= 0):
        r = row_of[i, j]
        np.testing.assert_array_equal(q[r].cpu().numpy(), want_q[i])
        np.testing.assert_array_equal(sf[:, r].cpu().numpy().astype(np.uint32), want_sf[:, i])
    back = torch.empty(rows, hidden, dtype=torch.bfloat16, device=dev)     # 4.3e9 bytes
    dg.dequantize_fp4(q, sf, back)
    np.testing.assert_array_equal(_f64(back[rows - 1]), F.values(want_q, want_sf)[0])
    back[-1] = x[2]
    dg.quantize_fp4(back, q, sf)
    np.testing.assert_array_equal(q[-1].cpu().numpy(), want_q[2])
    np.testing.assert_array_equal(sf[:, rows - 1].cpu().numpy().astype(np.uint32), want_sf[:, 2])
    del back
    inner, m = 2048, 524_800
    gu = torch.zeros(m, 2 * inner, dtype=torch.bfloat16, device=dev)
    gu[-3:] = _randn(3, 2 * inner, seed=61)
    q, sf = _room((m, inner // 2), (inner // 128, m), dev)
    moe.swiglu_fp4(gu, q, sf)
    want_q, want_sf = F.quantize(M.swiglu(_f64(gu[-3:])))
    np.testing.assert_array_equal(q[-3:].cpu().numpy(), want_q)
    np.testing.assert_array_equal(sf[:, -3:].cpu().numpy().astype(np.uint32), want_sf)


@pytest.mark.parametrize("layout", ["masked", "nopad", "contiguous"])
def test_a_block_in_fp4(dev, layout):
    """Dispatch, product, activation, product and combine, as a layer runs them: each
    product against its own operands, and the layer against the definition with its
    operands' roundings."""
    _say(f"a block in FP4, {layout}")
    t, k, g, hidden, inner = 61, 3, 5, 384, 256
    rows = {"masked": 40, "nopad": None, "contiguous": None}[layout]
    plan, ids, ids_d = _moved(layout, t, k, g, hidden, rows, dev)
    x = _randn(t, hidden, seed=3)
    w1, w2 = _randn(g, 2 * inner, hidden, seed=4, scale=0.06), _randn(g, hidden, inner, seed=5, scale=0.06, dtype=torch.float32)

    def operand(shape):
        *lead, m, c = shape
        return (torch.zeros(*lead, m, c // 2, dtype=torch.uint8, device=dev),
                torch.zeros(*lead, c // 128, dg.get_tma_aligned_size(m, 4), dtype=torch.int32, device=dev))

    b1, b2 = dg.quantize_fp4(w1, *operand(w1.shape)), dg.quantize_fp4(w2, *operand(w2.shape))
    gemm = {"masked": dg.m_grouped_fp4_gemm_nt_masked, "nopad": dg.m_grouped_fp4_gemm_nt_nopad,
            "contiguous": dg.m_grouped_fp4_gemm_nt_contiguous}[layout]
    lead = plan.rows_shape[:-1]
    gu, yp = (torch.zeros(*lead, n, dtype=torch.bfloat16, device=dev) for n in (2 * inner, hidden))
    weights = torch.rand(t, k, device=dev)
    q1, q2 = operand((*lead, hidden)), operand((*lead, inner))
    moe.dispatch_fp4(plan, x, *q1, topk_ids=ids_d)
    of = plan.grouped_layout if layout == "contiguous" else plan.group_rows
    gemm(*q1, *b1, gu, of)
    moe.swiglu_fp4(gu, *q2, rows=of, layout=layout)
    gemm(*q2, *b2, yp, of)
    y = moe.combine(plan, yp, torch.empty(t, hidden, dtype=torch.bfloat16, device=dev), weights=weights)

    row_of = _check_sorted(plan, ids)
    v1, v2 = F.values(*(v.cpu().numpy() for v in b1)), F.values(*(v.cpu().numpy() for v in b2))
    xq = F.values(*F.quantize(_f64(x)))
    flat_gu, flat_yp = _f64(gu).reshape(-1, 2 * inner), _f64(yp).reshape(-1, hidden)
    want = np.zeros((t, hidden))
    for i, j in np.argwhere(row_of >= 0):
        e, r = ids[i, j], row_of[i, j]
        for got, w, v, c in ((flat_gu[r], v1[e], xq[i], hidden),
                             (flat_yp[r], v2[e], F.values(*F.quantize(M.swiglu(flat_gu[r])[None]))[0], inner)):
            ref, mag = w @ v, np.abs(w) @ np.abs(v)
            assert np.all(np.abs(got - ref) <= bf16_ulp(np.maximum(np.abs(got), np.abs(ref))) + element_bound(mag, c))
        want[i] += float(weights[i, j]) * flat_yp[r]
    err = 8 * 2.0 ** -24 * M.combine_mag(flat_yp, row_of, _f64(weights))
    assert np.all(np.abs(_f64(y) - want) <= bf16_ulp(np.abs(want) + err) / 2 + err)


@pytest.mark.parametrize("layout", ["masked", "nopad", "contiguous"])
def test_a_captured_block(dev, layout):
    """Quantiser, dispatch, products, activation, combine and an expert layer over the same
    weights in one graph, replayed between eager calls with other tokens, ids and weights: each
    replay gives the eager calls' bits."""
    _say(f"a captured block in FP4, {layout}")
    t, k, g, hidden, inner = 20, 3, 5, 256, 384
    plan, _, ids = _moved(layout, t, k, g, hidden, {"masked": t}.get(layout), dev)
    master = _randn(g, hidden, inner, seed=5, scale=0.06, dtype=torch.float32)
    x = _randn(t, hidden, seed=3)
    weights = torch.rand(t, k, device=dev)

    def operand(*shape):
        *lead, m, c = shape
        return (torch.zeros(*lead, m, c // 2, dtype=torch.uint8, device=dev),
                torch.zeros(*lead, c // 128, dg.get_tma_aligned_size(m, 4), dtype=torch.int32, device=dev))

    b1 = dg.quantize_fp4(_randn(g, 2 * inner, hidden, seed=4, scale=0.06), *operand(g, 2 * inner, hidden))
    b2 = operand(g, hidden, inner)
    gemm = getattr(dg, f"m_grouped_fp4_gemm_nt_{layout}")
    lead = plan.rows_shape[:-1]
    gu, yp = (torch.zeros(*lead, n, dtype=torch.bfloat16, device=dev) for n in (2 * inner, hidden))
    q1, q2 = operand(*lead, hidden), operand(*lead, inner)
    y, z = (torch.zeros(t, hidden, dtype=torch.bfloat16, device=dev) for _ in range(2))
    back = torch.zeros(g, hidden, inner, dtype=torch.bfloat16, device=dev)
    of = plan.grouped_layout if layout == "contiguous" else plan.group_rows
    ws = moe.experts_workspace(t, k, g, inner, dev)

    def block():
        dg.quantize_fp4(master, *b2)
        moe.dispatch_fp4(plan, x, *q1, topk_ids=ids)
        gemm(*q1, *b1, gu, of)
        moe.swiglu_fp4(gu, *q2, rows=of, layout=layout)
        gemm(*q2, *b2, yp, of)
        moe.combine(plan, yp, y, weights=weights)
        moe.experts(x, ids, weights, *b1, *b2, z, ws)
        dg.dequantize_fp4(*b2, back)

    block()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block()
    for seed in range(4):
        x.copy_(_randn(t, hidden, seed=70 + seed))
        ids.copy_(torch.from_numpy(np.random.default_rng(seed).integers(-1, g, (t, k)).astype(np.int32)))
        master.mul_(-1.25)
        weights.uniform_()
        block()
        want = [v.clone() for v in (y, z, back)]
        for v in (y, z, back, gu, yp, ws, *b2):
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for got, ref in zip((y, z, back), want):
            assert torch.equal(got.view(torch.int16), ref.view(torch.int16))
        assert y.abs().sum() > 0 and z.abs().sum() > 0
