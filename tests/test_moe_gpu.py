"""GPU parity of the steps around the GEMMs against their float64 definitions
(oracle/moe_oracle.py), through the Python entry points.

Rows, counts, copies and FP8 codes of BF16 inputs are compared bit for bit.
Elsewhere, with u = 2^-24 and `mag` the sum of the magnitudes of the terms a
value is made of, a float32 result is within E = (D + c) u mag of the exact
one, where D bounds the additions that any one term passes through: a thread
adds at most H/64 terms of a row of H (a wave or more shares it), and a tree
over lanes and waves follows, so D = H/64 + 64; c counts the roundings around
the sum. A BF16 result adds the half ulp of its one rounding.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

from moe_grouped_gemm_amd import dg, moe, synth
from oracle import dg_oracle as O
from oracle import moe_oracle as M
from parity import bf16_ulp, element_bound

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SENTINEL = -1                     # 0xFFFF / 0xFF: a NaN in BF16 and E4M3


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()
    return torch.device("cuda:0")


def _say(msg):
    print(msg, flush=True)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(*shape, seed, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=_gen(seed), device="cuda") * scale).to(dtype)


def _f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _bits(t):
    width = {2: torch.int16, 1: torch.uint8, 4: torch.int32}[t.element_size()]
    return t.detach().view(width).cpu().numpy()


def _unwritten(shape, dtype=torch.bfloat16):
    if dtype is torch.float8_e4m3fn:
        return torch.full(shape, 0xFF, dtype=torch.uint8, device="cuda").view(dtype)
    if dtype is torch.float32:
        return torch.full(shape, -7.0, dtype=dtype, device="cuda")
    return torch.full(shape, SENTINEL, dtype=torch.int16, device="cuda").view(dtype)


def _depth(hidden):
    return hidden / 64 + 64


def check_bf16(got, ref, err, what=""):
    d = _f64(got)
    assert d.shape == ref.shape, (what, d.shape, ref.shape)
    assert np.all(np.isfinite(d)), f"{what}: non-finite"
    bound = bf16_ulp(np.maximum(np.abs(d), np.abs(ref) + err)) / 2 + err
    bad = np.abs(d - ref) > bound
    assert not bad.any(), f"{what}: {bad.sum()} beyond the bound, first {np.argwhere(bad)[:3].tolist()}"


def check_f32(got, ref, err, what=""):
    d = _f64(got)
    assert d.shape == ref.shape, (what, d.shape, ref.shape)
    bad = ~(np.abs(d - ref) <= err + 2.0 ** -149)
    assert not bad.any(), f"{what}: {bad.sum()} beyond the bound, first {np.argwhere(bad)[:3].tolist()}"


# ---------------------------------------------------------------------------
# Sorting
# ---------------------------------------------------------------------------

def _ids(t, k, g, seed, drop=0.1):
    r = np.random.default_rng(seed)
    ids = r.integers(0, g, (t, k))
    ids[r.random((t, k)) < drop] = -1
    return ids.astype(np.int32)


def _make_plan(t, k, g, layout, rows, hidden=256, dev="cuda"):
    if rows is None:
        rows = {"nopad": t * k, "contiguous": moe.contiguous_rows(t * k, g), "masked": max(1, t)}[layout]
    return moe.Plan(t, k, g, layout, rows, hidden, dev)


def _check_sorted(plan, ids, what=""):
    t = ids.shape[0]
    row_of, kept, layout = M.sort(ids, plan.num_groups, plan.layout, plan.rows)
    np.testing.assert_array_equal(plan.row_of[:t].cpu().numpy(), row_of, what)
    np.testing.assert_array_equal(plan.group_rows.cpu().numpy(), kept, what)
    if layout is not None:
        np.testing.assert_array_equal(plan.grouped_layout.cpu().numpy(), layout, what)
    return row_of


SORTS = [
    # tokens, top_k, groups, rows (None: as many as can be needed)
    (1, 1, 1, None), (1, 8, 16, None), (5, 8, 16, None), (64, 4, 8, None), (259, 8, 16, None), (1023, 1, 3, None),
    (700, 7, 129, None), (1025, 8, 64, None), (3001, 5, 33, None), (8192, 8, 32, None), (20000, 3, 257, None),
    (300, 2, 4, 128), (2500, 4, 8, 1280), (40, 32, 2, None), (512, 32, 40, None), (2048, 8, 8, None), (2049, 8, 8, None),
]


@pytest.mark.parametrize("layout", ["contiguous", "nopad", "masked"])
@pytest.mark.parametrize("t,k,g,rows", SORTS)
def test_sort(dev, t, k, g, rows, layout):
    _say(f"sort {layout} {t}x{k} over {g}, rows {rows}")
    plan = _make_plan(t, k, g, layout, rows)
    ids = _ids(t, k, g, t + k)
    moe.sort(plan, torch.from_numpy(ids).to(dev))
    _check_sorted(plan, ids)


@pytest.mark.parametrize("layout,g", [("masked", 4096), ("contiguous", 4096), ("nopad", 2048)])
@pytest.mark.parametrize("t", [3, 900, 5000])
def test_sort_maximum_groups(dev, layout, g, t):
    _say(f"sort {layout} {g} groups, {t} tokens")
    plan = _make_plan(t, 4, g, layout, 16 if layout == "masked" else None)
    ids = _ids(t, 4, g, g)
    moe.sort(plan, torch.from_numpy(ids).to(dev))
    _check_sorted(plan, ids)


@pytest.mark.parametrize("t", [200, 4000])
@pytest.mark.parametrize("layout", ["contiguous", "nopad", "masked"])
def test_sort_extreme_ids(dev, layout, t):
    """One group takes all; all dropped; ids at the ends of int32."""
    _say(f"sort extreme ids {layout} {t}")
    lo, hi = np.iinfo(np.int32).min, np.iinfo(np.int32).max
    plan = _make_plan(t, 2, 9, layout, None)
    ids = np.full((t, 2), 8, np.int32)
    for ids in (ids, np.full_like(ids, -1), np.where(np.arange(2 * t).reshape(t, 2) % 3 == 0, lo, hi).astype(np.int32),
                np.where(np.arange(2 * t).reshape(t, 2) % 3 == 0, 9, 0).astype(np.int32)):
        moe.sort(plan, torch.from_numpy(ids).to(dev))
        _check_sorted(plan, ids)


def test_empty_plan(dev):
    _say("a plan for no tokens")
    for layout, rows in (("nopad", 0), ("contiguous", 0), ("masked", 4)):
        plan = moe.Plan(0, 2, 4, layout, rows, 128, dev)
        moe.sort(plan, torch.empty(0, 2, dtype=torch.int32, device=dev))
        assert plan.group_rows.tolist() == [0, 0, 0, 0]
        none = torch.empty(0, 128, dtype=torch.bfloat16, device=dev)
        xp = torch.zeros(plan.rows_shape, dtype=torch.bfloat16, device=dev)
        moe.dispatch(plan, none, xp, topk_ids=torch.empty(0, 2, dtype=torch.int32, device=dev))
        moe.combine(plan, xp, none)


def test_plan_serves_fewer_tokens_and_none(dev):
    _say("plan with fewer tokens")
    for layout in ("contiguous", "nopad", "masked"):
        plan = _make_plan(600, 4, 8, layout, None)
        for t in (600, 3, 0, 257):
            ids = _ids(t, 4, 8, t)
            x = _randn(t, 256, seed=t)
            xp = _unwritten(plan.rows_shape)
            if t % 2:
                moe.sort(plan, torch.from_numpy(ids).to(dev))
                moe.dispatch(plan, x, xp)
            else:
                moe.dispatch(plan, x, xp, topk_ids=torch.from_numpy(ids).to(dev))
            row_of = _check_sorted(plan, ids, f"{layout} {t}")
            want = M.dispatch(_bits(x), row_of, np.full((xp.numel() // 256, 256), SENTINEL, np.int16))
            np.testing.assert_array_equal(_bits(xp).reshape(want.shape), want)
            y = _unwritten((t, 256))
            moe.combine(plan, xp, y)
            if t:
                check_bf16(y, M.combine(np.nan_to_num(_f64(xp)).reshape(-1, 256), row_of),
                           8 * U * M.combine_mag(np.nan_to_num(_f64(xp)).reshape(-1, 256), row_of), f"{layout} {t}")


@pytest.mark.parametrize("layout", ["contiguous", "nopad", "masked"])
def test_sort_extreme_ids_many_slots(dev, layout):
    test_sort_extreme_ids(dev, layout, 10000)


@pytest.mark.parametrize("layout", ["contiguous", "nopad", "masked"])
def test_plan_across_the_limit_of_one_launch(dev, layout):
    """One plan with more and fewer slots in turn than one launch takes, by sort and
    by dispatch: nothing of a call is left for the next."""
    _say(f"a plan across the limit of one launch, {layout}")
    k, g = 4, 8
    plan = _make_plan(6000, k, g, layout, None)
    for t in (6000, 5, 4097, 4096, 0, 6000, 257, 4099):
        ids = _ids(t, k, g, t)
        x, xp = _randn(t, 256, seed=t), _unwritten(plan.rows_shape)
        if t % 2:
            moe.sort(plan, torch.from_numpy(ids).to(dev))
            moe.dispatch(plan, x, xp)
        else:
            moe.dispatch(plan, x, xp, topk_ids=torch.from_numpy(ids).to(dev))
        row_of = _check_sorted(plan, ids, f"{t}")
        want = M.dispatch(_bits(x), row_of, np.full((xp.numel() // 256, 256), SENTINEL, np.int16))
        np.testing.assert_array_equal(_bits(xp).reshape(want.shape), want)


# ---------------------------------------------------------------------------
# Dispatch
# ---------------------------------------------------------------------------

MOVES = [
    # layout, tokens, top_k, groups, hidden, rows
    ("masked", 1, 1, 1, 128, 4), ("masked", 5, 8, 16, 7168, 256), ("masked", 64, 6, 8, 640, 9),
    ("nopad", 3, 2, 4, 128, None), ("nopad", 130, 4, 8, 1920, None), ("nopad", 601, 8, 32, 384, 3000),
    ("contiguous", 17, 3, 5, 256, None), ("contiguous", 333, 4, 8, 2048, 1024), ("contiguous", 1500, 3, 40, 128, None),
    ("nopad", 2100, 4, 16, 512, None), ("masked", 2048, 8, 16, 256, 1000), ("contiguous", 2049, 8, 16, 128, None),
    # more than 16 slots a token, with blocks that leave part of a wave idle
    ("masked", 9, 32, 40, 128, 16), ("contiguous", 30, 17, 64, 4224, None), ("nopad", 200, 24, 32, 640, None),
]


def _moved(layout, t, k, g, hidden, rows, dev, drop=0.15):
    plan = _make_plan(t, k, g, layout, rows, hidden)
    ids = _ids(t, k, g, t + g, drop)
    return plan, ids, torch.from_numpy(ids).to(dev)


@pytest.mark.parametrize("with_sort", [True, False])
@pytest.mark.parametrize("case", MOVES)
def test_dispatch_bf16(dev, case, with_sort):
    _say(f"dispatch {case} sort={with_sort}")
    layout, t, k, g, hidden, rows = case
    plan, ids, ids_d = _moved(*case, dev)
    x = _randn(t, hidden, seed=1)
    xp = _unwritten(plan.rows_shape)
    if not with_sort:
        moe.sort(plan, ids_d)
    moe.dispatch(plan, x, xp, topk_ids=ids_d if with_sort else None)
    row_of = _check_sorted(plan, ids)
    want = M.dispatch(_bits(x), row_of, np.full((xp.numel() // hidden, hidden), SENTINEL, np.int16))
    np.testing.assert_array_equal(_bits(xp).reshape(want.shape), want)


def _special(x):
    """NaN, infinities, zeros, subnormals and ties in some blocks of x."""
    n = x.numel() // 128
    b = x.view(n, 128)
    b[0] = 0.0
    b[n // 2, 5] = float("nan")
    b[n // 3, 7] = float("inf")
    b[n // 4, 9] = -float("inf")
    b[n // 5] *= 1e-38
    b[n // 6, 0] = 7.0 * 2.0 ** 6                  # scale 1: exact ties of E4M3
    b[n // 6, 1:4] = torch.tensor([17.0, -19.0, 0.0009765625])
    b[n // 7] = 51.0 / 4                           # 51 / 3 = 17, a tie, under a scale of 3 * 2^k
    b[n // 7, 0] = 21.0 * 2.0 ** 6
    return x


def _check_codes(q, sfa, x32, row_of, ue8m0, plan):
    hidden, rows = plan.hidden, plan.rows
    vals, scales = M.quantize(x32, ue8m0)
    total = q.numel() // hidden
    held = np.zeros(total, bool)
    held[row_of[row_of >= 0]] = True
    want_q = M.dispatch(vals, row_of, np.zeros((total, hidden)))
    np.testing.assert_array_equal(q.float().cpu().numpy().reshape(total, hidden)[held], want_q[held])
    assert (_bits(q).reshape(total, hidden)[~held] == 0xFF).all()
    want_s = np.full((total // rows, plan.scale_shape[-1], hidden // 128), -7.0)
    flat = M.dispatch(scales, row_of, np.full((total, hidden // 128), -7.0))
    want_s[:, :rows] = flat.reshape(-1, rows, hidden // 128)
    np.testing.assert_array_equal(_f64(sfa).reshape(-1, hidden // 128, plan.scale_shape[-1]), want_s.transpose(0, 2, 1))


@pytest.mark.parametrize("special", [False, True])
@pytest.mark.parametrize("ue8m0", [False, True])
@pytest.mark.parametrize("case", MOVES)
def test_dispatch_fp8(dev, case, ue8m0, special):
    _say(f"dispatch_fp8 {case} ue8m0={ue8m0} special={special}")
    layout, t, k, g, hidden, rows = case
    plan, ids, ids_d = _moved(*case, dev)
    x = _randn(t, hidden, seed=2, scale=3.0)
    if special:
        x = _special(x)
    q, sfa = _unwritten(plan.rows_shape, torch.float8_e4m3fn), _unwritten(plan.scale_shape, torch.float32)
    moe.dispatch_fp8(plan, x, q, sfa, topk_ids=ids_d, ue8m0=ue8m0)
    _check_codes(q, sfa, _f64(x).astype(np.float32), _check_sorted(plan, ids), ue8m0, plan)


# more slots than one launch ever sorts and moves (16384)
LARGE_MOVES = [
    ("masked", 2500, 8, 16, 384, 1001), ("masked", 1100, 17, 64, 1152, 301), ("nopad", 900, 24, 40, 640, 15000),
    ("nopad", 2060, 8, 256, 1920, None), ("contiguous", 700, 32, 33, 256, None), ("contiguous", 4100, 5, 9, 512, 12800),
]


@pytest.mark.parametrize("special", [False, True])
@pytest.mark.parametrize("ue8m0", [False, True])
@pytest.mark.parametrize("with_sort", [True, False])
@pytest.mark.parametrize("case", LARGE_MOVES)
def test_dispatch_fp8_many_slots(dev, case, with_sort, ue8m0, special):
    _say(f"dispatch_fp8 {case} sort={with_sort} ue8m0={ue8m0} special={special}")
    _dispatch_fp8(dev, case, with_sort, ue8m0, special)


@pytest.mark.parametrize("ue8m0", [False, True])
@pytest.mark.parametrize("case", [("masked", 1500, 8, 16, 4224, 901), ("contiguous", 600, 25, 40, 4096, None),
                                  ("nopad", 4000, 4, 7, 4096, 14000)])
def test_dispatch_fp8_long_rows_in_one_launch(dev, case, ue8m0):
    """As many slots as one launch takes with long rows; several tokens a workgroup."""
    _say(f"dispatch_fp8 {case} ue8m0={ue8m0}")
    _dispatch_fp8(dev, case, True, ue8m0, True)


@pytest.mark.parametrize("special", [False, True])
@pytest.mark.parametrize("ue8m0", [False, True])
@pytest.mark.parametrize("case", MOVES)
def test_dispatch_fp8_after_sort(dev, case, ue8m0, special):
    _say(f"dispatch_fp8 {case} after sort, ue8m0={ue8m0} special={special}")
    _dispatch_fp8(dev, case, False, ue8m0, special)


def _dispatch_fp8(dev, case, with_sort, ue8m0, special):
    layout, t, k, g, hidden, rows = case
    plan, ids, ids_d = _moved(*case, dev)
    x = _randn(t, hidden, seed=2, scale=3.0)
    if special:
        x = _special(x)
    q, sfa = _unwritten(plan.rows_shape, torch.float8_e4m3fn), _unwritten(plan.scale_shape, torch.float32)
    if not with_sort:
        moe.sort(plan, ids_d)
    moe.dispatch_fp8(plan, x, q, sfa, topk_ids=ids_d if with_sort else None, ue8m0=ue8m0)
    _check_codes(q, sfa, _f64(x).astype(np.float32), _check_sorted(plan, ids), ue8m0, plan)


@pytest.mark.parametrize("with_sort", [True, False])
@pytest.mark.parametrize("case", LARGE_MOVES)
def test_dispatch_bf16_many_slots(dev, case, with_sort):
    test_dispatch_bf16(dev, case, with_sort)


@pytest.mark.parametrize("case", LARGE_MOVES)
def test_combine_and_gradient_many_slots(dev, case):
    test_combine(dev, case, True)
    test_combine_bwd(dev, case, True)


def test_dispatch_fp8_feeds_the_gemm(dev):
    """The same operand as the rows quantised one by one: the GEMM's output
    equals, bit for bit, the one on operands laid out by hand."""
    _say("dispatch_fp8 into the masked GEMM")
    t, k, g, hidden, n, max_m = 50, 4, 6, 512, 256, 64
    plan, ids, ids_d = _moved("masked", t, k, g, hidden, max_m, dev)
    x = _randn(t, hidden, seed=3)
    q = torch.zeros(plan.rows_shape, dtype=torch.float8_e4m3fn, device=dev)
    sfa = torch.zeros(plan.scale_shape, device=dev)
    moe.dispatch_fp8(plan, x, q, sfa, topk_ids=ids_d)
    b = _randn(g, n, hidden, seed=4).to(torch.float8_e4m3fn)
    sfb = torch.rand(g, n // 128, hidden // 128, generator=_gen(5), device=dev) + 0.5
    d = _unwritten((g, max_m, n))
    dg.m_grouped_fp8_gemm_nt_masked(q, sfa, b, sfb, d, plan.group_rows)
    vals, scales = M.quantize(_f64(x).astype(np.float32), False)
    deq = vals * np.repeat(scales.astype(np.float64), 128, 1)
    w = b.float().cpu().numpy() * np.repeat(np.repeat(_f64(sfb), 128, 1), 128, 2)
    out = _f64(d).reshape(-1, n)
    row_of = M.sort(ids, g, "masked", max_m)[0]
    for (i, j) in np.argwhere(row_of >= 0)[::7]:
        ref = w[ids[i, j]] @ deq[i]
        mag = np.abs(w[ids[i, j]]) @ np.abs(deq[i])
        assert np.all(np.abs(out[row_of[i, j]] - ref) <= bf16_ulp(np.abs(ref) + mag * 2 ** -14) + mag * 2 ** -14)


def _masked_gemm_inputs(layout, t, k, g, hidden, max_m, dev, ue8m0):
    plan, ids, ids_d = _moved(layout, t, k, g, hidden, max_m, dev)
    x = _randn(t, hidden, seed=3)
    x *= torch.linspace(0.3, 3.0, t, device=dev)[:, None].to(torch.bfloat16)     # scales of many mantissas
    q = torch.zeros(plan.rows_shape, dtype=torch.float8_e4m3fn, device=dev)
    sfa = torch.zeros(plan.scale_shape, device=dev)
    moe.dispatch_fp8(plan, x, q, sfa, topk_ids=ids_d, ue8m0=ue8m0)
    vals, scales = M.quantize(_f64(x).astype(np.float32), ue8m0)
    return plan, ids, q, sfa, vals * np.repeat(scales.astype(np.float64), 128, 1)


def _check_product(d, ids, deq, w, max_m, g, k):
    """Rows of a masked product against the tokens' dequantised values times the
    groups' weights w [G, N, K]: the GEMM's own bound."""
    out = _f64(d).reshape(-1, w.shape[1])
    row_of = M.sort(ids, g, "masked", max_m)[0]
    for i, j in np.argwhere(row_of >= 0)[::5]:
        ref, mag = w[ids[i, j]] @ deq[i], np.abs(w[ids[i, j]]) @ np.abs(deq[i])
        got = out[row_of[i, j]]
        assert np.all(np.abs(got - ref) <= bf16_ulp(np.maximum(np.abs(got), np.abs(ref))) + element_bound(mag, k))


def test_dispatch_fp8_feeds_the_ue8m0_gemm(dev):
    """Power-of-two scales into the calls that read a scale's exponent only."""
    _say("dispatch_fp8 into the masked UE8M0 GEMM")
    t, k, g, hidden, n, max_m = 50, 4, 6, 512, 256, 64
    plan, ids, q, sfa, deq = _masked_gemm_inputs("masked", t, k, g, hidden, max_m, dev, True)
    b = _randn(g, n, hidden, seed=4).to(torch.float8_e4m3fn)
    sfb = 2.0 ** torch.randint(-3, 4, (g, n // 128, hidden // 128), generator=_gen(5), device=dev).float()
    d = _unwritten((g, max_m, n))
    dg.m_grouped_fp8_gemm_nt_masked(q, sfa, b, sfb, d, plan.group_rows, ue8m0=True)
    w = b.float().cpu().numpy().astype(np.float64) * np.repeat(np.repeat(_f64(sfb), 128, 1), 128, 2)
    _check_product(d, ids, deq, w, max_m, g, hidden)


def test_dispatch_and_activation_feed_the_w4a8_gemm(dev):
    """ue8m0=True operands of dispatch_fp8 and of swiglu_fp8 in the FP8 x FP4 product,
    which reads every scale's exponent only."""
    _say("dispatch_fp8 and swiglu_fp8 into the masked W4A8 GEMM")
    t, k, g, hidden, n, max_m = 50, 4, 6, 512, 512, 64
    plan, ids, q, sfa, deq = _masked_gemm_inputs("masked", t, k, g, hidden, max_m, dev, True)
    parts = [synth.quantize_rhs_e2m1(torch.randn(n, hidden, generator=_gen(6 + e), device=dev)) for e in range(g)]
    b, sfb = torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])
    d = _unwritten((g, max_m, n))
    dg.m_grouped_fp8_fp4_gemm_nt_masked(q, sfa, b, sfb, d, plan.group_rows)
    w = np.stack([O.dequant_rhs_e2m1(e.cpu().numpy(), f.cpu().numpy()) for e, f in zip(b, sfb)])
    _check_product(d, ids, deq, w, max_m, g, hidden)
    # the product's rows through the activation into a second one, of the first n / 2 inputs
    inner = n // 2
    aq, asf = _unwritten((g, max_m, inner), torch.float8_e4m3fn), _unwritten((g, inner // 128, max_m), torch.float32)
    moe.swiglu_fp8(d, aq, asf, rows=plan.group_rows, layout="masked", ue8m0=True)
    parts = [synth.quantize_rhs_e2m1(torch.randn(hidden, inner, generator=_gen(20 + e), device=dev)) for e in range(g)]
    b2, sfb2 = torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])
    yp = _unwritten((g, max_m, hidden))
    dg.m_grouped_fp8_fp4_gemm_nt_masked(aq, asf, b2, sfb2, yp, plan.group_rows)
    counts = plan.group_rows.tolist()
    gu, out = _f64(d), _f64(yp)
    for e in range(g):
        w2 = O.dequant_rhs_e2m1(b2[e].cpu().numpy(), sfb2[e].cpu().numpy())
        act = M.swiglu(gu[e, :counts[e]])
        ref, mag = act @ w2.T, np.abs(act) @ np.abs(w2).T
        # each code is within 2^-4 of its value, or 2^-10 of the block's scale, which power-of-two
        # rounding takes up to twice amax / 448; a scale taken for another one would double or halve a block
        top = np.repeat(np.abs(act).reshape(counts[e], -1, 128).max(-1), 128, -1)
        off = (np.abs(act) * 2.0 ** -4 + top * 2.0 ** -9 / 448) @ np.abs(w2).T
        bound = off * 1.01 + np.abs(ref) * 2.0 ** -8 + element_bound(mag, inner) * 2
        assert np.all(np.abs(out[e, :counts[e]] - ref) <= bound)


@pytest.mark.parametrize("call,t,k,hidden,passes", [
    ("sort", 4096, 1, 128, False), ("sort", 4100, 1, 128, True), ("sort", 2048, 8, 7168, True),
    ("dispatch", 1024, 8, 128, False), ("dispatch", 1025, 8, 128, True), ("dispatch", 4096, 2, 7168, False),
    ("dispatch", 4097, 1, 7168, True), ("dispatch", 2048, 8, 4096, False), ("dispatch", 2049, 8, 4096, True),
])
def test_few_slots_take_one_launch(dev, call, t, k, hidden, passes):
    """Which of the two ways a call takes, by whether its workspace is written: only
    the passes over chunks leave their counts there."""
    _say(f"{call} of {t}x{k}, rows of {hidden}")
    plan = _make_plan(t, k, 64, "nopad", None, hidden)
    plan.workspace.fill_(0xAB)
    ids = _ids(t, k, 64, t)
    if call == "sort":
        moe.sort(plan, torch.from_numpy(ids).to(dev))
    else:
        x, xp = _randn(t, hidden, seed=t), _unwritten(plan.rows_shape)
        moe.dispatch(plan, x, xp, topk_ids=torch.from_numpy(ids).to(dev))
    row_of = _check_sorted(plan, ids)
    if call == "dispatch":
        for i, j in np.argwhere(row_of >= 0)[::997]:
            assert torch.equal(xp[row_of[i, j]], x[i])
    assert passes != bool((plan.workspace == 0xAB).all())


# ---------------------------------------------------------------------------
# Combine
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("case", MOVES)
def test_combine(dev, case, weighted):
    _say(f"combine {case} weighted={weighted}")
    layout, t, k, g, hidden, rows = case
    plan, ids, ids_d = _moved(*case, dev, drop=0.4)
    moe.sort(plan, ids_d)
    row_of = _check_sorted(plan, ids)
    yp = _randn(*plan.rows_shape, seed=5)
    used = np.zeros(yp.numel() // hidden, bool)
    used[row_of[row_of >= 0]] = True
    yp.view(-1, hidden)[torch.from_numpy(~used).to(dev)] = float("nan")      # rows no slot names
    w = None
    if weighted:
        w = torch.softmax(_randn(t, k, seed=6, dtype=torch.float32), 1)
        w[torch.from_numpy(row_of < 0).to(dev)] = float("nan")               # weights of dropped slots
    y = _unwritten((t, hidden))
    moe.combine(plan, yp, y, weights=w)
    src = np.nan_to_num(_f64(yp)).reshape(-1, hidden)
    wn = None if w is None else np.nan_to_num(_f64(w))
    check_bf16(y, M.combine(src, row_of, wn), (k + 2) * U * M.combine_mag(src, row_of, wn), str(case))
    empty = (row_of < 0).all(1)
    assert not _bits(y)[empty].any()                                         # zeros, not -0 or NaN


@pytest.mark.parametrize("with_dw", [True, False])
@pytest.mark.parametrize("case", MOVES)
def test_combine_bwd(dev, case, with_dw):
    _say(f"combine_bwd {case} dw={with_dw}")
    layout, t, k, g, hidden, rows = case
    plan, ids, ids_d = _moved(*case, dev, drop=0.3)
    moe.sort(plan, ids_d)
    row_of = _check_sorted(plan, ids)
    yp, dy = _randn(*plan.rows_shape, seed=7), _randn(t, hidden, seed=8)
    w = _randn(t, k, seed=9, dtype=torch.float32)
    dyp = _unwritten(plan.rows_shape)
    dw = _unwritten((t, k), torch.float32) if with_dw else None
    moe.combine_bwd(plan, dy, yp if with_dw else None, w, dyp, dw)
    src, d, wn = _f64(yp).reshape(-1, hidden), _f64(dy), _f64(w)
    want, want_dw = M.combine_bwd(d, src, row_of, wn, np.full_like(src, np.nan))
    got = dyp.view(-1, hidden)
    held = ~np.isnan(want[:, 0])
    assert (_bits(got)[~held] == SENTINEL).all()
    check_bf16(got[torch.from_numpy(held).to(dev)], want[held], 2 * U * np.abs(want[held]), str(case))
    if with_dw:
        mag = M.combine_bwd(np.abs(d), np.abs(src), row_of, wn, np.zeros_like(src))[1]
        check_f32(dw, want_dw, (_depth(hidden) + 2) * U * mag, str(case))


@pytest.mark.parametrize("t,hidden", [(300, 1024), (65, 4224)])
def test_combine_bwd_blocks_without_rows(dev, t, hidden):
    """Tokens whose slots have rows only in some stretches of the top_k."""
    _say(f"combine_bwd {t} tokens of {hidden} with stretches of dropped slots")
    k, g = 32, 40
    plan = _make_plan(t, k, g, "nopad", None, hidden)
    ids = _ids(t, k, g, t, 0.1)
    for i in range(t):
        for b in range(4):
            if (i * 7 + i // 16) >> b & 1:
                ids[i, 8 * b:8 * b + 8] = -1
    moe.sort(plan, torch.from_numpy(ids).to(dev))
    row_of = _check_sorted(plan, ids)
    yp, dy = _randn(*plan.rows_shape, seed=17), _randn(t, hidden, seed=18)
    w = _randn(t, k, seed=19, dtype=torch.float32)
    dyp, dw = _unwritten(plan.rows_shape), _unwritten((t, k), torch.float32)
    moe.combine_bwd(plan, dy, yp, w, dyp, dw)
    src, d, wn = _f64(yp).reshape(-1, hidden), _f64(dy), _f64(w)
    want, want_dw = M.combine_bwd(d, src, row_of, wn, np.full_like(src, np.nan))
    held = ~np.isnan(want[:, 0])
    got = dyp.view(-1, hidden)
    assert (_bits(got)[~held] == SENTINEL).all()
    check_bf16(got[torch.from_numpy(held).to(dev)], want[held], 2 * U * np.abs(want[held]))
    mag = M.combine_bwd(np.abs(d), np.abs(src), row_of, wn, np.zeros_like(src))[1]
    check_f32(dw, want_dw, (_depth(hidden) + 2) * U * mag)
    assert not _f64(dw)[row_of < 0].any()


@pytest.mark.parametrize("layout", ["contiguous", "nopad", "masked"])
@pytest.mark.parametrize("t,k,g", [(1025, 1, 1), (3000, 5, 5), (8192, 2, 2), (700, 6, 63), (1100, 4, 64)])
def test_dispatch_few_groups(dev, layout, t, k, g):
    """Many slots over few groups, with most of them in one group."""
    _say(f"dispatch {layout} {t}x{k} over {g}")
    plan = _make_plan(t, k, g, layout, None, 128)
    ids = _ids(t, k, g, t + g)
    if g >= k + 1:
        ids[: t // 2, 0] = np.where((ids[: t // 2, 1:] == g - 1).any(1), -1, g - 1)
    x, xp = _randn(t, 128, seed=21), _unwritten(plan.rows_shape)
    moe.dispatch(plan, x, xp, topk_ids=torch.from_numpy(ids).to(dev))
    row_of = _check_sorted(plan, ids)
    want = M.dispatch(_bits(x), row_of, np.full((xp.numel() // 128, 128), SENTINEL, np.int16))
    np.testing.assert_array_equal(_bits(xp).reshape(want.shape), want)


# ---------------------------------------------------------------------------
# Norms
# ---------------------------------------------------------------------------

NORM_SIZES = [(1, 8), (3, 64), (5, 520), (2, 1000), (7, 7168), (33, 2048), (300, 384), (2, 8192), (3, 8200), (2, 12296),
              (300, 16384), (600, 1024)]
GATES = ["none", "channel", "token", "full"]


def _norm_inputs(t, h, gate, seed=11):
    d = {"x": _randn(t, h, seed=seed, scale=2.0), "y": _randn(t, h, seed=seed + 1, scale=3.0),
         "post": 1.0 + _randn(h, seed=seed + 2, scale=0.2, dtype=torch.float32),
         "pre": 1.0 + _randn(h, seed=seed + 3, scale=0.2, dtype=torch.float32)}
    d["gate"] = {"none": lambda: None, "channel": lambda: _randn(h, seed=seed + 4, dtype=torch.float32),
                 "token": lambda: _randn(t, 1, seed=seed + 4, dtype=torch.float32),
                 "full": lambda: _randn(t, h, seed=seed + 4)}[gate]()
    return d


def _check_norm(got, d, y, post, pre, rs, eps, what):
    """got: (h, n, r1, r2) tensors or None."""
    x, gate = _f64(d["x"]), _f64(d["gate"]) if y is not None else None
    hidden = x.shape[1]
    h, n, r1, r2 = M.block_norm(x, y, post, gate, pre, rs, eps)
    rel = (_depth(hidden) + 8) * U                  # of a float32 rstd
    err_h = np.zeros_like(x)
    if y is not None:
        v = y if post is None else y * r1[:, None] * post
        err_h = (rel + 8 * U) * (np.abs(rs * x) + np.abs((1.0 if gate is None else gate) * v))
        check_bf16(got[0], h, err_h, what + " h")
        if got[2] is not None:
            check_f32(got[2], r1, rel * r1, what + " rstd_post")
    if pre is None:
        return
    moved = (np.abs(h) * err_h).sum(1) / np.maximum((h * h).sum(1), 1e-300) + rel   # relative, of rstd_pre
    if got[3] is not None:
        check_f32(got[3], r2, moved * r2, what + " rstd_pre")
    check_bf16(got[1], n, np.abs(r2[:, None] * pre) * err_h + np.abs(n) * (moved[:, None] + 4 * U), what + " n")


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("t,h", NORM_SIZES)
def test_block_norm(dev, t, h, gate):
    _say(f"block_norm {t}x{h} gate={gate}")
    d = _norm_inputs(t, h, gate)
    out_h, out_n = _unwritten((t, h)), _unwritten((t, h))
    r1, r2 = _unwritten((t,), torch.float32), _unwritten((t,), torch.float32)
    moe.block_norm(d["x"], d["y"], d["post"], d["gate"], d["pre"], out_h, out_n, r1, r2, residual_scale=0.5, eps=1e-5)
    _check_norm((out_h, out_n, r1, r2), d, _f64(d["y"]), _f64(d["post"]), _f64(d["pre"]), 0.5, 1e-5, f"{t}x{h} {gate}")


@pytest.mark.parametrize("part", ["no_post", "no_pre", "only_pre", "no_rstd", "in_place"])
@pytest.mark.parametrize("t,h", [(4, 64), (37, 7168), (3, 8192 + 64)])
def test_block_norm_parts(dev, t, h, part):
    _say(f"block_norm {part} {t}x{h}")
    d = _norm_inputs(t, h, "none" if part == "only_pre" else "channel")
    y, post, pre, rs = d["y"], d["post"], d["pre"], 0.25
    out_h, out_n = _unwritten((t, h)), _unwritten((t, h))
    r1, r2 = _unwritten((t,), torch.float32), _unwritten((t,), torch.float32)
    if part == "no_post":
        post, r1 = None, None
    elif part == "no_pre":
        pre, out_n, r2 = None, None, None
    elif part == "only_pre":
        y, post, out_h, r1, rs = None, None, None, None, 1.0
    elif part == "no_rstd":
        r1 = r2 = None
    ref = {k: None if v is None else v.clone() for k, v in d.items()}
    y64, post64, pre64 = _f64(y), _f64(post), _f64(pre)
    if part == "in_place":
        out_h, out_n = d["x"], d["y"]
    moe.block_norm(d["x"], y, post, d["gate"], pre, out_h, out_n, r1, r2, residual_scale=rs, eps=1e-6)
    _check_norm((out_h, out_n, r1, r2), ref, y64, post64, pre64, rs, 1e-6, part)


def test_block_norm_zero_and_special_rows(dev):
    """A row of zeros normalises to zeros; NaN and infinity stay in their row."""
    _say("block_norm special rows")
    d = _norm_inputs(6, 512, "channel")
    d["y"][0] = 0
    d["x"][0] = 0
    d["y"][2, 17] = float("nan")
    d["x"][4, 3] = float("inf")
    h, n = _unwritten((6, 512)), _unwritten((6, 512))
    moe.block_norm(d["x"], d["y"], d["post"], d["gate"], d["pre"], h, n)
    assert not (_f64(h)[0].any() or _f64(n)[0].any())
    assert np.isnan(_f64(h)[2]).all() and np.isnan(_f64(n)[2]).all()
    assert np.isinf(_f64(h)[4, 3]) and np.isnan(_f64(n)[4, 3])
    assert np.isfinite(_f64(h)[[1, 3, 5]]).all() and np.isfinite(_f64(n)[[1, 3, 5]]).all()


@pytest.mark.parametrize("h", [8, 520, 7168, 8200])
@pytest.mark.parametrize("by", ["gate", "residual_scale"])
def test_block_norm_infinite_rows(dev, h, by):
    """A row that an infinite gate or factor makes infinite in every column has
    1 / sqrt(infinity) = 0 for its second rstd, whatever part of a wave its columns
    leave idle, and the other rows are not touched by it."""
    _say(f"block_norm infinite {by}, {h} columns")
    d = _norm_inputs(3, h, "token")
    for name in ("x", "y"):
        d[name][d[name] == 0] = 1.0
    rs = 0.5
    if by == "gate":
        d["gate"][1] = float("inf")
    else:
        d["x"][:] = d["x"].abs()
        rs = float("inf")
    out_h, out_n = _unwritten((3, h)), _unwritten((3, h))
    r1, r2 = _unwritten((3,), torch.float32), _unwritten((3,), torch.float32)
    moe.block_norm(d["x"], d["y"], d["post"], d["gate"], d["pre"], out_h, out_n, r1, r2, residual_scale=rs)
    rows = [1] if by == "gate" else [0, 1, 2]
    assert np.isinf(_f64(out_h)[rows]).all() and np.isnan(_f64(out_n)[rows]).all()
    assert np.isfinite(_f64(r1)).all() and not _f64(r2)[rows].any()
    if by == "gate":
        rest = {k: v[[0, 2]] if k in ("x", "y", "gate") else v for k, v in d.items()}
        _check_norm([v[[0, 2]] for v in (out_h, out_n, r1, r2)], rest, _f64(rest["y"]), _f64(d["post"]), _f64(d["pre"]),
                    rs, 1e-6, "rows beside it")


def _bwd(d, dh, dn, h, r1, r2, rs, parts=("dpost", "dgate", "dpre")):
    t, hid = (dh if dh is not None else dn).shape
    out = {"dx": _unwritten((t, hid)), "dy": None if d["y"] is None else _unwritten((t, hid))}
    out["dpost"] = torch.full((hid,), -7.0, device="cuda") if d["post"] is not None and "dpost" in parts else None
    out["dpre"] = torch.full((hid,), -7.0, device="cuda") if dn is not None and "dpre" in parts else None
    out["dgate"] = torch.full_like(d["gate"], -7.0) if d["gate"] is not None and "dgate" in parts else None
    ws = moe.block_norm_workspace(t, hid, "cuda")
    moe.block_norm_bwd(dh, dn, h, d["y"], d["post"], d["gate"], d["pre"], r1, r2, out["dx"], out["dy"], out["dpost"],
                       out["dgate"], out["dpre"], ws, residual_scale=rs)
    return out


def _check_bwd(out, d, dh, dn, h, r1, r2, rs, what):
    args = [_f64(v) for v in (dh, dn, h, d["y"], d["post"], d["gate"], d["pre"], r1, r2)]
    want, mag = M.block_norm_bwd(*args, rs), M.block_norm_bwd(*args, rs, mag=True)
    t, hid = _f64(out["dx"]).shape
    row = (2 * _depth(hid) + 32) * U
    for key, got in out.items():
        if got is None:
            continue
        # column sums add up to t rows; a token gate's one more row
        err = (row + ((t + 8) * U if want[key].shape != (t, hid) else 0) + _depth(hid) * U) * mag[key]
        (check_bf16 if got.dtype == torch.bfloat16 else check_f32)(got, want[key], err, f"{what} {key}")


def _rstds(d, h, eps=1e-5):
    r1 = torch.rsqrt(d["y"].float().square().mean(1) + eps)
    return r1, torch.rsqrt(h.float().square().mean(1) + eps)


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("t,h", NORM_SIZES)
def test_block_norm_bwd(dev, t, h, gate):
    _say(f"block_norm_bwd {t}x{h} gate={gate}")
    d = _norm_inputs(t, h, gate)
    res, dh, dn = _randn(t, h, seed=31, scale=2.0), _randn(t, h, seed=32), _randn(t, h, seed=33)
    r1, r2 = _rstds(d, res)
    _check_bwd(_bwd(d, dh, dn, res, r1, r2, 0.5), d, dh, dn, res, r1, r2, 0.5, f"{t}x{h} {gate}")


@pytest.mark.parametrize("part", ["no_dh", "no_dn", "no_post", "only_pre", "no_column_grads", "in_place"])
@pytest.mark.parametrize("t,h", [(4, 64), (270, 1920), (3, 8192 + 64)])
def test_block_norm_bwd_parts(dev, t, h, part):
    _say(f"block_norm_bwd {part} {t}x{h}")
    d = _norm_inputs(t, h, "none" if part == "only_pre" else "channel")
    res, dh, dn = _randn(t, h, seed=31, scale=2.0), _randn(t, h, seed=32), _randn(t, h, seed=33)
    r1, r2 = _rstds(d, res)
    rs, parts = 0.5, ("dpost", "dgate", "dpre")
    if part == "no_dh":
        dh = None
    elif part == "no_dn":
        dn, d["pre"], r2, res = None, None, None, None
    elif part == "no_post":
        d["post"], r1 = None, None
    elif part == "only_pre":
        d["y"], d["post"], r1, rs = None, None, None, 1.0
    elif part == "no_column_grads":
        parts = ()
    if part == "in_place":
        ws = moe.block_norm_workspace(t, h, dev)
        keep_h, keep_n = dh.clone(), dn.clone()
        out = {"dx": dh, "dy": dn, "dpost": torch.empty(h, device=dev), "dgate": torch.empty(h, device=dev),
               "dpre": torch.empty(h, device=dev)}
        moe.block_norm_bwd(dh, dn, res, d["y"], d["post"], d["gate"], d["pre"], r1, r2, dh, dn, out["dpost"],
                           out["dgate"], out["dpre"], ws, residual_scale=rs)
        dh, dn = keep_h, keep_n
    else:
        out = _bwd(d, dh, dn, res, r1, r2, rs, parts)
    _check_bwd(out, d, dh, dn, res, r1, r2, rs, part)


# Several rounds of rows a workgroup (256 workgroups, as many teams as fit them): one
# team of 9 and of 14 waves, 8 teams of 2, 16 teams of one wave, which has no barrier.
NORM_ROUNDS = [(600, 4104), (1100, 7168), (2100, 1024), (9000, 384)]


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("t,h", NORM_ROUNDS)
def test_block_norm_rounds(dev, t, h, gate):
    test_block_norm(dev, t, h, gate)


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("t,h", NORM_ROUNDS)
def test_block_norm_bwd_rounds(dev, t, h, gate):
    test_block_norm_bwd(dev, t, h, gate)


@pytest.mark.parametrize("part", ["no_pre", "no_post", "only_pre", "in_place"])
@pytest.mark.parametrize("t,h", [(1100, 4104), (9000, 384)])
def test_block_norm_parts_rounds(dev, t, h, part):
    test_block_norm_parts(dev, t, h, part)


@pytest.mark.parametrize("part", ["no_dh", "no_dn", "no_post", "only_pre", "in_place"])
@pytest.mark.parametrize("t,h", [(1100, 4104), (9000, 384)])
def test_block_norm_bwd_parts_rounds(dev, t, h, part):
    test_block_norm_bwd_parts(dev, t, h, part)


@pytest.mark.parametrize("t,h", [(1100, 7168), (9000, 384), (1100, 8200)])
def test_block_norm_bwd_every_row_counts(dev, t, h):
    """Column sums in which each row shows: dH yn and dn hn of row r are a power of
    two that is its own for 20 successive rows, so a row that is left out or taken
    twice changes the exact sums."""
    _say(f"block_norm_bwd row by row, {t}x{h}")
    for first in (0, t // 2, t - 20):
        dh = torch.zeros(t, h, dtype=torch.bfloat16, device=dev)
        dn = torch.zeros_like(dh)
        dh[first:first + 20] = (2.0 ** torch.arange(20, device=dev))[:, None].to(torch.bfloat16)
        one = torch.ones(t, h, dtype=torch.bfloat16, device=dev)
        w, r = torch.ones(h, device=dev), torch.ones(t, device=dev)
        dx, dy = torch.empty_like(dh), torch.empty_like(dh)
        dpost, dgate = torch.empty(h, device=dev), torch.empty(h, device=dev)
        moe.block_norm_bwd(dh, None, None, one, w, w, None, r, None, dx, dy, dpost, dgate, None,
                           moe.block_norm_workspace(t, h, dev))
        # dy is zero but for the mean, a sum of h equal terms times 1 / h: two roundings
        assert torch.equal(dx, dh) and bool((dy.abs() <= dh * 2.0 ** -22).all())
        assert bool((dpost == 2.0 ** 20 - 1).all()) and bool((dgate == 2.0 ** 20 - 1).all())
        # dn alternating in sign by column pairs: its mean with hn is zero, dH = dn
        dn[first:first + 20] = dh[first:first + 20]
        dn[:, 1::2] *= -1
        dpre = torch.empty(h, device=dev)
        moe.block_norm_bwd(None, dn, one, None, None, None, w, None, r, dx, None, None, None, dpre,
                           moe.block_norm_workspace(t, h, dev))
        assert torch.equal(dx, dn)
        assert bool((dpre[::2] == 2.0 ** 20 - 1).all()) and bool((dpre[1::2] == 1 - 2.0 ** 20).all())


def test_block_norm_bwd_against_differences(dev):
    """Central differences of the forward kernel's float64 definition at the
    kernel's own inputs: dx, dy and the weights along random directions."""
    _say("block_norm_bwd differences")
    t, h, rs, eps = 6, 256, 0.5, 1e-5
    d = _norm_inputs(t, h, "channel")
    dh, dn = _randn(t, h, seed=32), _randn(t, h, seed=33)
    v = {k: _f64(d[k]) for k in ("x", "y", "post", "gate", "pre")}
    hx, _, r1, r2 = M.block_norm(v["x"], v["y"], v["post"], v["gate"], v["pre"], rs, eps)
    res = torch.from_numpy(hx).to(dev).to(torch.bfloat16)
    out = _bwd(d, dh, dn, res, torch.from_numpy(r1).float().to(dev), torch.from_numpy(r2).float().to(dev), rs)
    r = np.random.default_rng(0)

    def loss(**kw):
        a = {**v, **kw}
        p, q, _, _ = M.block_norm(a["x"], a["y"], a["post"], a["gate"], a["pre"], rs, eps)
        return (p * _f64(dh)).sum() + (q * _f64(dn)).sum()

    for name, key in (("x", "dx"), ("y", "dy"), ("post", "dpost"), ("gate", "dgate"), ("pre", "dpre")):
        got = _f64(out[key])
        way = r.normal(size=v[name].shape)
        step = 1e-4
        slope = (loss(**{name: v[name] + step * way}) - loss(**{name: v[name] - step * way})) / (2 * step)
        # the gradient's rounding and the rounding of the kept h to BF16 (2^-9 of each value, independent):
        # 2^-8 of the 2-norm of the summed terms, five times over
        assert abs((got * way).sum() - slope) <= 5 * 2.0 ** -8 * np.linalg.norm(got * way) + 1e-6, name


def test_block_norm_no_tokens(dev):
    _say("block_norm without tokens")
    d = {k: v for k, v in _norm_inputs(4, 256, "channel").items()}
    none = torch.empty(0, 256, dtype=torch.bfloat16, device=dev)
    no = torch.empty(0, device=dev)
    moe.block_norm(none, none, d["post"], d["gate"], d["pre"], none.clone(), none.clone(), no, no.clone())
    out = [torch.full((256,), -7.0, device=dev) for _ in range(3)]
    moe.block_norm_bwd(none, none, none, none, d["post"], d["gate"], d["pre"], no, no, none.clone(), none.clone(),
                       out[0], out[1], out[2], moe.block_norm_workspace(0, 256, dev))
    assert not any(v.any().item() for v in out)


@pytest.mark.parametrize("cus", [1, 5, 100])
@pytest.mark.parametrize("t,h", [(300, 384), (70, 7168), (9, 8200)])
def test_norms_keep_to_the_compute_units_set(dev, t, h, cus):
    """With dg.set_num_cus(n) a row comes out as before and the gradient leaves at
    most n workgroups' partial column sums; its workspace serves any setting."""
    _say(f"norms on {cus} compute units, {t}x{h}")
    d = _norm_inputs(t, h, "channel")
    res, dh, dn = _randn(t, h, seed=31, scale=2.0), _randn(t, h, seed=32), _randn(t, h, seed=33)
    r1, r2 = _rstds(d, res)
    full = _bwd(d, dh, dn, res, r1, r2, 0.5)
    fwd = [_unwritten((t, h)) for _ in range(4)]
    moe.block_norm(d["x"], d["y"], d["post"], d["gate"], d["pre"], fwd[0], fwd[1])
    out = {k: torch.empty_like(v) for k, v in full.items()}
    try:
        dg.set_num_cus(cus)
        moe.block_norm(d["x"], d["y"], d["post"], d["gate"], d["pre"], fwd[2], fwd[3])
        ws = moe.block_norm_workspace(t, h, dev)
        ws.fill_(0xAB)
        moe.block_norm_bwd(dh, dn, res, d["y"], d["post"], d["gate"], d["pre"], r1, r2, out["dx"], out["dy"],
                           out["dpost"], out["dgate"], out["dpre"], ws, residual_scale=0.5)
    finally:
        dg.set_num_cus(0)
    assert torch.equal(fwd[0], fwd[2]) and torch.equal(fwd[1], fwd[3])
    assert torch.equal(out["dx"], full["dx"]) and torch.equal(out["dy"], full["dy"])
    _check_bwd(out, d, dh, dn, res, r1, r2, 0.5, f"{cus} compute units")
    assert ws.numel() >= min(t, 256) * 2 * h * 4
    assert bool((ws[min(t, cus) * 2 * h * 4:] == 0xAB).all())


# ---------------------------------------------------------------------------
# Gated activation
# ---------------------------------------------------------------------------

GLUS = [
    # layout, groups, rows (masked: max_m; contiguous: mean), inner
    ("dense", 1, 1, 128), ("dense", 1, 37, 384), ("dense", 1, 300, 2048), ("masked", 4, 33, 256), ("masked", 16, 256, 640),
    ("masked", 3, 5, 128), ("nopad", 5, 40, 384), ("nopad", 64, 3, 256), ("nopad", 300, 2, 128),
    ("contiguous", 4, 100, 256), ("contiguous", 9, 200, 896),
]


def _glu_inputs(layout, g, r, inner, dev, seed=41):
    rng = np.random.default_rng(seed + g)
    if layout == "dense":
        rows, shape = None, (r,)
    elif layout == "masked":
        rows, shape = rng.integers(-1, r + 3, g), (g, r)        # below zero and past max_m too
        rows[0] = 0
    elif layout == "nopad":
        rows, shape = rng.integers(-2, 2 * r, g), (g * r,)
    else:
        shape = (g * (-(-2 * r // 128) * 128),)
        rows = np.full(shape, -1)
        at = 0
        for i in range(g):
            c = int(rng.integers(0, 2 * r))
            rows[at:at + c] = i
            at += -(-c // 128) * 128
    gu = _randn(*shape, 2 * inner, seed=seed, scale=2.5)
    held = M.held_rows(rows, layout, shape[-1], g)
    gu[torch.from_numpy(~held).to(dev)] = float("nan")
    return None if rows is None else torch.from_numpy(np.asarray(rows, np.int32)).to(dev), gu, held


def _check_glu_codes(q, sfa, gu, held, ue8m0, what):
    """The activation's relative error is at most (|g| + 12) 2^-23: the
    exponential's argument is rounded once (|g| 2^-24) and carries a few ulp
    through it, the reciprocal and the products. A block's scale errs by the
    largest of its elements' errors, and a code must be the rounding of some
    value that close to the exact quotient by the scale that came out."""
    inner = q.shape[-1]
    a = M.swiglu(_f64(gu)[held])
    rel = (np.abs(_f64(gu)[held][:, :inner]) + 12) * 2.0 ** -23
    m = q.shape[-2]
    s = _f64(sfa)[..., :m].swapaxes(-1, -2)[held]
    top = np.maximum(np.abs(a).reshape(len(a), -1, 128).max(-1), np.float32(1e-4)) / 448.0
    off = rel.reshape(len(a), -1, 128).max(-1) + 4 * U
    if ue8m0:
        up = lambda v: 2.0 ** np.ceil(np.log2(v))  # noqa: E731
        assert ((s == up(top * (1 - off))) | (s == up(top * (1 + off)))).all(), what
    else:
        assert (np.abs(s - top) <= off * top).all(), what
    got = q.float().cpu().numpy()[held].astype(np.float64)
    wide = np.repeat(s, 128, -1)
    ends = [M.e4m3_round(np.clip(a * (1 + f * (rel + 4 * U)) / wide + f * 1e-30, -448, 448)) for f in (-1, 1)]
    assert ((got >= np.minimum(*ends)) & (got <= np.maximum(*ends))).all(), what
    # and nothing else was written
    assert (_bits(q)[~held] == 0xFF).all(), what
    rest = np.ones(sfa.shape, bool)
    rest[..., :m] = ~np.broadcast_to(held[..., None, :], (*held.shape[:-1], inner // 128, m))
    assert (_f64(sfa)[rest] == -7.0).all(), what


@pytest.mark.parametrize("ue8m0", [False, True])
@pytest.mark.parametrize("case", GLUS)
def test_swiglu_fp8(dev, case, ue8m0):
    _say(f"swiglu_fp8 {case} ue8m0={ue8m0}")
    layout, g, r, inner = case
    rows, gu, held = _glu_inputs(layout, g, r, inner, dev)
    m = gu.shape[-2]
    q = _unwritten((*gu.shape[:-1], inner), torch.float8_e4m3fn)
    sfa = _unwritten((*gu.shape[:-2], inner // 128, dg.get_tma_aligned_size(m, 4)), torch.float32)
    moe.swiglu_fp8(gu, q, sfa, rows=rows, layout=layout, ue8m0=ue8m0)
    _check_glu_codes(q, sfa, gu, held, ue8m0, str(case))


# a row a workgroup (an inner above 1024) in every layout, and more than one pass
# over a row (above 4096)
LONG_GLUS = [
    ("masked", 5, 70, 2048), ("masked", 11, 300, 1152), ("masked", 9, 9, 4480), ("masked", 3, 1, 2048),
    ("nopad", 7, 45, 1280), ("nopad", 3, 120, 4224), ("contiguous", 4, 100, 2048), ("contiguous", 3, 150, 5248),
    ("dense", 1, 70, 8320), ("dense", 1, 3, 1152),
]


@pytest.mark.parametrize("ue8m0", [False, True])
@pytest.mark.parametrize("case", LONG_GLUS)
def test_swiglu_fp8_long_rows(dev, case, ue8m0):
    test_swiglu_fp8(dev, case, ue8m0)


@pytest.mark.parametrize("case", LONG_GLUS)
def test_swiglu_bwd_long_rows(dev, case):
    test_swiglu_bwd(dev, case)


def test_swiglu_fp8_special_values(dev):
    _say("swiglu_fp8 special values")
    gu = _randn(6, 512, seed=50)
    gu[0] = 0
    gu[1, 3] = float("nan")           # g of block 0
    gu[2, 256 + 130] = float("inf")   # u of block 1
    gu[3, :256] = -200.0              # the sigmoid underflows
    gu[4, :256] = 200.0
    q, sfa = _unwritten((6, 256), torch.float8_e4m3fn), _unwritten((2, 8), torch.float32)
    moe.swiglu_fp8(gu, q, sfa)
    v, s = q.float().cpu().numpy(), _f64(sfa)
    assert not v[0].any() and (s[:, 0] == np.float32(np.float32(1e-4) / np.float32(448))).all()
    assert np.isnan(v[1, :128]).all() and np.isnan(s[0, 1]) and np.isfinite(v[1, 128:]).all() and np.isfinite(s[1, 1])
    assert np.isinf(s[1, 2]) and np.isnan(v[2, 130]) and not np.delete(v[2, 128:], 2).any()
    assert np.isfinite(v[2, :128]).all()
    assert not v[3].any()
    a = 200.0 * _f64(gu)[4, 256:]
    assert np.array_equal(s[:, 4], (np.abs(a).reshape(2, 128).max(1).astype(np.float32) / np.float32(448)))


def test_swiglu_smallest_sigmoids(dev):
    """Gates from -87.5 to -88.5, whose sigmoids are below 2^-126: with a u as large
    as BF16's, what they make is no less exact than elsewhere."""
    _say("swiglu, sigmoids below 2^-126")
    inner = 256
    gate = torch.tensor([-87.0, -87.5, -88.0, -88.5]).repeat_interleave(inner).view(4, inner)
    up = torch.linspace(1.0, 3.0, inner).repeat(4, 1) * 2.0 ** 126
    gu = torch.cat([gate, up], 1).to(dev).to(torch.bfloat16)
    rows, held = None, np.ones(4, bool)
    q, sfa = _unwritten((4, inner), torch.float8_e4m3fn), _unwritten((inner // 128, 4), torch.float32)
    moe.swiglu_fp8(gu, q, sfa, rows=rows)
    _check_glu_codes(q, sfa, gu, held, False, "smallest sigmoids")
    da, dgu = _randn(4, inner, seed=44), _unwritten((4, 2 * inner))
    moe.swiglu_bwd(da, gu, dgu)
    x, d = _f64(gu), _f64(da)
    s, rel = M.sigmoid(x[:, :inner]), (np.abs(x[:, :inner]) + 16) * 2.0 ** -23
    mag = np.concatenate([np.abs(d * x[:, inner:]) * s * (1 + np.abs(x[:, :inner])), np.abs(d * x[:, :inner]) * s], -1)
    check_bf16(dgu, M.swiglu_bwd(d, x), mag * np.concatenate([rel, rel], -1), "smallest sigmoids")


@pytest.mark.parametrize("case", GLUS)
def test_swiglu_bwd(dev, case):
    _say(f"swiglu_bwd {case}")
    layout, g, r, inner = case
    rows, gu, held = _glu_inputs(layout, g, r, inner, dev)
    da = _randn(*gu.shape[:-1], inner, seed=43)
    da[torch.from_numpy(~held).to(dev)] = float("nan")
    dgu = _unwritten(gu.shape)
    moe.swiglu_bwd(da, gu, dgu, rows=rows, layout=layout)
    assert (_bits(dgu)[~held] == SENTINEL).all()
    if not held.any():
        return
    x, d = _f64(gu)[held], _f64(da)[held]
    gate, up = x[:, :inner], x[:, inner:]
    s, rel = M.sigmoid(gate), (np.abs(gate) + 16) * 2.0 ** -23
    mag = np.concatenate([np.abs(d * up) * s * (1 + np.abs(gate)), np.abs(d * gate) * s], -1)
    check_bf16(dgu[torch.from_numpy(held).to(dev)], M.swiglu_bwd(d, x), mag * np.concatenate([rel, rel], -1) + 1e-30,
               str(case))


# ---------------------------------------------------------------------------
# Addresses, streams, graphs, repeatability, refusals
# ---------------------------------------------------------------------------

def test_offsets_past_32_bits(dev):
    """Permuted buffers past 2^31 elements (and 2^32 bytes): the last rows."""
    _say("offsets past 32 bits")
    hidden, rows = 7168, 300_032                       # 2.15e9 elements, 4.3e9 bytes in BF16
    plan = moe.Plan(4, 2, 8, "nopad", rows, hidden, dev)
    row_of = np.array([[rows - 1, 0], [rows - 2, -1], [5, rows - 300], [1, 2]])
    plan.row_of.copy_(torch.from_numpy(row_of.astype(np.int32)))
    x = _randn(4, hidden, seed=60)
    xp = torch.zeros(rows, hidden, dtype=torch.bfloat16, device=dev)
    moe.dispatch(plan, x, xp)
    for i, j in np.argwhere(row_of >= 0):
        assert torch.equal(xp[row_of[i, j]], x[i])
    y = _unwritten((4, hidden))
    moe.combine(plan, xp, y)
    assert torch.equal(y[1], x[1]) and torch.equal(y[3], (x[3].float() * 2).to(torch.bfloat16))
    w = torch.ones(4, 2, device=dev)
    dw = torch.zeros(4, 2, device=dev)
    xp2 = torch.zeros_like(xp)
    moe.combine_bwd(plan, x, xp, w, xp2, dw)
    assert torch.equal(xp2[rows - 1], x[0]) and torch.equal(xp2[rows - 300], x[2])
    assert dw[1, 1].item() == 0 and abs(dw[0, 0].item() - x[0].double().square().sum().item()) < 1e-2
    del xp2
    q = torch.zeros(rows, hidden, dtype=torch.float8_e4m3fn, device=dev)
    sfa = torch.zeros(plan.scale_shape, device=dev)
    moe.dispatch_fp8(plan, x, q, sfa)
    vals, scales = M.quantize(_f64(x).astype(np.float32), False)
    assert np.array_equal(q[rows - 1].float().cpu().numpy(), vals[0]) and np.array_equal(_f64(sfa[:, rows - 1]), scales[0])
    assert np.array_equal(q[rows - 300].float().cpu().numpy(), vals[2])


def test_norm_offsets_past_32_bits(dev):
    """The last of 300000 rows of 7168 (2.15e9 elements) as when normalised alone."""
    _say("norm offsets past 32 bits")
    t, h, last = 300_000, 7168, 5
    d = _norm_inputs(last, h, "channel")
    x, y = torch.zeros(t, h, dtype=torch.bfloat16, device=dev), torch.zeros(t, h, dtype=torch.bfloat16, device=dev)
    x[-last:], y[-last:] = d["x"], d["y"]
    r1, r2 = torch.zeros(t, device=dev), torch.zeros(t, device=dev)
    small = [torch.zeros(last, h, dtype=torch.bfloat16, device=dev) for _ in range(4)]
    s1, s2 = torch.zeros(last, device=dev), torch.zeros(last, device=dev)
    moe.block_norm(d["x"], d["y"], d["post"], d["gate"], d["pre"], small[0], small[1], s1, s2)
    moe.block_norm(x, y, d["post"], d["gate"], d["pre"], x, y, r1, r2)               # in place
    assert torch.equal(x[-last:], small[0]) and torch.equal(y[-last:], small[1])
    assert torch.equal(r1[-last:], s1) and torch.equal(r2[-last:], s2)
    # and the gradient, dh = h and dn = n standing in
    cols = [torch.zeros(h, device=dev) for _ in range(3)]
    moe.block_norm_bwd(small[0], small[1], small[0], d["y"], d["post"], d["gate"], d["pre"], s1, s2, small[2], small[3],
                       *cols, moe.block_norm_workspace(last, h, dev))
    yin = torch.zeros(t, h, dtype=torch.bfloat16, device=dev)
    yin[-last:] = d["y"]
    dx, dy = torch.zeros_like(x), torch.zeros_like(x)
    moe.block_norm_bwd(x, y, x, yin, d["post"], d["gate"], d["pre"], r1, r2, dx, dy, None, None, None,
                       moe.block_norm_workspace(t, h, dev))
    assert torch.equal(dx[-last:], small[2]) and torch.equal(dy[-last:], small[3]) and not dx[:-last].any()


def test_glu_offsets_past_32_bits(dev):
    _say("activation offsets past 32 bits")
    inner, m = 2048, 524_800                           # gu: 2.15e9 elements, 4.3e9 bytes
    gu = torch.zeros(m, 2 * inner, dtype=torch.bfloat16, device=dev)
    gu[-3:] = _randn(3, 2 * inner, seed=61)
    q = torch.zeros(m, inner, dtype=torch.float8_e4m3fn, device=dev)
    sfa = torch.zeros(inner // 128, m, device=dev)
    moe.swiglu_fp8(gu, q, sfa)
    small_q, small_s = _unwritten((3, inner), torch.float8_e4m3fn), _unwritten((inner // 128, 4), torch.float32)
    moe.swiglu_fp8(gu[-3:].clone(), small_q, small_s)
    assert np.array_equal(_bits(q[-3:]), _bits(small_q)) and torch.equal(sfa[:, -3:], small_s[:, :3])
    da = torch.zeros(m, inner, dtype=torch.bfloat16, device=dev)
    da[-3:] = _randn(3, inner, seed=62)
    dgu = torch.zeros_like(gu)
    moe.swiglu_bwd(da, gu, dgu)
    small = _unwritten((3, 2 * inner))
    moe.swiglu_bwd(da[-3:].clone(), gu[-3:].clone(), small)
    assert torch.equal(dgu[-3:], small) and not dgu[:-3].any()


def _block_calls(dev, t=70, k=4, g=6, hidden=512, inner=256, layout="nopad", seed=70):
    """Every entry point once, on buffers of its own: (inputs to refill, calls, outputs)."""
    plan = _make_plan(t, k, g, layout, None, hidden)
    x, dy, y = _randn(t, hidden, seed=seed), _randn(t, hidden, seed=seed + 1), _unwritten((t, hidden))
    ids = torch.from_numpy(_ids(t, k, g, seed)).to(dev)
    w = torch.softmax(_randn(t, k, seed=seed + 2, dtype=torch.float32), 1)
    yp = _randn(*plan.rows_shape, seed=seed + 3)
    xp, dyp = torch.zeros_like(yp), torch.zeros_like(yp)
    q, sfa = torch.zeros(plan.rows_shape, dtype=torch.float8_e4m3fn, device=dev), torch.zeros(plan.scale_shape, device=dev)
    dw = torch.zeros(t, k, device=dev)
    m = plan.rows
    gu, da = _randn(m, 2 * inner, seed=seed + 4), _randn(m, inner, seed=seed + 5)
    gq = torch.zeros(m, inner, dtype=torch.float8_e4m3fn, device=dev)
    gs, dgu = torch.zeros(inner // 128, dg.get_tma_aligned_size(m, 4), device=dev), torch.zeros_like(gu)
    d = _norm_inputs(t, hidden, "channel", seed + 6)
    h, n, dx, dyn = (torch.zeros(t, hidden, dtype=torch.bfloat16, device=dev) for _ in range(4))
    r1, r2 = torch.zeros(t, device=dev), torch.zeros(t, device=dev)
    cols = [torch.zeros(hidden, device=dev) for _ in range(3)]
    ws = moe.block_norm_workspace(t, hidden, dev)

    def run():
        moe.dispatch(plan, x, xp, topk_ids=ids)
        moe.dispatch_fp8(plan, x, q, sfa, topk_ids=ids)
        moe.sort(plan, ids)
        moe.combine(plan, yp, y, weights=w)
        moe.combine_bwd(plan, dy, yp, w, dyp, dw)
        moe.swiglu_fp8(gu, gq, gs, rows=plan.group_rows, layout=layout)
        moe.swiglu_bwd(da, gu, dgu, rows=plan.group_rows, layout=layout)
        moe.block_norm(d["x"], y, d["post"], d["gate"], d["pre"], h, n, r1, r2)
        moe.block_norm_bwd(dy, x, h, y, d["post"], d["gate"], d["pre"], r1, r2, dx, dyn, cols[0], cols[1], cols[2], ws)

    outs = [plan.row_of, plan.group_rows, xp, q, sfa, y, dyp, dw, gq, gs, dgu, h, n, r1, r2, dx, dyn, *cols]
    return (x, dy, yp, gu, da, ids), run, outs


def _snap(outs):
    return [_bits(o).copy() for o in outs]


@pytest.mark.parametrize("t", [70, 1500])
def test_graph_replay_and_repeatability(dev, t):
    """Captured once, replayed with new inputs between eager work: every replay
    gives the bits of eager calls, and so does a second eager run."""
    _say(f"graph replay {t}")
    inputs, run, outs = _block_calls(dev, t=t)
    run()
    torch.cuda.synchronize()
    first = _snap(outs)
    run()
    torch.cuda.synchronize()
    assert all(np.array_equal(a, b) for a, b in zip(first, _snap(outs)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for i in range(3):
        for v in inputs[:-1]:
            v.copy_(_randn(*v.shape, seed=100 + i))
        inputs[-1].copy_(torch.from_numpy(_ids(*inputs[-1].shape, 6, 200 + i)).to(dev))
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        replayed = _snap(outs)
        for o in outs:
            o.zero_()
        run()
        torch.cuda.synchronize()
        assert all(np.array_equal(a, b) for a, b in zip(replayed, _snap(outs))), i


def test_streams(dev):
    """Two sets of calls in flight on two streams, each as when run alone."""
    _say("two streams")
    sets = [_block_calls(dev, t=900, seed=s) for s in (300, 400)]
    for _, run, _ in sets:
        run()
    torch.cuda.synchronize()
    alone = [_snap(outs) for _, _, outs in sets]
    for _, _, outs in sets:
        for o in outs:
            o.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        for s, (_, run, _) in zip(streams, sets):
            with torch.cuda.stream(s):
                run()
    torch.cuda.synchronize()
    for want, (_, _, outs) in zip(alone, sets):
        assert all(np.array_equal(a, b) for a, b in zip(want, _snap(outs)))


def test_graph_replay_and_repeatability_many_slots(dev):
    test_graph_replay_and_repeatability(dev, 4200)


def test_streams_many_slots(dev):
    """As test_streams, with more slots than one launch sorts."""
    _say("two streams, many slots")
    sets = [_block_calls(dev, t=t, seed=s) for t, s in ((4200, 500), (4500, 600))]
    torch.cuda.synchronize()
    alone = []
    for _, run, outs in sets:
        run()
        torch.cuda.synchronize()
        alone.append(_snap(outs))
        for o in outs:
            o.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        for s, (_, run, _) in zip(streams, sets):
            with torch.cuda.stream(s):
                run()
    torch.cuda.synchronize()
    for want, (_, _, outs) in zip(alone, sets):
        assert all(np.array_equal(a, b) for a, b in zip(want, _snap(outs)))


def test_refusals(dev):
    _say("refusals")
    plan = _make_plan(8, 2, 4, "masked", 16)
    x, ids = _randn(8, 256, seed=1), torch.zeros(8, 2, dtype=torch.int32, device=dev)
    xp = torch.zeros(plan.rows_shape, dtype=torch.bfloat16, device=dev)
    with pytest.raises(TypeError):
        moe.sort(plan, ids.long())
    with pytest.raises(ValueError):
        moe.sort(plan, ids[:, :1])
    with pytest.raises(ValueError):
        moe.sort(plan, ids.cpu())
    with pytest.raises(ValueError):
        moe.dispatch(plan, _randn(9, 256, seed=1), xp, topk_ids=None)
    with pytest.raises(ValueError):
        moe.dispatch(plan, x, xp.view(-1, 256))
    with pytest.raises(ValueError):
        moe.dispatch(plan, _randn(256, 8, seed=1).t(), xp)
    with pytest.raises(TypeError):
        moe.dispatch(plan, x.float(), xp)
    with pytest.raises(ValueError):
        moe.dispatch(plan, x[:4], xp, topk_ids=ids)
    with pytest.raises(TypeError):
        moe.dispatch_fp8(plan, x, xp, torch.zeros(plan.scale_shape, device=dev))
    with pytest.raises(ValueError):
        moe.dispatch_fp8(plan, x, xp.to(torch.float8_e4m3fn), torch.zeros(plan.scale_shape, device=dev)[:, :, :12])
    with pytest.raises(ValueError):
        moe.combine(plan, xp, x, weights=torch.zeros(8, 3, device=dev))
    with pytest.raises(TypeError):
        moe.combine_bwd(plan, x, None, torch.zeros(8, 2, device=dev), xp, torch.zeros(8, 2, device=dev))
    with pytest.raises(dg.DGError):                      # 2-byte shift: not 16-byte aligned
        moe.combine(plan, xp, torch.zeros(8 * 256 + 1, dtype=torch.bfloat16, device=dev)[1:].view(8, 256))
    gu = _randn(16, 512, seed=1)
    q, s = torch.zeros(16, 256, dtype=torch.float8_e4m3fn, device=dev), torch.zeros(2, 16, device=dev)
    with pytest.raises(ValueError):
        moe.swiglu_fp8(gu, q, s, layout="ragged")
    with pytest.raises(ValueError):
        moe.swiglu_fp8(gu, q, s, rows=plan.group_rows)
    with pytest.raises(TypeError):
        moe.swiglu_fp8(gu, q, s, layout="nopad")
    with pytest.raises(ValueError):
        moe.swiglu_fp8(gu, q, s, rows=plan.group_rows, layout="contiguous")
    with pytest.raises(ValueError):
        moe.swiglu_fp8(gu[:, :384], q, s)
    with pytest.raises(ValueError):
        moe.swiglu_bwd(gu, gu, gu.clone())
    d = _norm_inputs(8, 256, "channel")
    h, n = torch.zeros_like(x), torch.zeros_like(x)
    with pytest.raises(ValueError):                      # one gate value a token has to be [tokens, 1]
        moe.block_norm(x, x, d["post"], torch.zeros(8, device=dev), d["pre"], h, n)
    with pytest.raises(TypeError):
        moe.block_norm(x, x, d["post"], 0.5, d["pre"], h, n)
    with pytest.raises(TypeError):
        moe.block_norm(x, x, d["post"].bfloat16(), None, d["pre"], h, n)
    with pytest.raises(dg.DGError):
        moe.block_norm(x, None, d["post"], None, d["pre"], None, n)
    with pytest.raises(dg.DGError):
        moe.block_norm(x, x, d["post"], None, d["pre"], None, n)
    with pytest.raises(dg.DGError):
        moe.block_norm_bwd(None, None, h, x, d["post"], None, None, None, None, h, n, None, None, None,
                           moe.block_norm_workspace(8, 256, dev))
    with pytest.raises(dg.DGError):
        r = torch.zeros(8, device=dev)
        moe.block_norm_bwd(x, x, x, x, d["post"], None, d["pre"], r, r, h, n, None, None, None,
                           torch.zeros(16, dtype=torch.uint8, device=dev))


def test_example_block(dev):
    """The block of examples/moe_block.py against float32 in the three layouts,
    and its gradients. Each FP8 operand is off by up to 2^-4 of a value, evenly
    spread: 2^-4 / sqrt(3) = 3.6% at most in norm an operand, four operands a
    forward pass and two more products on the way back; the residual stream
    and the norms only dilute it. 15% would be a wrong row or weight."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")
    spec = importlib.util.spec_from_file_location("moe_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    errors = mod.compare()
    _say(errors)
    assert len(errors) == 12 and all(e < 0.15 for e in errors.values()), errors


def test_workspace_serves_smaller_chunks(dev):
    """Just past 256 chunks of 1024 slots a chunk doubles: fewer slots then need
    more rows of the workspace than the most slots do."""
    _say("sort with more chunks than the plan's most slots take")
    plan = moe.Plan(263_000, 1, 7, "nopad", 263_000, 128, dev)
    for t in (262_144, 263_000):
        ids = _ids(t, 1, 7, t)
        moe.sort(plan, torch.from_numpy(ids).to(dev))
        _check_sorted(plan, ids)
    assert plan.workspace.numel() >= 256 * 7 * 4
