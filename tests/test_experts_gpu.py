"""GPU parity of the expert layer for a few tokens against its float64 definition.

With u = 2^-24: a float32 sum of K products on the matrix cores is within
(4 K / 32 + 64) u of the sum of their magnitudes (32 products an instruction,
taken as four roundings, and a few additions across waves), and silu within (|g| + 12)
2^-23. silu(g) u is rounded to BF16, 2^-8 of its size at most, and y once more.
Weights and tokens chosen so that every step is exact have to give bf16(y) bit for bit.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

from moe_grouped_gemm_amd import dg, moe, synth
from oracle import dg_oracle as O
from oracle import fp4_oracle as F
from parity import bf16_ulp

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()
    return torch.device("cuda:0")


def _say(msg):
    print(msg, flush=True)


def _weights(fp4, g, n, k, seed, dev):
    """(b, sfb, values): N(0, 1/K) weights quantised for the products."""
    gen = torch.Generator().manual_seed(seed)
    b, sf, v = [], [], []
    for _ in range(g):
        w = torch.randn(n, k, generator=gen) * k ** -0.5
        if fp4:
            q, s = F.quantize(w.double().numpy())
            v.append(F.values(q, s))
            b.append(torch.from_numpy(q))
            sf.append(torch.from_numpy(s.astype(np.uint32).view(np.int32)))
        else:
            q, s = synth.quantize_rhs(w)
            b.append(q)
            sf.append(s)
            v.append(q.double().numpy() * np.repeat(np.repeat(s.double().numpy(), 128, 0), 128, 1))
    return torch.stack(b).to(dev), torch.stack(sf).contiguous().to(dev), np.stack(v)


def _ids(t, k, g, seed, drop=0.1):
    r = np.random.default_rng(seed)
    ids = np.stack([r.permutation(max(g, k))[:k] for _ in range(t)]).astype(np.int32) if t else np.zeros((0, k), np.int32)
    ids[r.random((t, k)) < drop] = -1
    return ids


def _run(x, ids, w, b1, sfb1, b2, sfb2, dev):
    t, hidden = x.shape
    ws = moe.experts_workspace(t, ids.shape[1], b1.shape[0], b1.shape[1] // 2, dev)
    ws.fill_(0xFF)                                   # NaN wherever nothing was written
    y = torch.full((t, hidden), -1, dtype=torch.int16, device=dev).view(torch.bfloat16)
    return moe.experts(x, torch.from_numpy(ids).to(dev), w, b1, sfb1, b2, sfb2, y, ws)


def _check(y, x, ids, w, v1, v2):
    ref, act_mag, mag, top = F.experts(x.double().cpu().numpy(), ids, w, v1, v2)
    hidden, inner = v1.shape[2], v2.shape[2]
    err = (2.0 ** -8 + (top + 12) * 2.0 ** -23 + (inner / 8 + 64) * U) * act_mag + (hidden / 8 + 64) * U * mag
    got = y.double().cpu().numpy()
    assert np.isfinite(got).all()
    bad = np.abs(got - ref) > bf16_ulp(np.maximum(np.abs(got), np.abs(ref) + err)) / 2 + err
    assert not bad.any(), f"{bad.sum()} beyond the bound, first {np.argwhere(bad)[:3].tolist()}"
    # the two BF16 roundings are 2^-8 each at most, and 0.6 of that in the 2-norm for values spread within their steps
    norm = np.linalg.norm(ref)
    assert np.linalg.norm(got - ref) <= 2.0 ** -8 * 1.25 * norm, np.linalg.norm(got - ref) / max(norm, 1e-300)


LAYERS = [
    # tokens, top_k, groups, hidden, inner
    (1, 1, 1, 128, 128), (1, 8, 16, 640, 256), (3, 2, 8, 2048, 512), (5, 8, 16, 384, 128), (16, 4, 6, 256, 384),
    (17, 3, 40, 512, 256), (33, 8, 9, 384, 128), (64, 2, 3, 256, 256), (100, 8, 12, 128, 256), (128, 8, 64, 256, 128),
    (7, 32, 32, 256, 128), (2, 3, 4096, 128, 128), (40, 1, 1, 896, 1152), (128, 1, 2, 128, 128),
    # rows so short that several workgroups share the experts of their columns
    (30, 8, 40, 256, 1024), (9, 4, 30, 384, 1280), (100, 3, 20, 128, 2048), (3, 8, 40, 2048, 640),
]


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("case", LAYERS)
def test_layer(dev, case, fp4):
    _say(f"experts {case} fp4={fp4}")
    t, k, g, hidden, inner = case
    b1, sfb1, v1 = _weights(fp4, min(g, 64), 2 * inner, hidden, 1, dev)
    b2, sfb2, v2 = _weights(fp4, min(g, 64), hidden, inner, 2, dev)
    ids = _ids(t, k, min(g, 64), t + g)
    if g > 64:                                       # few of many: the others' weights are never read
        b1, b2 = (torch.cat([b, torch.full((g - 64, *b.shape[1:]), 0x7F, dtype=torch.uint8, device=dev).view(b.dtype)]) for b in (b1, b2))
        sfb1, sfb2 = (torch.cat([s, torch.full((g - 64, *s.shape[1:]), -1, device=dev).to(s.dtype)]) for s in (sfb1, sfb2))
    x = torch.randn(t, hidden, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).to(dev)
    w = torch.rand(t, k, generator=torch.Generator().manual_seed(4)).to(dev)
    y = _run(x, ids, w, b1, sfb1, b2, sfb2, dev)
    _check(y, x, ids, w.cpu().numpy(), v1, v2)
    again = _run(x, ids, w, b1, sfb1, b2, sfb2, dev)
    assert torch.equal(again.view(torch.int16), y.view(torch.int16))
    ones = _run(x, ids, None, b1, sfb1, b2, sfb2, dev)
    _check(ones, x, ids, np.ones((t, k)), v1, v2)


def _exact_layer(fp4, t, g, hidden, inner, seed, dev):
    """Gates of 32 (their sigmoid is 1 in float32), ups of a whole number picked out of
    x, second weights whole: everything is exact but the last rounding."""
    r = np.random.default_rng(seed)
    v1, v2 = np.zeros((g, 2 * inner, hidden)), r.choice([-2.0, -1.0, 0.0, 0.0, 1.0, 3.0], (g, hidden, inner))
    pick = 1 + r.integers(0, hidden - 1, (g, inner))
    for e in range(g):
        v1[e, :inner, 0] = 1.0
        v1[e, inner + np.arange(inner), pick[e]] = r.choice([-1.0, 1.0, 2.0], inner)
    x = r.integers(-4, 5, (t, hidden)).astype(np.float64)
    x[:, 0] = 32.0
    sent = []
    for v in (v1, v2):
        if fp4:
            scale = np.full((g, v.shape[1], v.shape[2] // 32), 127, np.uint8)
            q, s = F.pack(F.codes(v, scale)), F.words(scale).astype(np.uint32).view(np.int32)
            sent += [torch.from_numpy(q).to(dev), torch.from_numpy(np.ascontiguousarray(s)).to(dev)]
        else:
            sent += [torch.from_numpy(v).to(torch.float8_e4m3fn).to(dev),
                     torch.ones(g, v.shape[1] // 128, v.shape[2] // 128, device=dev)]
    return torch.from_numpy(x).to(torch.bfloat16).to(dev), sent, v1, v2


def _exact(x, ids, w, v1, v2):
    """The layer of _exact_layer: silu(g) u = g u, since 1 + e^-32 is 1 in float32 (e^-32 <
    2^-25). Whole numbers, so float64 sums are exact."""
    y = np.zeros((x.shape[0], v2.shape[1]))
    inner = v2.shape[2]
    for t, j in np.argwhere((ids >= 0) & (ids < v1.shape[0])):
        gu = v1[ids[t, j]] @ x[t]
        y[t] += w[t, j] * (v2[ids[t, j]] @ (gu[:inner] * gu[inner:]))
    assert np.abs(y).max(initial=0) * 4 < 2 ** 24
    return y


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("t,k,g,hidden,inner", [(1, 2, 4, 384, 128), (9, 3, 5, 256, 384), (61, 4, 8, 640, 256),
                                                (128, 8, 10, 128, 640), (30, 8, 256, 256, 128), (1, 1, 2, 1152, 2048)])
def test_exact_layer(dev, t, k, g, hidden, inner, fp4):
    _say(f"experts, exact: {(t, k, g, hidden, inner)} fp4={fp4}")
    x, sent, v1, v2 = _exact_layer(fp4, t, g, hidden, inner, t, dev)
    ids = _ids(t, k, g, t)
    w = np.random.default_rng(t).choice([0.25, 0.5, 1.0, -2.0], (t, k))
    y = _run(x, ids, torch.from_numpy(w).float().to(dev), *sent, dev)
    ref = _exact(x.double().cpu().numpy(), ids, w, v1, v2)
    np.testing.assert_array_equal(y.view(torch.int16).cpu().numpy().view(np.uint16), O.bf16_bits(ref))


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("t,k,g,hidden,inner", [(1, 2, 4, 384, 128), (3, 4, 9, 256, 1024), (9, 3, 5, 256, 384), (16, 2, 4, 4224, 128),
                                                (30, 4, 40, 256, 512), (61, 4, 8, 640, 256), (128, 4, 10, 128, 384)])
def test_activations_of_more_bits_than_bf16_has(dev, t, k, g, hidden, inner, fp4):
    """As _exact_layer, with ups 6 a + b / 2 of whole a and b up to 127: silu(g) u = 32 u has up to 11
    significant bits, which reach the second products whole. Everything is a multiple of 4."""
    _say(f"experts, long activations: {(t, k, g, hidden, inner)} fp4={fp4}")
    x, sent, v1, v2 = _exact_layer(fp4, t, g, hidden, inner, t, dev)
    r = np.random.default_rng(t + 1)
    x[:, 1:] = torch.from_numpy(r.integers(-127, 128, (t, hidden - 1))).to(x)
    v1[:, inner:] = 0.0
    for e in range(g):
        two = np.stack([1 + r.permutation(hidden - 1)[:2] for _ in range(inner)])
        v1[e, inner + np.arange(inner), two[:, 0]] = 6.0
        v1[e, inner + np.arange(inner), two[:, 1]] = 0.5
    if fp4:
        scale = np.full((g, 2 * inner, hidden // 32), 127, np.uint8)
        sent[0] = torch.from_numpy(F.pack(F.codes(v1, scale))).to(dev)
    else:
        sent[0] = torch.from_numpy(v1).to(torch.float8_e4m3fn).to(dev)
    ids = _ids(t, k, g, t)
    w = r.choice([0.25, 0.5, 1.0, -1.0], (t, k))
    y = _run(x, ids, torch.from_numpy(w).float().to(dev), *sent, dev)
    xs = x.double().cpu().numpy()
    ref, mag = np.zeros((t, hidden)), np.zeros((t, hidden))
    long = 0
    for i, j in np.argwhere(ids >= 0):
        gu = v1[ids[i, j]] @ xs[i]
        a = gu[:inner] * gu[inner:]
        long += (O.bf16_round(a) != a).sum()
        ref[i] += w[i, j] * (v2[ids[i, j]] @ a)
        mag[i] += abs(w[i, j]) * (np.abs(v2[ids[i, j]]) @ np.abs(a))
    assert mag.max() / 4 < 2 ** 24 and long > inner // 4
    np.testing.assert_array_equal(y.view(torch.int16).cpu().numpy().view(np.uint16), O.bf16_bits(ref))


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("t,k,g", [(9, 2, 24), (16, 1, 17), (17, 4, 70), (24, 2, 48), (33, 2, 96), (128, 1, 128)])
def test_many_tokens_of_an_expert_among_more_experts_than_slots(dev, t, k, g, fp4):
    """Tiles of activations known by their first pairs' slots, several an expert."""
    _say(f"experts, crowded: {(t, k, g)} fp4={fp4}")
    hidden, inner = 256, 256
    x, sent, v1, v2 = _exact_layer(fp4, t, g, hidden, inner, t, dev)
    r = np.random.default_rng(t)
    for crowd in (1, 2):
        ids = np.asarray(r.choice(r.permutation(g)[:crowd], (t, k)), np.int32)
        ids[:, 1:][r.random((t, k - 1)) < 0.3] = -1
        w = r.choice([0.25, 0.5, 1.0, -2.0], (t, k))
        y = _run(x, ids, torch.from_numpy(w).float().to(dev), *sent, dev)
        ref = _exact(x.double().cpu().numpy(), ids, w, v1, v2)
        np.testing.assert_array_equal(y.view(torch.int16).cpu().numpy().view(np.uint16), O.bf16_bits(ref))


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("t", [1, 6, 20])
def test_infinite_activations_stay_infinite(dev, t, fp4):
    """An activation past float32's range is infinite, with nothing left over beside it: so are
    the outputs that it reaches through weights of one sign, and no other token's."""
    _say(f"experts, infinite activations t={t} fp4={fp4}")
    g, hidden, inner = 2, 256, 128
    x, sent, v1, v2 = _exact_layer(fp4, t, g, hidden, inner, t, dev)
    ids = np.zeros((t, 1), np.int32)
    first = int(np.flatnonzero(v1[0, inner])[0])         # what the first activation's up is picked from
    x[:, 1:] = x[:, 1:].abs()
    x[0, first] = 2.0 ** 127
    up, ones = np.abs(v1), np.ones_like(v2)
    for i, v in ((0, up), (2, ones)):
        if fp4:
            sent[i] = torch.from_numpy(F.pack(F.codes(v, np.full((g, v.shape[1], v.shape[2] // 32), 127, np.uint8)))).to(dev)
        else:
            sent[i] = torch.from_numpy(v).to(torch.float8_e4m3fn).to(dev)
    y = _run(x, ids, None, *sent, dev)
    assert torch.equal(y[0], torch.full_like(y[0], float("inf")))
    ref = _exact(x[1:].double().cpu().numpy(), ids[1:], np.ones((t - 1, 1)), up, ones)
    np.testing.assert_array_equal(y[1:].view(torch.int16).cpu().numpy().view(np.uint16), O.bf16_bits(ref))


@pytest.mark.parametrize("fp4", [False, True])
def test_ids_and_weights_at_their_ends(dev, fp4):
    """An expert named twice by a token, ids outside the experts with weights that are not
    numbers, tokens without experts, one expert for all."""
    _say(f"experts, ids fp4={fp4}")
    t, k, g, hidden, inner = 40, 4, 7, 256, 256
    x, sent, v1, v2 = _exact_layer(fp4, t, g, hidden, inner, 5, dev)
    r = np.random.default_rng(0)
    lo, hi = np.iinfo(np.int32).min, np.iinfo(np.int32).max
    for kind in ("twice", "outside", "none", "one"):
        ids = r.integers(0, g, (t, k)).astype(np.int32)                    # with repeats
        w = r.choice([0.25, 0.5, 1.0, -2.0], (t, k))
        if kind == "twice":
            ids[:, 2] = ids[:, 0]
        elif kind == "outside":
            ids[r.random((t, k)) < 0.5] = -1
            ids[0], ids[3] = [lo, hi, g, -1], [g, 0, lo, 0]
            w[(ids < 0) | (ids >= g)] = np.nan
        elif kind == "none":
            ids[:] = -1
            ids[7, 1] = g - 1
        else:
            ids[:] = 3
        y = _run(x, ids, torch.from_numpy(w).float().to(dev), *sent, dev)
        ref = _exact(x.double().cpu().numpy(), ids, w, v1, v2)
        np.testing.assert_array_equal(y.view(torch.int16).cpu().numpy().view(np.uint16), O.bf16_bits(ref), kind)


@pytest.mark.parametrize("fp4", [False, True])
def test_not_finite(dev, fp4):
    """A NaN or an infinity in a token reaches that token alone."""
    _say(f"experts, not finite fp4={fp4}")
    t, k, g, hidden, inner = 20, 2, 3, 256, 128
    x, sent, v1, v2 = _exact_layer(fp4, t, g, hidden, inner, 6, dev)
    ids = r = np.random.default_rng(1).integers(0, g, (t, k)).astype(np.int32)
    ids[4] = [1, 2]
    clean = _run(x, ids, None, *sent, dev)
    x[4, 17] = float("nan")
    x[9, 0] = float("inf")
    y = _run(x, ids, None, *sent, dev)
    rest = [i for i in range(t) if i not in (4, 9)]
    assert torch.equal(y[rest].view(torch.int16), clean[rest].view(torch.int16))
    assert torch.isnan(y[4]).all() and not torch.isfinite(y[9]).any() and len(r) == t


def test_no_tokens(dev):
    _say("experts, no tokens")
    x, sent, _, _ = _exact_layer(False, 0, 2, 128, 128, 1, dev)
    assert _run(x, np.zeros((0, 3), np.int32), None, *sent, dev).shape == (0, 128)


@pytest.mark.parametrize("fp4", [False, True])
def test_graph_with_other_tokens_and_ids(dev, fp4):
    """Captured once, replayed with other tokens, ids and weights; and a second graph
    that shares the workspace, replayed in between."""
    _say(f"experts in a graph, fp4={fp4}")
    t, k, g, hidden, inner = 12, 3, 6, 256, 256
    x0, sent, v1, v2 = _exact_layer(fp4, t, g, hidden, inner, 8, dev)
    ws = moe.experts_workspace(t, k, g, inner, dev)
    calls = []
    for n in (t, 5):
        x, ids, w = x0[:n].clone(), torch.zeros(n, k, dtype=torch.int32, device=dev), torch.ones(n, k, device=dev)
        y = torch.zeros(n, hidden, dtype=torch.bfloat16, device=dev)
        moe.experts(x, ids, w, *sent, y, ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            moe.experts(x, ids, w, *sent, y, ws)
        calls.append((graph, x, ids, w, y))
    for seed in range(4):
        for graph, x, ids, w, y in calls:
            r = np.random.default_rng(seed)
            new = r.integers(-1, g, tuple(ids.shape)).astype(np.int32)
            x[:, 1:] = torch.from_numpy(r.integers(-4, 5, (x.shape[0], hidden - 1))).to(x)
            ids.copy_(torch.from_numpy(new))
            weight = r.choice([0.5, 1.0, -2.0], new.shape)
            w.copy_(torch.from_numpy(weight))
            graph.replay()
            torch.cuda.synchronize()
            ref = _exact(x.double().cpu().numpy(), new, weight, v1, v2)
            np.testing.assert_array_equal(y.view(torch.int16).cpu().numpy().view(np.uint16), O.bf16_bits(ref))


def test_two_streams_with_workspaces_of_their_own(dev):
    _say("experts on two streams")
    t, k, g, hidden, inner = 20, 4, 6, 512, 384
    layers = [_exact_layer(fp4, t, g, hidden, inner, 11 + fp4, dev) for fp4 in (False, True)]
    ids = _ids(t, k, g, 3)
    ids_d = torch.from_numpy(ids).to(dev)
    ws = [moe.experts_workspace(t, k, g, inner, dev) for _ in layers]
    ys = [torch.zeros(t, hidden, dtype=torch.bfloat16, device=dev) for _ in layers]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(5):
        for s, (x, sent, _, _), w, y in zip(streams, layers, ws, ys):
            with torch.cuda.stream(s):
                moe.experts(x, ids_d, None, *sent, y, w)
    torch.cuda.synchronize()
    for (x, _, v1, v2), y in zip(layers, ys):
        ref = _exact(x.double().cpu().numpy(), ids, np.ones((t, k)), v1, v2)
        np.testing.assert_array_equal(y.view(torch.int16).cpu().numpy().view(np.uint16), O.bf16_bits(ref))


def test_large_layer(dev):
    """Rows of 7168 and 2048, and an expert whose weights lie past 2^32 bytes: sampled
    tokens against the definition."""
    g, hidden, inner, t, k = 152, 7168, 2048, 6, 2            # the gate and up weights: 4.46e9 bytes
    _say(f"experts {(t, k, g, hidden, inner)}")
    b1 = torch.zeros(g, 2 * inner, hidden, dtype=torch.float8_e4m3fn, device=dev)
    b2 = torch.zeros(g, hidden, inner, dtype=torch.float8_e4m3fn, device=dev)
    sfb1 = torch.zeros(g, 2 * inner // 128, hidden // 128, device=dev)
    sfb2 = torch.zeros(g, hidden // 128, inner // 128, device=dev)
    v1, v2 = {}, {}
    for e in (0, g - 1):
        q1, s1, w1 = _weights(False, 1, 2 * inner, hidden, e, dev)
        q2, s2, w2 = _weights(False, 1, hidden, inner, e + 1, dev)
        b1[e], sfb1[e], b2[e], sfb2[e] = q1[0], s1[0], q2[0], s2[0]
        v1[e], v2[e] = w1[0], w2[0]
    ids = np.array([[0, g - 1], [g - 1, -1], [0, -1], [-1, -1], [g - 1, 0], [g - 1, g]], np.int32)
    x = torch.randn(t, hidden, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).to(dev)
    w = torch.rand(t, k, generator=torch.Generator().manual_seed(4)).to(dev)
    y = _run(x, ids, w, b1, sfb1, b2, sfb2, dev)
    two = np.where(ids == g - 1, 1, np.where(ids == 0, 0, -1))
    _check(y, x, two, w.cpu().numpy(), np.stack([v1[0], v1[g - 1]]), np.stack([v2[0], v2[g - 1]]))


def test_agrees_with_the_grouped_products(dev):
    """The same layer through dispatch, the grouped FP8 products, the activation and
    combine, whose operands are rounded to FP8 on the way: the same up to those roundings."""
    _say("experts against the grouped products")
    t, k, g, hidden, inner = 24, 3, 6, 512, 384
    b1, sfb1, v1 = _weights(False, g, 2 * inner, hidden, 1, dev)
    b2, sfb2, v2 = _weights(False, g, hidden, inner, 2, dev)
    ids, ids_d = _ids(t, k, g, 9), None
    ids_d = torch.from_numpy(ids).to(dev)
    x = torch.randn(t, hidden, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).to(dev)
    w = torch.rand(t, k, generator=torch.Generator().manual_seed(4)).to(dev)
    y = _run(x, ids, w, b1, sfb1, b2, sfb2, dev)
    plan = moe.Plan(t, k, g, "masked", t, hidden, dev)
    q, sfa = torch.zeros(plan.rows_shape, dtype=torch.float8_e4m3fn, device=dev), torch.zeros(plan.scale_shape, device=dev)
    moe.dispatch_fp8(plan, x, q, sfa, topk_ids=ids_d)
    gu = torch.zeros(g, t, 2 * inner, dtype=torch.bfloat16, device=dev)
    dg.m_grouped_fp8_gemm_nt_masked(q, sfa, b1, sfb1, gu, plan.group_rows)
    a, sfa2 = torch.zeros(g, t, inner, dtype=torch.float8_e4m3fn, device=dev), torch.zeros(g, inner // 128, dg.get_tma_aligned_size(t, 4), device=dev)
    moe.swiglu_fp8(gu, a, sfa2, rows=plan.group_rows, layout="masked")
    yp = torch.zeros(plan.rows_shape, dtype=torch.bfloat16, device=dev)
    dg.m_grouped_fp8_gemm_nt_masked(a, sfa2, b2, sfb2, yp, plan.group_rows)
    z = moe.combine(plan, yp, torch.empty_like(y), weights=w)
    # FP8 rounds x and a by 2^-4 at most each, by about 0.6 2^-4 / sqrt(3) in the 2-norm; x enters both g and u
    off = (y.double() - z.double()).norm() / y.double().norm()
    assert off < 3 * 2.0 ** -4, off.item()


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("case", LAYERS)
def test_few_compute_units_give_the_same_bits(dev, case, fp4):
    """As few compute units as make every workgroup take more rows of the weights, several
    tiles and several experts in turn."""
    _say(f"experts on few compute units {case} fp4={fp4}")
    t, k, g, hidden, inner = case
    g = min(g, 64)
    b1, sfb1, _ = _weights(fp4, g, 2 * inner, hidden, 1, dev)
    b2, sfb2, _ = _weights(fp4, g, hidden, inner, 2, dev)
    ids = _ids(t, k, g, t + g)
    x = torch.randn(t, hidden, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).to(dev)
    w = torch.rand(t, k, generator=torch.Generator().manual_seed(4)).to(dev)
    want = _run(x, ids, w, b1, sfb1, b2, sfb2, dev)
    for cus in (1, 3):
        dg.set_num_cus(cus)
        try:
            y = _run(x, ids, w, b1, sfb1, b2, sfb2, dev)
        finally:
            dg.set_num_cus(0)
        assert torch.equal(y.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("t", [2, 11, 31, 90])
def test_long_rows(dev, t, fp4):
    """Rows of 4224, the first length that takes 32 columns a workgroup on 256 compute units,
    with an odd number of blocks."""
    _say(f"experts, long rows t={t} fp4={fp4}")
    g, k, hidden, inner = 3, 2, 4224, 384
    b1, sfb1, v1 = _weights(fp4, g, 2 * inner, hidden, 1, dev)
    b2, sfb2, v2 = _weights(fp4, g, hidden, inner, 2, dev)
    ids = _ids(t, k, g, t)
    x = torch.randn(t, hidden, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).to(dev)
    w = torch.rand(t, k, generator=torch.Generator().manual_seed(4)).to(dev)
    _check(_run(x, ids, w, b1, sfb1, b2, sfb2, dev), x, ids, w.cpu().numpy(), v1, v2)


@pytest.mark.parametrize("fp4", [False, True])
def test_workgroups_that_share_columns_captured_and_on_two_streams(dev, fp4):
    """Short rows, whose sums meet in the workspace: replays of two graphs over one workspace
    and calls on two streams give the bits of calls made alone."""
    _say(f"experts, shared columns, fp4={fp4}")
    k, g, hidden, inner = 4, 30, 256, 1024
    b1, sfb1, _ = _weights(fp4, g, 2 * inner, hidden, 1, dev)
    b2, sfb2, _ = _weights(fp4, g, hidden, inner, 2, dev)
    sent = (b1, sfb1, b2, sfb2)
    ws = moe.experts_workspace(40, k, g, inner, dev)
    calls = []
    for t in (40, 7):
        x, w = torch.zeros(t, hidden, dtype=torch.bfloat16, device=dev), torch.ones(t, k, device=dev)
        ids, y = torch.zeros(t, k, dtype=torch.int32, device=dev), torch.zeros(t, hidden, dtype=torch.bfloat16, device=dev)
        moe.experts(x, ids, w, *sent, y, ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            moe.experts(x, ids, w, *sent, y, ws)
        calls.append((graph, x, ids, w, y))
    streams = [torch.cuda.Stream() for _ in calls]
    spaces = [moe.experts_workspace(40, k, g, inner, dev) for _ in calls]
    for seed in range(4):
        want = []
        for _, x, ids, w, _ in calls:
            x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(seed)))
            ids.copy_(torch.from_numpy(_ids(*ids.shape, g, seed)))
            w.uniform_()
            want.append(_run(x, ids.cpu().numpy(), w, *sent, dev).view(torch.int16))
        for (graph, *_, y), ref in zip(calls, want):
            y.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y.view(torch.int16), ref)
        outs = [torch.zeros_like(c[4]) for c in calls]
        torch.cuda.synchronize()
        for _ in range(3):
            for s, space, (_, x, ids, w, _), out in zip(streams, spaces, calls, outs):
                with torch.cuda.stream(s):
                    moe.experts(x, ids, w, *sent, out, space)
        torch.cuda.synchronize()
        for out, ref in zip(outs, want):
            assert torch.equal(out.view(torch.int16), ref)
