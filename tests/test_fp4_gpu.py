"""GPU parity of the FP4 quantiser and products against their float64 definitions
(oracle/fp4_oracle.py). The quantiser and what reads it back are compared bit for
bit; a product's element as parity.py derives it, and bit for bit where sums of
whole numbers below 2^24 leave nothing to round but the result."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from moe_grouped_gemm_amd import dg, synth
from oracle import dg_oracle as O
from oracle import fp4_oracle as F
from parity import check_close, check_untouched

pytestmark = pytest.mark.gpu

SENTINEL_WORD = 0x5A5A5A5A


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dg.lib()
    return torch.device("cuda:0")


def _say(msg):
    print(msg, flush=True)


def _bits(t):
    return t.detach().view({2: torch.int16, 1: torch.uint8, 4: torch.int32}[t.element_size()]).cpu().numpy()


def _operand(lead, rows, k, dev):
    """Room for an operand, every byte and word set to something else."""
    q = torch.full((*lead, rows, k // 2), 0xA5, dtype=torch.uint8, device=dev)
    sf = torch.full((*lead, k // 128, synth.tma_aligned_size(rows)), SENTINEL_WORD, dtype=torch.int32, device=dev)
    return q, sf


# ---------------------------------------------------------------------------
# Rows to codes and back
# ---------------------------------------------------------------------------

SHAPES = [(1, 128), (3, 256), (67, 7168), (33, 640), (1027, 512), (4, 3, 128), (5, 31, 384), (2, 64, 1152), (1, 1, 2048)]


def _rows(shape, dtype, special, seed):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=gen) * 3
    x = x * torch.exp2(torch.randint(-20, 20, (*shape[:-1], shape[-1] // 32), generator=gen).float()
                       ).repeat_interleave(32, -1)
    x = x.to(dtype)
    if special:
        b = x.view(-1, 32)
        n = b.shape[0]
        b[0] = 0.0
        b[n // 2, 5] = float("nan")
        b[n // 3, 7] = float("inf")
        b[n // 4, 31] = -float("inf")
        b[n - 1] = torch.tensor([0.25, -0.25, 0.75, 1.25, -1.75, 2.5, 3.5, -5.0, 6.0] + [0.0] * 23)     # ties
        if n > 8:
            b[n // 5] *= 2.0 ** -126                                    # subnormal scales, subnormal values
            b[n // 6] = torch.finfo(dtype).max
            b[n // 7] = torch.finfo(dtype).tiny / 64
            b[n // 8, :] = torch.tensor([1.5 + (0.0078125 if dtype is torch.bfloat16 else 2.0 ** -22)] + [-0.0] * 31)
            b[n // 9, :] = torch.tensor([1.5] + [-1e-9] * 31)
    return x


@pytest.mark.parametrize("special", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES)
def test_quantize_and_back(dev, shape, dtype, special):
    _say(f"quantize {shape} {dtype} special={special}")
    x = _rows(shape, dtype, special, sum(shape))
    q, sf = _operand(shape[:-2], *shape[-2:], dev)
    dg.quantize_fp4(x.to(dev), q, sf)
    want_q, want_sf = F.quantize(x.double().numpy())
    rows = shape[-2]
    np.testing.assert_array_equal(_bits(sf).astype(np.uint32)[..., :rows], want_sf)
    np.testing.assert_array_equal(_bits(q), want_q)
    assert (_bits(sf)[..., rows:] == SENTINEL_WORD).all()
    back = torch.full(shape, -7.0, dtype=torch.bfloat16, device=dev)
    dg.dequantize_fp4(q, sf, back)
    # values from 1.75 2^127 on are nearest to 4 2^126 = 2^128, which BF16 has only as infinity
    want = torch.from_numpy(F.values(want_q, want_sf)).to(torch.bfloat16)
    np.testing.assert_array_equal(back.double().cpu().numpy(), want.double().numpy())


def test_read_back_every_code_under_every_scale(dev):
    """All 16 codes under all 256 scales; past BF16's largest value: infinite."""
    _say("dequantize every code and scale")
    s = np.arange(256, dtype=np.uint8).reshape(64, 4)
    packed = np.tile(np.array([0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE], np.uint8), (64, 8))
    sf = F.words(s).astype(np.uint32)
    out = torch.zeros(64, 128, dtype=torch.bfloat16, device=dev)
    dg.dequantize_fp4(torch.from_numpy(packed).to(dev), torch.from_numpy(sf.view(np.int32)).to(dev), out)
    want = torch.from_numpy(F.values(packed, sf)).to(torch.bfloat16).double().numpy()
    np.testing.assert_array_equal(out.double().cpu().numpy(), want)


def test_empty_rows(dev):
    _say("no rows")
    for shape in ((0, 256), (0, 4, 256), (3, 0, 256)):
        x = torch.zeros(shape, dtype=torch.bfloat16, device=dev)
        q, sf = _operand(shape[:-2], *shape[-2:], dev)
        dg.quantize_fp4(x, q, sf)
        dg.dequantize_fp4(q, sf, x)


# ---------------------------------------------------------------------------
# Products
# ---------------------------------------------------------------------------

def _codes(seed, lead, rows, k, whole=False, spread=7):
    """Random codes and scales on the host: (packed, words padded to the aligned rows)."""
    r = np.random.default_rng(seed)
    if whole:                                   # whole numbers up to 12, one scale for all
        code = r.choice(np.array([0, 2, 4, 5, 10, 12, 13], np.uint8), (*lead, rows, k))
        s = np.full((*lead, rows, k // 32), 127, np.uint8) + r.integers(0, 2, (*lead, rows, k // 32), dtype=np.uint8)
    else:
        code = r.integers(0, 16, (*lead, rows, k), dtype=np.uint8)
        s = r.integers(127 - spread, 127 + spread, (*lead, rows, k // 32)).astype(np.uint8)
    sf = np.full((*lead, k // 128, synth.tma_aligned_size(rows)), 0xFFFFFFFF, np.uint32)     # NaN scales past the rows
    sf[..., :rows] = F.words(s)
    return F.pack(code), sf


def _put(dev, *arrays):
    return [torch.from_numpy(np.ascontiguousarray(a if a.dtype == np.uint8 else a.view(np.int32))).to(dev)
            for a in arrays]


def _out(*shape):
    return torch.full(shape, -1, dtype=torch.int16, device="cuda").view(torch.bfloat16)


def _check(got_bits, a, sfa, b, sfb, k, whole, what):
    """One group's rows: got uint16 [rows, n]."""
    if got_bits.size == 0:
        return
    ref, mag = F.gemm(a, sfa, b, sfb)
    if whole:
        assert np.abs(ref).max() < 2 ** 24 and mag.max() < 2 ** 24
        np.testing.assert_array_equal(got_bits, O.bf16_bits(ref), what)
    else:
        check_close(got_bits, ref, what, mag, k)


# Few tiles, more, and as many as take the largest ones.
DENSE = [(1, 128, 128), (15, 128, 384), (130, 384, 256), (257, 256, 512), (300, 640, 1152), (513, 128, 2048), (64, 512, 7168),
         (1, 49280, 128), (15, 49280, 640), (257, 9984, 384), (513, 5632, 256), (64, 49280, 1152), (700, 4608, 2048),
         (1, 65792, 128), (15, 65792, 640), (257, 22272, 384), (513, 13312, 256), (64, 65792, 1152), (700, 11008, 640)]


@pytest.mark.parametrize("whole", [False, True])
@pytest.mark.parametrize("m,n,k", DENSE)
def test_dense(dev, m, n, k, whole):
    _say(f"dense {m}x{n}x{k} whole={whole}")
    a, sfa = _codes(m, (), m, k, whole)
    b, sfb = _codes(n + 1, (), n, k, whole)
    d = _out(m, n)
    dg.fp4_gemm_nt(*_put(dev, a, sfa, b, sfb), d)
    _check(_bits(d).view(np.uint16), a, sfa, b, sfb, k, whole, f"dense {m}x{n}x{k}")


def test_dense_many_tiles(dev):
    """More tiles than one round of workgroups, checked at sampled rows and columns."""
    m, n, k = 4097, 7168, 640
    _say(f"dense {m}x{n}x{k}")
    a, sfa = _codes(1, (), m, k)
    b, sfb = _codes(2, (), n, k)
    d = _out(m, n)
    dg.fp4_gemm_nt(*_put(dev, a, sfa, b, sfb), d)
    got = _bits(d).view(np.uint16)
    r = np.random.default_rng(0)
    rows = np.unique(np.r_[0, 127, 128, 255, 256, m - 1, r.integers(0, m, 200)])
    cols = np.unique(np.r_[0, 63, 64, 255, 256, n - 1, r.integers(0, n, 200)])
    ref, mag = F.gemm(a[rows], sfa[:, rows], b[cols], sfb[:, cols])
    check_close(got[np.ix_(rows, cols)], ref, "sampled", mag, k)


@pytest.mark.parametrize("n", [256, 24832, 65792])
@pytest.mark.parametrize("k", [128, 896])
def test_nan_scales_stay_in_their_rows(dev, k, n):
    _say(f"NaN scales, K {k}, N {n}")
    m = 70
    a, sfa = _codes(5, (), m, k)
    b, sfb = _codes(6, (), n, k)
    sfa[k // 128 - 1, 3] |= 0xFF00                   # the second block of the last 128 values
    sfb[0, 200] |= 0xFF000000
    d = _out(m, n)
    dg.fp4_gemm_nt(*_put(dev, a, sfa, b, sfb), d)
    nan = np.isnan(O.bf16_bits_to_f64(_bits(d).view(np.uint16)))
    want = np.zeros((m, n), bool)
    want[3], want[:, 200] = True, True
    np.testing.assert_array_equal(nan, want)


@pytest.mark.parametrize("n", [128, 49280, 65792])
def test_scales_at_their_ends(dev, n):
    """2^-127 times 2^127, and sums below BF16's smallest."""
    _say(f"extreme scales, N {n}")
    m, k = 16, 384
    a, sfa = _codes(7, (), m, k, True)
    b, sfb = _codes(8, (), n, k, True)
    ones = sfa.copy(), sfb.copy()
    ones[0][:, :m], ones[1][:, :n] = 0x7F7F7F7F, 0x7F7F7F7F
    ref, _ = F.gemm(a, ones[0], b, ones[1])
    for lo, hi, shift in ((0x00000000, 0xFEFEFEFE, 0), (0xFEFEFEFE, 0x00000000, 0), (0x00000000, 0x00000000, -254)):
        sfa[:, :m], sfb[:, :n] = lo, hi
        d = _out(m, n)
        dg.fp4_gemm_nt(*_put(dev, a, sfa, b, sfb), d)
        np.testing.assert_array_equal(O.bf16_bits_to_f64(_bits(d).view(np.uint16)), O.bf16_round(ref) * (shift == 0))


def _layout(counts, m):
    ids = np.full(m, -1, np.int32)
    at = 0
    for g, c in enumerate(counts):
        ids[at:at + c] = g
        at += -(-c // 128) * 128
    return ids


@pytest.mark.parametrize("whole", [False, True])
@pytest.mark.parametrize("counts,n,k", [([5, 0, 300, 128, 1], 256, 384), ([700], 128, 128), ([127, 129, 640], 640, 1024),
                                        ([5, 0, 300, 128, 1], 3584, 384), ([700], 4992, 128), ([127, 129, 640], 2816, 1024),
                                        ([5, 0, 300, 128, 1], 9472, 384), ([700], 9472, 128), ([127, 129, 640], 7424, 512)])
def test_contiguous(dev, counts, n, k, whole):
    _say(f"contiguous {counts} n={n} k={k} whole={whole}")
    m, g = sum(-(-c // 128) * 128 for c in counts) + 128, len(counts)
    ids = _layout(counts, m)
    a, sfa = _codes(3, (), m, k, whole)
    sfa[:, :m][:, ids < 0] = 0xFFFFFFFF              # rows of no group do not reach the others
    b, sfb = _codes(4, (g,), n, k, whole)
    d = _out(m, n)
    dg.m_grouped_fp4_gemm_nt_contiguous(*_put(dev, a, sfa, b, sfb), d, torch.from_numpy(ids).to(dev))
    got = _bits(d).view(np.uint16)
    check_untouched(got[ids < 0], "padding")
    for e in range(g):
        rows = ids == e
        _check(got[rows], a[rows], sfa[:, :m][:, rows], b[e], sfb[e], k, whole, f"group {e}")


@pytest.mark.parametrize("n", [128, 4992, 13312])
def test_contiguous_ids_that_change_inside_blocks(dev, n):
    """The row rule of the layout: a 128-row block is its first row's group's."""
    _say(f"contiguous, ids that change inside blocks, n={n}")
    m, k, g = 640, 256, 3
    ids = np.random.default_rng(0).integers(-1, 5, m).astype(np.int32)
    ids[0], ids[128], ids[256], ids[384], ids[512] = 1, -1, 7, 2, 0
    a, sfa = _codes(3, (), m, k, True)
    b, sfb = _codes(4, (g,), n, k, True)
    d = _out(m, n)
    dg.m_grouped_fp4_gemm_nt_contiguous(*_put(dev, a, sfa, b, sfb), d, torch.from_numpy(ids).to(dev))
    got, owner = _bits(d).view(np.uint16), O.contiguous_row_groups(ids, g)
    check_untouched(got[owner < 0], "rows of no group")
    for e in range(g):
        _check(got[owner == e], a[owner == e], sfa[:, owner == e], b[e], sfb[e], k, True, f"group {e}")


@pytest.mark.parametrize("whole", [False, True])
@pytest.mark.parametrize("counts,max_m,n,k", [([5, 0, 64, 63], 64, 128, 384), ([300, -2, 17, 999, 129], 300, 384, 256),
                                              ([1] * 40, 8, 256, 1152), ([0, 0], 16, 128, 128), ([97, 160], 257, 128, 512),
                                              ([300, -2, 17, 999, 129], 300, 2048, 256), ([1, 8] * 20, 8, 1280, 1152),
                                              ([0, 0], 16, 24704, 128), ([97, 160], 257, 4992, 512),
                                              ([300, -2, 17, 999, 129], 300, 4608, 256), ([97, 160], 257, 11008, 512),
                                              ([128, 1] * 20, 128, 1792, 384)])
def test_masked(dev, counts, max_m, n, k, whole):
    _say(f"masked {counts} of {max_m} n={n} k={k} whole={whole}")
    g = len(counts)
    a, sfa = _codes(5, (g,), max_m, k, whole)
    for e, c in enumerate(counts):
        sfa[e, :, max(c, 0):] = 0xFFFFFFFF
    b, sfb = _codes(6, (g,), n, k, whole)
    d = _out(g, max_m, n)
    rows = torch.tensor(counts, dtype=torch.int32, device=dev)
    dg.m_grouped_fp4_gemm_nt_masked(*_put(dev, a, sfa, b, sfb), d, rows)
    got = _bits(d).view(np.uint16)
    for e, c in enumerate(counts):
        c = min(max(c, 0), max_m)
        check_untouched(got[e, c:], f"group {e}")
        _check(got[e, :c], a[e, :c], sfa[e][:, :c], b[e], sfb[e], k, whole, f"group {e}")


@pytest.mark.parametrize("whole", [False, True])
@pytest.mark.parametrize("counts,m,n,k", [([3, 0, 200, 31], 240, 256, 384), ([5, -4, 90, 400, 7], 260, 128, 640),
                                          ([1, 2, 3] * 20, 120, 128, 256), ([513], 513, 384, 128),
                                          ([5, -4, 90, 400, 7], 260, 4992, 640), ([1, 2, 3] * 20, 120, 896, 256),
                                          ([513], 513, 4992, 128), ([5, -4, 90, 400, 7], 260, 8448, 640),
                                          ([1, 2, 3] * 20, 120, 1280, 256), ([513], 513, 11008, 128)])
def test_nopad(dev, counts, m, n, k, whole):
    _say(f"nopad {counts} of {m} n={n} k={k} whole={whole}")
    g = len(counts)
    a, sfa = _codes(7, (), m, k, whole)
    ends = np.minimum(np.cumsum(np.maximum(counts, 0)), m)
    sfa[:, ends[-1]:] = 0xFFFFFFFF
    b, sfb = _codes(8, (g,), n, k, whole)
    d = _out(m, n)
    dg.m_grouped_fp4_gemm_nt_nopad(*_put(dev, a, sfa, b, sfb), d, torch.tensor(counts, dtype=torch.int32, device=dev))
    got = _bits(d).view(np.uint16)
    check_untouched(got[ends[-1]:], "rows of no group")
    for e, (lo, hi) in enumerate(zip(np.r_[0, ends], ends)):
        _check(got[lo:hi], a[lo:hi], sfa[:, lo:hi], b[e], sfb[e], k, whole, f"group {e}")


@pytest.mark.parametrize("whole", [False, True])
@pytest.mark.parametrize("m,g,n,k", [(1, 2048, 128, 384), (8, 128, 2048, 512), (8, 128, 2048, 7168), (3, 40, 8448, 256),
                                     (14, 60, 4096, 384), (40, 256, 4096, 256), (100, 300, 2560, 128), (300, 200, 512, 384)])
def test_nopad_of_more_groups_than_most_have_rows(dev, m, g, n, k, whole):
    """A step of few tokens over many experts: most groups have none, in runs and by turns."""
    _say(f"nopad, {m} rows of {g} groups, n={n} k={k} whole={whole}")
    r = np.random.default_rng(m + g)
    counts = np.bincount(r.choice(g, m), minlength=g).astype(np.int32)
    if m < g:                                        # as many groups as rows, the last one among them
        counts[:] = 0
        counts[np.r_[r.permutation(g - 1)[:m - 1], g - 1]] = 1
    a, sfa = _codes(7, (), m, k, whole)
    b, sfb = _codes(8, (min(g, 3),), n, k, whole)
    pick = np.arange(g) % len(b)                     # groups share three matrices' values
    ad, sfad, bd, sfbd = _put(dev, a, sfa, b, sfb)
    every = torch.from_numpy(pick).to(dev)
    d = _out(m, n)
    dg.m_grouped_fp4_gemm_nt_nopad(ad, sfad, bd[every].contiguous(), sfbd[every].contiguous(), d, torch.from_numpy(counts).to(dev))
    got = _bits(d).view(np.uint16)
    owner = np.repeat(np.arange(g), counts)
    for e in range(len(b)):
        mine = pick[owner] == e
        _check(got[mine], a[mine], sfa[:, :m][:, mine], b[e], sfb[e], k, whole, f"matrix {e}")


def test_no_rows_no_groups(dev):
    _say("empty products")
    a, sfa = _codes(1, (), 0, 256)
    b, sfb = _codes(2, (), 128, 256)
    dg.fp4_gemm_nt(*_put(dev, a, sfa, b, sfb), _out(0, 128))
    gb, gsfb = b[None], sfb[None]
    dg.m_grouped_fp4_gemm_nt_contiguous(*_put(dev, a, sfa, gb, gsfb), _out(0, 128), torch.zeros(0, dtype=torch.int32, device=dev))
    dg.m_grouped_fp4_gemm_nt_nopad(*_put(dev, a, sfa, gb, gsfb), _out(0, 128), torch.zeros(1, dtype=torch.int32, device=dev))
    a, sfa = _codes(1, (0,), 4, 256)
    gb, gsfb = _codes(2, (0,), 128, 256)
    dg.m_grouped_fp4_gemm_nt_masked(*_put(dev, a, sfa, gb, gsfb), _out(0, 4, 128), torch.zeros(0, dtype=torch.int32, device=dev))


def test_a_captured_product_reads_its_counts_on_the_device(dev):
    """Quantiser and masked product in one graph, replayed with other rows and counts."""
    _say("graph of a quantiser and a masked product")
    g, max_m, n, k = 3, 70, 256, 384
    x = torch.zeros(g, max_m, k, dtype=torch.bfloat16, device=dev)
    q, sf = _operand((g,), max_m, k, dev)
    b, sfb = _codes(6, (g,), n, k)
    bd, sfbd = _put(dev, b, sfb)
    d = _out(g, max_m, n)
    rows = torch.zeros(g, dtype=torch.int32, device=dev)

    def both():
        dg.quantize_fp4(x, q, sf)
        dg.m_grouped_fp4_gemm_nt_masked(q, sf, bd, sfbd, d, rows)

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for seed, counts in ((1, [70, 0, 3]), (2, [1, 69, 12]), (3, [0, 0, 70])):
        x.copy_(torch.randn(g, max_m, k, generator=torch.Generator(device=dev).manual_seed(seed), device=dev))
        rows.copy_(torch.tensor(counts, dtype=torch.int32))
        d.view(torch.int16).fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        a, sfa = F.quantize(x.double().cpu().numpy())
        got = _bits(d).view(np.uint16)
        for e, c in enumerate(counts):
            check_untouched(got[e, c:], f"group {e}")
            _check(got[e, :c], a[e, :c], sfa[e][:, :c], b[e], sfb[e], k, False, f"group {e}")


def test_two_streams_at_once(dev):
    _say("products on two streams")
    m, n, k = 500, 384, 1024
    ops = [(*_codes(s, (), m, k), *_codes(s + 9, (), n, k)) for s in (1, 2)]
    on = [_put(dev, *o) for o in ops]
    outs = [_out(m, n) for _ in ops]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ops]
    for _ in range(3):
        for s, o, d in zip(streams, on, outs):
            with torch.cuda.stream(s):
                dg.fp4_gemm_nt(*o, d)
    torch.cuda.synchronize()
    for o, d in zip(ops, outs):
        _check(_bits(d).view(np.uint16), *o, k, False, "stream")


@pytest.mark.parametrize("n", [640, 2560, 6912])
@pytest.mark.parametrize("k", [128, 256, 384, 640])
def test_few_workgroups_give_the_same_bits(dev, k, n):
    """One, three and eight workgroups for all tiles: tiles of one, two and three steps that
    follow one another in a workgroup's pipeline, valid rows that end next to the copies of
    the K loop."""
    _say(f"few workgroups, n={n} k={k}")
    g = 5
    b, sfb = _codes(4, (g,), n, k)
    flat, sf_flat = _codes(5, (), 1280, k)
    many, sf_many = _codes(6, (g,), 300, k)
    bd, sfbd, ad, sfad, md, sfmd = _put(dev, b, sfb, flat, sf_flat, many, sf_many)
    ids = torch.from_numpy(_layout([200, 0, 129, 512, 100], 1280)).to(dev)
    counts = torch.tensor([64, 65, 300, 0, 193], dtype=torch.int32, device=dev)

    def calls():
        d = [_out(1280, n), _out(1280, n), _out(g, 300, n), _out(1280, n)]
        dg.fp4_gemm_nt(ad, sfad, bd[1], sfbd[1], d[0])
        dg.m_grouped_fp4_gemm_nt_contiguous(ad, sfad, bd, sfbd, d[1], ids)
        dg.m_grouped_fp4_gemm_nt_masked(md, sfmd, bd, sfbd, d[2], counts)
        dg.m_grouped_fp4_gemm_nt_nopad(ad, sfad, bd, sfbd, d[3], counts)
        return [_bits(v) for v in d]

    want = calls()
    _check(want[0].view(np.uint16), flat, sf_flat, b[1], sfb[1], k, False, "dense")
    for cus in (1, 3, 8):
        dg.set_num_cus(cus)
        try:
            got = calls()
        finally:
            dg.set_num_cus(0)
        for what, x, y in zip(("dense", "contiguous", "masked", "no padding"), got, want):
            np.testing.assert_array_equal(x, y, f"{what}, {cus} workgroups")
