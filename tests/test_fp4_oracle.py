"""Pins of the FP4 oracle (CPU): the codes against an exact search over every
level, the scale against exact rationals, words and packing by hand."""

from fractions import Fraction

import numpy as np
import pytest
import torch

from moe_grouped_gemm_amd import synth
from oracle import dg_oracle as O
from oracle import fp4_oracle as F


def _bf16(bits):
    return O.bf16_bits_to_f64(np.asarray(bits, np.uint16))


def test_scale_is_the_smallest_power_of_two_that_does_not_saturate():
    tops = np.concatenate([_bf16(np.arange(0, 0x7F80, 37)), _bf16([0x7F7F, 1, 0x40, 0x3FC0, 0x3FC1, 0x3FBF])])
    for top, code in zip(tops, F.scale_codes(np.repeat(tops[:, None], 32, 1))[:, 0]):
        scale = Fraction(2) ** (int(code) - 127)
        assert Fraction(top) <= 6 * scale
        assert code == 0 or Fraction(top) > 3 * scale


def test_codes_are_the_nearest_level_and_ties_even():
    a = np.linspace(0, 6, 24 * 32 + 1)[: 24 * 32]
    got = F.codes(a.reshape(-1, 32), np.full((24, 1), 127, np.uint8)).reshape(-1)
    for v, c in zip(a, got):
        dist = [abs(Fraction(v) - Fraction(level)) for level in F.LEVELS]
        best = [i for i, d in enumerate(dist) if d == min(dist)]
        assert c in best and (len(best) == 1 or c % 2 == 0)
    for tie, code in ((0.25, 0), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6)):
        assert F.codes(np.full((1, 32), tie), np.full((1, 1), 127, np.uint8))[0, 0] == code
        assert F.codes(np.full((1, 32), -tie), np.full((1, 1), 127, np.uint8))[0, 0] == code + 8


def test_blocks_that_are_not_finite():
    x = np.ones((4, 64))
    x[0, 3], x[1, 40], x[2, 0], x[3, 63] = np.nan, np.inf, -np.inf, 3.5e38
    np.testing.assert_array_equal(F.scale_codes(x), [[255, 125], [125, 255], [255, 125], [125, 255]])
    v = F.values(*F.quantize(np.tile(x, 2)))
    assert np.isnan(v[0, :32]).all() and (v[0, 32:64] == 1).all() and np.isnan(v[3, 32:64]).all()


def test_words_and_packing_by_hand():
    s = np.array([[1, 2, 3, 4, 5, 6, 7, 8], [9, 10, 11, 12, 13, 14, 15, 255]], np.uint8)
    np.testing.assert_array_equal(F.words(s), [[0x04030201, 0x0C0B0A09], [0x08070605, 0xFF0F0E0D]])
    np.testing.assert_array_equal(F.pack(np.array([1, 15, 8, 2], np.uint8)), [0xF1, 0x28])
    packed, sf = np.zeros((1, 64), np.uint8), np.array([[0x80_7F_7E_81]], np.uint32)
    packed[0, 0], packed[0, 16], packed[0, 32], packed[0, 48] = 0x07, 0x70, 0x0F, 0x21
    v = F.values(packed, sf)[0]
    assert (v[0], v[32], v[33], v[64], v[96], v[97]) == (24.0, 0.0, 3.0, -6.0, 1.0, 2.0)


def test_values_read_back_what_was_quantised():
    x = np.random.default_rng(0).choice(F.LEVELS, (5, 256)) * np.repeat(2.0 ** np.arange(-4, 4), 32)[None]
    x[:, ::32] = 6.0 * 2.0 ** np.arange(-4, 4)     # so that every block has its scale
    np.testing.assert_array_equal(F.values(*F.quantize(x)), x)


def test_agrees_with_the_w4a8_operand():
    """synth's quantiser of the FP8 x FP4 GEMMs' weights makes the same codes and scales."""
    x = torch.randn(7, 256, generator=torch.Generator().manual_seed(3))
    packed, sfb = synth.quantize_rhs_e2m1(x)
    mine, sf = F.quantize(x.double().numpy())
    # (synth leaves out the sign of what rounds to zero)
    np.testing.assert_array_equal(O.e2m1_decode_table()[O.unpack_e2m1(mine)],
                                  O.e2m1_decode_table()[O.unpack_e2m1(packed.numpy())])
    np.testing.assert_array_equal(F.values(mine, sf), O.dequant_rhs_e2m1(packed.numpy(), sfb.numpy()))


def test_experts_by_hand():
    """One expert of one inner value, all numbers small: y = w * W2 silu(g) u."""
    x = np.array([[2.0, -1.0], [0.0, 3.0]])
    w1 = np.array([[[1.0, 0.5], [0.0, 2.0]], [[0.0, 1.0], [1.0, 0.0]]])
    w2 = np.array([[[3.0], [-1.0]], [[0.5], [2.0]]])
    ids, w = np.array([[0, 5], [1, -1]]), np.array([[0.25, 9.0], [4.0, 9.0]])
    silu = lambda v: v / (1 + np.exp(-v))  # noqa: E731
    y, act_mag, mag, top = F.experts(x, ids, w, w1, w2)
    a0 = silu(1.5) * -2.0
    np.testing.assert_allclose(y[0], 0.25 * a0 * np.array([3.0, -1.0]), rtol=1e-15)
    np.testing.assert_allclose(y[1], 4.0 * silu(3.0) * 0.0 * np.array([0.5, 2.0]), atol=0)
    assert (act_mag >= np.abs(y)).all() and (mag >= act_mag).all() and top == 3.0


@pytest.mark.parametrize("mistake", ["floor", "nibbles", "words", "ties"])
def test_planted_mistakes_are_seen(mistake, monkeypatch):
    x = np.random.default_rng(1).normal(size=(3, 256))
    x[0, :8] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0]
    good = F.values(*F.quantize(x))
    if mistake == "floor":
        real = F.scale_codes
        monkeypatch.setattr(F, "scale_codes", lambda v: real(v) - 1)
    elif mistake == "nibbles":
        monkeypatch.setattr(F, "pack", lambda c: c[..., 1::2] | c[..., 0::2] << 4)
    elif mistake == "words":
        real_w = F.words
        monkeypatch.setattr(F, "words", lambda s: real_w(s[..., ::-1]))
    else:
        monkeypatch.setattr(F, "LEVELS", np.nextafter(F.LEVELS, 9.0))
    assert (F.values(*F.quantize(x)) != good).any()
