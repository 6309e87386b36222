"""Pins of the oracle of the quantised cache and of the log probabilities: worked numbers and laws."""
import math

import numpy as np
import pytest

from oracle import quant_oracle as Q


def test_scales_are_floats_of_five_and_three_bits():
    s = Q.scale_values()
    assert s[0] == 0 and s[1] == 2.0 ** -17 and s[7] == 7 * 2.0 ** -17 and s[8] == 2.0 ** -14
    assert s[120] == 1.0 and s[121] == 1.125 and s[127] == 1.875 and s[128] == 2.0
    assert all(np.diff(s[:0xF8]) > 0)
    assert Q.top_byte(4) == 0xDF and s[0xDF] == 7680 and Q.top_byte(8) == 0xC0 and s[0xC0] == 512


@pytest.mark.parametrize("bits", [4, 8])
def test_the_least_scale_that_reaches_the_largest(bits):
    most, s = Q.most_of(bits), Q.scale_values()
    for top in (1.0, 0.37, most * 1.125, np.nextafter(most * 1.125, 2e9), 1e-7, 0.0, 3.3e4):
        x = np.zeros(16)
        x[5] = -top
        codes, byte, bad = Q.quantise(x, bits)
        b = int(byte[0])
        assert s[b] * most >= top and (b == 0 or s[b - 1] * most < top) and not bad
        assert abs(Q.values(codes, byte) - x).max() <= s[b] / 2


def test_codes_round_to_nearest_ties_to_even():
    x = np.zeros(16)
    x[:6] = [7, 0.5, 1.5, -2.5, 2.5000001, -7]          # scale 1 in 4 bits
    codes, byte, _ = Q.quantise(x, 4)
    assert byte[0] == 120 and codes[:6].tolist() == [7, 0, 2, -2, 3, -7]


def test_what_does_not_fit():
    x = np.zeros((2, 16))
    x[0, 0], x[1, 3] = np.nan, -np.inf
    codes, byte, bad = Q.quantise(x, 4)
    assert bad and codes[0, 0] == 0 and codes[1, 3] == -7 and byte[1, 0] == 0xDF


@pytest.mark.parametrize("bits,dim,ps", [(4, 128, 16), (4, 80, 5), (8, 64, 3), (8, 256, 20)])
def test_bytes_and_back(bits, dim, ps):
    g = np.random.default_rng(dim)
    code, scale, size = Q.sizes(ps, dim, bits)
    assert size % 16 == 0 and size >= ps * (dim * bits // 8 + dim // 16) and scale % 4 == 0
    head, want = np.full(size, 0xAA, np.uint8), []
    for t in range(ps):
        codes, byte, _ = Q.quantise(g.normal(size=dim), bits)
        Q.put(head, t, codes, byte, ps, bits)
        want.append(Q.values(codes, byte))
    for t in range(ps):
        assert (Q.get(head, t, ps, dim, bits) == want[t]).all()
    used = ps * (code + scale)
    assert (head[used:] == 0xAA).all()


def test_a_word_of_four_bit_codes():
    head = np.zeros(Q.sizes(1, 16, 4)[2], np.uint8)
    codes = np.array([-8, -7, -6, -5, -4, -3, -2, -1] + [0] * 8) + 0
    Q.put(head, 0, codes, np.array([120]), 1, 4)
    # dims 0, 2, 4, 6 in the low half, 1, 3, 5, 7 in the high one
    assert head[:4].view(np.uint32)[0] == 0x75316420 and head[8] == 120


def test_attention_of_one_and_of_no_key():
    g = np.random.default_rng(0)
    q, k, v = g.normal(size=(2, 4, 8)), g.normal(size=(3, 2, 8)), g.normal(size=(3, 2, 8))
    out, lse, mean, _ = Q.attention(q, k, v, [0, 1], 0.5)
    assert (out[0] == 0).all() and (lse[0] == -np.inf).all()
    assert np.allclose(out[1, 1], v[0, 0]) and np.allclose(out[1, 3], v[0, 1])
    assert np.isclose(lse[1, 2], 0.5 * q[1, 2] @ k[0, 1]) and np.allclose(mean[1, 0], abs(v[0, 0]))


def test_logprobs_of_a_worked_row():
    row = [math.log(4.0), -np.inf, math.log(2.0), math.log(2.0), np.nan]
    lp, h, rank, ids, tops = Q.logprobs(row, 3, 1.0, 5)
    assert np.isclose(lp, math.log(0.25)) and np.isclose(h, 1.5 * math.log(2)) and rank == 3
    assert ids == [0, 2, 3, -1, -1] and np.allclose(tops[:3], np.log([0.5, 0.25, 0.25]))
    assert tops[3:] == [-np.inf] * 2
    # twice the temperature: square roots
    assert np.isclose(Q.logprobs(row, 0, 2.0, 0)[0], math.log(2 / (2 + 2 * math.sqrt(2))))
    assert Q.logprobs(row, 2, 0.0, 2) == (-np.inf, 0.0, 2, [0, 2], [0.0, -np.inf])
    assert Q.logprobs(row, 4, 1.0, 0)[:3] == (-np.inf, pytest.approx(1.5 * math.log(2)), 5)
    assert Q.logprobs(row, -1, 1.0, 2) == (0.0, 0.0, 0, [-1, -1], [0.0, 0.0])
    assert Q.logprobs([np.nan, -np.inf], 1, 1.0, 1) == (-np.inf, 0.0, 2, [-1], [-np.inf])
