"""Pins of the rotary and 4-bit cache oracle (oracle/kv4.py) against closed
forms and hand-worked blocks. CPU only."""
from fractions import Fraction

import numpy as np
import pytest

import oracle.kv4 as o


def test_rope_quarter_turns():
    # freq 1 at position 0 leaves a head alone; an angle of pi / 2 (fp32 pi / 2
    # times 1) turns (1, 0) into (0, 1) to that frequency's own rounding
    x = np.arange(1.0, 9.0).reshape(1, 1, 8)
    assert np.array_equal(o.rope(x, [0], [1.0, 0.5]), x)
    f = np.float32(np.pi / 2)
    half = o.rope(np.array([[[1.0, 0.0, 0.0, 0.0, 7.0]]]), [1], [f, f])[0, 0]
    assert np.allclose(half, [0, 0, 1, 0, 7], atol=1e-7)
    inter = o.rope(np.array([[[1.0, 0.0, 0.0, 1.0, 7.0]]]), [1], [f, f], interleaved=True)[0, 0]
    assert np.allclose(inter, [0, 1, -1, 0, 7], atol=1e-7)


def test_rope_is_a_rotation_and_scores_depend_on_the_distance():
    rng = np.random.default_rng(1)
    f = (10000.0 ** (-np.arange(0, 16, 2) / 16)).astype(np.float32)
    q, k = rng.standard_normal((2, 1, 1, 20))
    for inter in (False, True):
        a = o.rope(q, [1000], f, inter)[0, 0] @ o.rope(k, [990], f, inter)[0, 0]
        b = o.rope(q, [17], f, inter)[0, 0] @ o.rope(k, [7], f, inter)[0, 0]
        assert abs(a - b) < 1e-10
        assert np.isclose(np.linalg.norm(o.rope(q, [5], f, inter)), np.linalg.norm(q))
        assert np.allclose(o.rope(q, [5], f, inter, mscale=2.0)[..., :16], 2 * o.rope(q, [5], f, inter)[..., :16])


def test_norm_closed_form():
    x = np.array([3.0, 4.0])
    assert np.allclose(o.norm(x, [1.0, 2.0], 0.0), np.array([3.0, 8.0]) / np.sqrt(12.5), rtol=1e-15)


@pytest.mark.parametrize("a,d", [
    (8.0, -1.0), (-8.0, 1.0), (0.0, 0.0),
    (8.0 * (1 + 2.0 ** -7), -(1 + 2.0 ** -7)),             # eight bits are kept
    (8.0 * (1 + 2.0 ** -8), -1.0),                         # half way: to even (128)
    (8.0 * (1 + 3 * 2.0 ** -8), -(1 + 2.0 ** -6)),         # half way: to even (130)
    (8.0 * (2 - 2.0 ** -9), -2.0),                         # up into the next binade
    (8 * 2.0 ** -24, -2.0 ** -24), (4 * 2.0 ** -24, 0.0), (5 * 2.0 ** -24, -2.0 ** -24),
    (12 * 2.0 ** -24, -2.0 ** -23),                        # steps of 2^-24, ties to even
    (65280.0, -8160.0), (65500.0, -8160.0), (1e30, -8160.0), (-np.inf, 8160.0),
])
def test_scale(a, d):
    assert o.scale_of(a) == d
    assert float(np.float16(d)) == d                        # held exactly


def test_every_held_value_is_exact_in_fp16():
    # 8 bits times 3 bits: all scales of one binade, the subnormal ones and the
    # largest, times all codes
    for s in list(range(128, 256)) + [1, 2, 127]:
        for e in (-24, -17, -7, 0, 5):
            d = s * 2.0 ** e
            if abs(d) <= 8160:
                assert o.scale_of(-8 * d) == d
                for c in range(-8, 8):
                    assert float(np.float16(c * d)) == c * d


def test_codes_hand_worked():
    x = np.zeros(32)
    x[:8] = [8.0, -7.0, 0.5, 1.5, -0.5, 7.4, -7.6, 2.4]     # d = -1: codes are 8 - x
    d, c = o.quantise(x)
    assert d[0] == -1.0
    # 8 -> -8; 7 -> 7; -0.5 -> 0 and -1.5 -> -2 (even); 0.5 -> 0; -7.4 -> -7; 7.6 -> 7 (clamped); -2.4 -> -2
    assert list(c[:8].astype(int) - 8) == [-8, 7, 0, -2, 0, -7, 7, -2]
    assert np.array_equal(o.values(d, c)[:8], [8, -7, 0, 2, 0, 7, -7, 2])
    # equal magnitudes: the lower channel decides
    x[:] = 0
    x[3], x[4] = -8.0, 8.0
    assert o.quantise(x)[0][0] == 1.0
    x[3], x[4] = 8.0, -8.0
    assert o.quantise(x)[0][0] == -1.0
    x[9] = np.nan
    assert np.isnan(o.quantise(x)[0][0])
    assert not o.quantise(np.zeros(32))[0].any()


def test_error_is_at_most_half_a_step():
    # |x - held| <= |d| / 2, but for the one code that is missing: x / d in
    # (7.5, 8 + 2^-8] is held as 7, and the scale's own rounding moves -8 by 2^-8 * 8 d
    rng = np.random.default_rng(2)
    x = rng.standard_normal((200, 64)) * np.exp2(rng.integers(-10, 10, (200, 1)))
    d, c = o.quantise(x)
    step = np.abs(np.repeat(d, 32, -1))
    assert (np.abs(x - o.values(d, c)) <= step * 1.04).all()
    inside = x / np.repeat(d, 32, -1) <= 7.5
    assert (np.abs(x - o.values(d, c))[inside] <= step[inside] * 0.5 + 2e-15).all()


def test_page_layout_and_round_trip():
    P, n_kv, hd = 16, 2, 64
    pages = np.zeros((3, o.page_bytes(P, n_kv, hd)), np.uint8)
    assert pages.shape[1] == 16 * 2 * 72
    x = np.zeros(64)
    x[0], x[1], x[33] = 8.0, 1.0, -16.0
    o.store(pages, 1, 5, P, hd, 1, 1, x)
    at = 3 * 16 * (32 + 4)                                  # head 1's values
    # d = -1: channel 0 is -8 (nibble 0 = 0), channel 1 is -1 (nibble 4 = 7), the rest 0 (8)
    assert list(pages[1, at + 5 * 32: at + 5 * 32 + 4]) == [0x80, 0x88, 0x87, 0x88]
    assert list(pages[1, at + 512 + 10: at + 512 + 12]) == [0x00, 0xBC]       # fp16(-1)
    assert list(pages[1, at + 512 + 32 + 10: at + 512 + 32 + 12]) == [0x00, 0x40]  # fp16(2)
    assert np.array_equal(o.load(pages, 1, 5, P, hd, 1, 1), x)
    assert not pages[0].any() and not pages[2].any()


def test_unpack_is_load_of_every_slot():
    rng = np.random.default_rng(3)
    P, n_kv, hd = 16, 2, 96
    pages = rng.integers(0, 120, (2, o.page_bytes(P, n_kv, hd)), dtype=np.uint8)   # no NaN scales
    x = o.unpack(pages, P, n_kv, hd)
    for page, slot, h, kv in [(0, 0, 0, 0), (1, 15, 1, 1), (0, 7, 1, 0), (1, 3, 0, 1)]:
        assert np.array_equal(x[page, slot, h, kv], o.load(pages, page, slot, P, hd, h, kv))
    K, V = o.sequence(pages, np.array([[1, 0], [5, -1]]), 0, 20, P, n_kv, hd)
    assert np.array_equal(K[17], x[0, 1, :, 0]) and np.array_equal(V[3], x[1, 3, :, 1])
    assert np.isnan(o.sequence(pages, np.array([[1, 0], [5, -1]]), 1, 20, P, n_kv, hd)[0]).all()


def test_rows():
    assert o.rows([0, 2, 2, 5], [7, 3, 3], 6) == [(0, 5), (0, 6), (2, 0), (2, 1), (2, 2), None]
    assert o.rows(None, [4, 1], 2) == [(0, 3), (1, 0)]


def test_attention_against_exact_sums():
    # scores chosen as multiples of ln 2, so the weights are powers of two and
    # the result a fraction
    K = np.zeros((3, 1, 32))
    K[:, 0, 0] = [0.0, 1.0, 3.0]
    V = np.arange(96.0).reshape(3, 1, 32)
    q = np.zeros((2, 32))
    q[:, 0] = np.log(2.0)
    out, mag, big = o.attention(q, 2, 3, K, V, 1.0)
    want = [float((Fraction(c) + 2 * Fraction(32 + c) + 8 * Fraction(64 + c)) / 11) for c in range(32)]
    assert np.allclose(out[0], want, rtol=1e-14) and np.array_equal(out[0], out[1])
    assert np.allclose(mag[0], want, rtol=1e-14) and np.allclose(big, 3 * np.log(2.0))
    # causal, window, nothing seen
    assert np.array_equal(o.attention(q, 0, 3, K, V, 1.0)[0][0], V[0, 0])
    assert np.array_equal(o.attention(q, 2, 3, K, V, 1.0, window=1)[0][0], V[2, 0])
    assert not o.attention(q, -1, 3, K, V, 1.0)[0].any()
    assert np.allclose(o.attention(q, 0, 3, K, V, 1.0, causal=False)[0][0], want, rtol=1e-14)
