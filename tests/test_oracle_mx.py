"""The oracle of the 4-bit gradients and 8-bit moments against hand cases,
PyTorch's own E4M3 type, every level's neighbours and exact probabilities."""

from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle
from oracle import mx

f = np.float32


def quantized(t):
    codes, scales, _ = mx.mx4_encode(np.asarray(t, f))
    return mx.mx4_decode(codes, scales, len(t)), scales


def test_hand_block():
    # maximum 6: scale 1; ties: 0.25 -> 0, 0.75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4
    t = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, 0.26, -5.01, 0.74]
    got, scales = quantized(t)
    assert scales.tolist() == [127]
    assert got.tolist() == [6, 0, 1, 1, 2, 2, 4, 4, 0, -1, 0.5, -6, 0.5]
    codes, _, _ = mx.mx4_encode(np.asarray(t, f))
    assert codes[0] == 0x07 and codes[1] == (0x2 << 4 | 0x2)     # the first of a pair in the low half
    assert codes.size == 16 and not codes[7:].any()              # zero behind the end
    assert codes[4] == (0xA << 4 | 0x8)                          # -0.25 keeps its sign


@pytest.mark.parametrize("top,scale", [(6.999, 127), (7.0, 128), (6.0, 127), (3.5, 127), (3.4999, 126), (1.0, 125),
                                       (2.0 ** -126 * 6, 1), (1e-45, 1), (0.0, 1), (1.7 * 2.0 ** 127, 252)])
def test_scale(top, scale):
    _, scales = quantized([top] + [0] * 31)
    assert scales.tolist() == [scale]


def test_half_a_step_at_most():
    rng = np.random.default_rng(0)
    t = (rng.standard_normal(64 * 32) * 2.0 ** rng.integers(-30, 30, 64).repeat(32)).astype(f)
    q, scales = quantized(t)
    x = np.abs(t.astype(np.float64)) / 2.0 ** (scales.astype(float).repeat(32) - 127)
    step = np.where(x < 2, 0.5, np.where(x < 4, 1, 2))
    assert (np.abs(t.astype(np.float64) - q) <= step / 2 * 2.0 ** (scales.astype(float).repeat(32) - 127)).all()


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan, 1.75 * 2.0 ** 127])
def test_blocks_without_numbers(bad):
    t = np.ones(96, f)
    t[40] = bad
    left = np.full(96, 0.125, f)
    codes, scales, new = mx.mx4_quantize(t, left)
    assert scales[1] == 255 and not codes[16:32].any() and scales[0] != 255 and scales[2] != 255
    q = mx.mx4_decode(codes, scales, 96)
    assert np.isnan(q[32:64]).all() and np.isfinite(q[:32]).all() and np.isfinite(q[64:]).all()
    assert (new[32:64] == left[32:64]).all()
    assert (new[:32] + q[:32] == f(1.125)).all()


def test_sent_adds_up_to_what_was_computed():
    """Over many steps the residual stays within half a step, so the sum of what
    was sent is the sum of the gradients to that."""
    rng = np.random.default_rng(1)
    left, sent, total = np.zeros(320, f), np.zeros(320), np.zeros(320)
    for _ in range(50):
        g = rng.standard_normal(320).astype(f)
        codes, scales, left = mx.mx4_quantize(g, left)
        sent += mx.mx4_decode(codes, scales, 320)
        total += g
    # float32 rounding of the 50 sums t: each at most 2^-24 of |t| < 8
    assert np.abs(total - sent - left).max() <= 50 * 8 * 2.0 ** -24
    assert np.abs(left).max() <= 2        # half a step of the largest scale met (maximum below 14: 2)


def test_m_codes_are_e4m3():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy()
    for s in (1, 64, 127, 200):
        got, _ = mx.moments_decode(codes, codes, np.array([s, 127] * 8, np.uint8))
        np.testing.assert_array_equal(got, want * f(2.0 ** (s - 127)))


def test_v_values():
    v = mx.V_VALUES
    assert (np.diff(v) > 0).all() and v[255] == 1.875 and v[248] == 1 and v[0] == 2.0 ** -31
    zero = np.zeros(40, np.uint8)
    assert not mx.moments_decode(zero, zero, np.zeros(4, np.uint8))[0].any()
    assert not mx.moments_decode(zero, zero, np.zeros(4, np.uint8))[1].any()


@pytest.mark.parametrize("which", ["m", "v"])
def test_rounding_at_random(which):
    """Between two codes, the number of the 65,536 random values that round up
    is the share cut off, to one of them; a code's own value never moves."""
    values = mx.M_VALUES if which == "m" else mx.V_VALUES
    r = np.arange(65536)
    for low in (0, 1, 7, 8, 60, 100):
        for part in (Fraction(0), Fraction(1, 1 << 20), Fraction(1, 3), Fraction(1, 2), Fraction(65535, 65536)):
            x = float(Fraction(values[low]) + part * (Fraction(values[low + 1]) - Fraction(values[low])))
            got = mx._round_at_random(np.full(65536, x), values, r)
            assert set(got) <= {low, low + 1}
            up = int((got == low + 1).sum())
            assert abs(up - float(part) * 65536) <= 1, (low, part, up)
            if part == 0:
                assert up == 0


def test_moment_scales():
    bits = np.zeros(32, np.int64)
    for top, sm in ((448, 127), (449, 128), (1.0, 119), (1.75, 119), (1.7501, 120), (0.0, 1)):
        _, _, s = mx.moments_encode(np.array([top] + [0] * 31, f), np.zeros(32, f), bits)
        assert s.tolist() == [sm, 0], top
    for top, sv in ((1.875, 127), (1.876, 128), (1.0, 127), (2.0 ** -100, 32), (2.0 ** 127, 254)):
        _, c, s = mx.moments_encode(np.zeros(32, f), np.array([top] + [0] * 31, f), bits)
        assert s.tolist() == [1, sv], top
        assert not c[1:].any()              # zeros beside it become 2^-31 scales
    m, v = np.zeros(64, f), np.zeros(64, f)
    m[3], v[40] = np.nan, np.inf
    mc, vc, s = mx.moments_encode(m, v, np.zeros(64, np.int64))
    assert s.tolist() == [255, 0, 1, 255] and (mc[:32] == 127).all() and not mc[32:].any() and not vc.any()
    dm, dv = mx.moments_decode(mc, vc, s)
    assert np.isnan(dm[:32]).all() and not dm[32:].any() and not dv[:32].any() and np.isinf(dv[32:]).all()


def test_moments_do_not_stop():
    """1,000 steps with g = 1 and b2 = 0.999: the mean second moment over 4,096
    elements is 1 - 0.999^1000 = 0.632.  A step's rounding has variance at most
    (change) * (gap) <= 0.001 * 0.0625 here (gaps below 1 are 1/16 at most), so
    the final one's is under 1000 * 6.25e-5 and its mean's deviation under
    0.25 / 64 = 0.0039; five of those."""
    n = 4096
    m = v = np.zeros(n, np.uint8)
    s = np.zeros(2 * n // 32, np.uint8)
    w = np.zeros(n, f)
    for t in range(1, 1001):
        w, m, v, s = mx.adamw8(np.ones(n, f), w, m, v, s, f(1), 1e-3, 0.9, 0.999, 1e-8, 0.0, t, 7, 0)
    _, got = mx.moments_decode(m, v, s)
    assert abs(float(got.astype(np.float64).mean()) - (1 - 0.999 ** 1000)) < 0.02


def test_random_bits():
    a = mx.random_bits(1000, 5, 9, 2)
    assert (a == mx.random_bits(500, 5, 9, 2, first=500)[np.arange(1000) % 500]).sum() >= 500
    for other in (mx.random_bits(1000, 6, 9, 2), mx.random_bits(1000, 5, 10, 2), mx.random_bits(1000, 5, 9, 3),
                  mx.random_bits(1000, 5 + (1 << 32), 9, 2), mx.random_bits(1000, 5, 9, 2, first=1 << 30)):
        assert (a != other).mean() > 0.99
    many = mx.random_bits(1 << 20, -1, 1, 0)
    for half in (many & 0xffff, many >> 16):
        # 2^20 draws, mean of 0 .. 65535: deviation 65536 / sqrt(12) / 1024 = 18.5; five of those
        assert abs(half.mean() - 32767.5) < 93
        counts = np.bincount(half >> 8, minlength=256)
        # 4096 expected in each of 256: deviation 64; six of those
        assert np.abs(counts - 4096).max() < 384
