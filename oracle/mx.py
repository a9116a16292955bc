"""Microscaled 4-bit gradients, their all-reduce, and AdamW with 8-bit moments.

TEST INFRASTRUCTURE ONLY (see the package docstring).

The pages count what an all-reduce moves ("Distributed Training",
"Communication costs") and what optimizer state costs ("Sharded data
parallelism"); none writes a compressed form.  Readings: blocks of 32
elements with a power-of-two scale, elements E2M1 for gradients and E4M3 for
first moments (the OCP microscaling formats), a sign-less 5-bit exponent and
3-bit mantissa for second moments; the rounding error of a gradient goes into
the next step's; moments are rounded at random, so that their expectation is
exact.

Everything is written from the definitions: levels and code values are
tables, a scale is found by trying exponents, the nearest level by comparing
distances, in float64 where they are exact.

Parity status: pinned by the tests against hand cases, PyTorch's E4M3 type,
exhaustive neighbours of every level and, for the rounding at random, exact
probabilities and the mean of a long run.
"""

import numpy as np

from .grads import _power, adamw

BLOCK = 32
LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def _blocks(x):
    """[n] as [blocks, 32], zeros behind the end."""
    x = np.asarray(x)
    out = np.zeros((-(-x.size // BLOCK), BLOCK), x.dtype)
    out.reshape(-1)[:x.size] = x
    return out


def _smallest_exponent(top, fits, least):
    """The smallest k >= least with fits(top, 2^k), for each block."""
    k = np.full(top.shape, least, np.int64)
    while True:
        more = ~fits(top, 2.0 ** k) & (k < 200)
        if not more.any():
            return k
        k[more] += 1


# ------------------------------------------------------------ 4 bits ----

def mx4_encode(t):
    """(codes [blocks * 16] uint8, scales [blocks] uint8, finite [n] bool) of
    float32 values [n]."""
    n = np.size(t)
    with np.errstate(invalid="ignore"):
        b = _blocks(np.asarray(t, np.float32)).astype(np.float64)
        top = np.abs(b).max(axis=1, initial=0)
        finite = np.isfinite(b).all(axis=1) & (top < 1.75 * 2.0 ** 127)
    b[~finite] = 0
    k = _smallest_exponent(np.where(finite, top, 0), lambda x, s: x < 7 * s, -126)
    x = np.abs(b) / 2.0 ** k[:, None]
    distance = np.abs(x[:, :, None] - LEVELS)
    # the nearest level; of two at the same distance the even code
    place = distance.argmin(axis=2)
    up = np.minimum(place + 1, 7)
    tie = (np.take_along_axis(distance, up[:, :, None], 2)[:, :, 0] == distance.min(axis=2)) & (up != place)
    place = np.where(tie & (place % 2 == 1), up, place)
    code = (place + 8 * np.signbit(b)).astype(np.uint8)
    code[~finite] = 0
    code = code.reshape(-1)
    scales = np.where(finite, k + 127, 255).astype(np.uint8)
    return code[0::2] | code[1::2] << 4, scales, np.repeat(finite, BLOCK)[:n]


def mx4_decode(codes, scales, n):
    """float32 values [n]."""
    code = np.stack([codes & 15, codes >> 4], -1).reshape(-1)[:n].astype(int)
    value = LEVELS[code & 7] * np.where(code & 8, -1.0, 1.0)
    s = np.repeat(np.asarray(scales, np.int64), BLOCK)[:n]
    value = np.where(s == 255, np.nan, value * 2.0 ** (s - 127.0))
    with np.errstate(over="ignore"):
        return value.astype(np.float32)


def mx4_quantize(g, residual=None):
    """(codes, scales, new residual float32 or None): g and residual float32."""
    g = np.asarray(g, np.float32)
    with np.errstate(all="ignore"):
        t = g + np.asarray(residual, np.float32) if residual is not None else g
    codes, scales, finite = mx4_encode(t)
    if residual is None:
        return codes, scales, None
    with np.errstate(all="ignore"):
        left = t - mx4_decode(codes, scales, g.size)
    return codes, scales, np.where(finite, left, residual).astype(np.float32)


def mx4_allreduce(rows, op):
    """float32 [n] of P decoded rows [P, n] float32: added in rank order."""
    with np.errstate(all="ignore"):
        g = rows[0].copy()
        for x in rows[1:]:
            g = g + x
        return g / np.float32(len(rows)) if op == "mean" else g


# ------------------------------------------------------------- 8 bits ----

# Values of m's codes 0 .. 126 (the sign apart) and of v's 0 .. 255, in scales.
M_VALUES = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7) for c in range(127)])
V_VALUES = np.array([(1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 31) for c in range(256)])


def moments_decode(m, v, scales):
    """float32 values (m, v) of codes [n] and scales [2 * blocks]."""
    n = m.size
    s = np.repeat(scales.reshape(-1, 2).astype(np.int64), BLOCK, axis=0)[:n]
    mag = np.where((m & 127) == 127, np.nan, M_VALUES[np.minimum(m & 127, 126)])
    with np.errstate(all="ignore"):
        mv = np.where(m & 128, -mag, mag) * 2.0 ** (s[:, 0] - 127.0)
        vv = V_VALUES[v] * np.where(s[:, 1] == 0, 0.0, 2.0 ** (s[:, 1] - 127.0))
        return (np.where(s[:, 0] == 255, np.nan, mv).astype(np.float32),
                np.where(s[:, 1] == 255, np.inf, vv).astype(np.float32))


def _round_at_random(x, values, r):
    """Codes of x >= 0, in scales: the code below, or the next one if the part
    cut off (20 bits of it, the nearest where m's steps are equal, all that a
    float32 has elsewhere) and 16 random bits and a half reach a whole."""
    low = np.clip(np.searchsorted(values, x, side="right") - 1, 0, None)
    high = np.minimum(low + 1, values.size - 1)
    gap = values[high] - values[low]
    with np.errstate(all="ignore"):
        part = np.where(gap > 0, (x - values[low]) / np.where(gap > 0, gap, 1), 0)
    part = np.clip(part, 0, None)          # below the least code: that code
    return np.where(np.rint(part * 2 ** 20) + 16 * r + 8 >= 2 ** 20, high, low)


def moments_encode(m, v, bits):
    """(m codes, v codes, scales) of float32 moments [n] with 32 random bits
    for each element."""
    n = m.size
    mb, vb = _blocks(np.asarray(m, np.float32)).astype(np.float64), _blocks(np.asarray(v, np.float32)).astype(np.float64)
    r = _blocks(np.asarray(bits, np.int64))
    m_ok, v_ok = np.isfinite(mb).all(axis=1), np.isfinite(vb).all(axis=1)
    signs = np.signbit(mb)
    mb, vb = np.abs(np.where(m_ok[:, None], mb, 0)), np.where(v_ok[:, None], vb, 0)
    mtop, vtop = mb.max(axis=1, initial=0), vb.max(axis=1, initial=0)
    v_ok &= vtop <= 1.875 * 2.0 ** 127
    vb[~v_ok], vtop[~v_ok] = 0, 0
    mk = _smallest_exponent(mtop, lambda x, s: x <= 448 * s, -126)
    vk = _smallest_exponent(vtop, lambda x, s: x <= 1.875 * s, -95)
    mc = _round_at_random(mb / 2.0 ** mk[:, None], M_VALUES, r & 0xffff) | np.where(signs, 128, 0)
    vc = _round_at_random(vb / 2.0 ** vk[:, None], V_VALUES, r >> 16)
    mc[~m_ok] = 127
    vc[~v_ok | (vtop == 0)] = 0
    scales = np.stack([np.where(m_ok, mk + 127, 255), np.where(v_ok, np.where(vtop > 0, vk + 127, 0), 255)], -1)
    return (mc.reshape(-1)[:n].astype(np.uint8), vc.reshape(-1)[:n].astype(np.uint8),
            scales.reshape(-1).astype(np.uint8))


def _mix(h, word):
    x = (h ^ word) + 0x9E3779B9 & 0xffffffff
    x ^= x >> 16
    x = x * 0xBB67AE85 & 0xffffffff
    x ^= x >> 15
    x = x * 0x3C6EF373 & 0xffffffff
    return x ^ x >> 16


def random_bits(n, seed, step, tensor, first=0):
    """32 bits for the elements first .. first + n - 1 of a tensor; pieces of
    2^30 elements have keys of their own."""
    i = np.arange(first, first + n, dtype=np.uint64)
    out = np.empty(n, np.uint64)
    for piece in np.unique(i >> np.uint64(30)):
        h = 0
        for word in (seed & 0xffffffff, seed >> 32 & 0xffffffff, step & 0xffffffff, step >> 32, tensor, int(piece)):
            h = _mix(h, word)
        at = (i >> np.uint64(30)) == piece
        x = ((i[at] & np.uint64(2 ** 30 - 1)) * np.uint64(0x9E3779B9) + np.uint64(h)) & np.uint64(0xffffffff)
        x ^= x >> np.uint64(15)
        x = x * np.uint64(0xBB67AE85) & np.uint64(0xffffffff)
        out[at] = x ^ x >> np.uint64(16)
    return out.astype(np.int64)


def adamw8(g, w, m, v, scales, c, lr, b1, b2, eps, wd, t, seed, tensor):
    """One step on one tensor: (w, m, v, scales).  The codes are what the kernel
    writes; the weights' root and quotient are rounded correctly here and within
    1 ulp each there, see weight_bound."""
    mv, vv = moments_decode(m, v, scales)
    f = np.float32
    _, mv, vv = adamw(g, w, mv, vv, c, lr, b1, b2, eps, wd, t)
    with np.errstate(all="ignore"):
        least = np.maximum(vv, f(2.0 ** -126))
        w = np.asarray(w, f) * f(1.0 - lr * wd) - _update(mv, least, lr, b1, b2, eps, t)
    return (w, *moments_encode(mv, vv, random_bits(m.size, seed, t, tensor)))


def _update(m, v, lr, b1, b2, eps, t):
    f = np.float32
    return f(lr / (1.0 - _power(b1, t))) * (m / (np.sqrt(v) * f(1.0 / np.sqrt(1.0 - _power(b2, t))) + f(eps)))


def weight_bound(g, w, m, v, scales, c, lr, b1, b2, eps, wd, t):
    """How far the kernel's new weights may be from adamw8's.  Relative errors in
    steps of 2^-24 of the quotient: here root, product, sum and quotient 1 each;
    there root 2, product 1, sum 1, reciprocal 2, product 1: 11 together.  Then on
    both sides the product with the step's size, 1 each, and the difference, 1
    each of the weight; products of these errors and of subnormal results are
    covered by one more of each."""
    mv, vv = moments_decode(m, v, scales)
    new, mv, vv = adamw(g, w, mv, vv, c, lr, b1, b2, eps, wd, t)
    with np.errstate(all="ignore"):
        u = np.abs(_update(mv, np.maximum(vv, np.float32(2.0 ** -126)), lr, b1, b2, eps, t).astype(np.float64))
        return 2.0 ** -24 * (14 * u + 3 * (np.abs(w.astype(np.float64)) + u)) + 2.0 ** -126
