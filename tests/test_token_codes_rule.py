"""The rule of the 8-bit codes as the kernels work it out: one factor a row in place of a division a value.

With v = a 2^i and top = b 2^j, 8-bit mantissas a, b in [128, 255], v / top = a / (b 2^s).  Enumerated here:
where v 127 / top is a tie, how near it comes to one otherwise, and that the factor (csrc/stream_dev.cuh,
code_factor, restated) gives the codes of two fp32 divisions for every a, b and s."""
from fractions import Fraction

import numpy as np

A, B, S = np.meshgrid(np.arange(128, 256), np.arange(128, 256), np.arange(12), indexing="ij")
KEEP = (S > 0) | (A <= B)  # |v| <= top
A, B, S = A[KEEP], B[KEEP], S[KEEP]


def test_ties_and_the_distance_to_them():
    # 127 a / (b 2^s) - (n + 1/2) = (254 a - (2 n + 1) b 2^s) / (2 b 2^s), whole numbers over 2 b 2^s
    unit = B << S
    n = (127 * A) // unit
    off = np.minimum(np.abs(254 * A - (2 * n + 1) * unit),
                     np.minimum(np.abs(254 * A - (2 * n - 1) * unit), np.abs(254 * A - (2 * n + 3) * unit)))
    tie = off == 0
    half = 2 * A == unit  # v = top / 2
    assert tie[half].all() and half[tie & (B != 254)].all()
    nearest = min(Fraction(int(o), int(2 * u)) * 2 ** int(s) for o, u, s in zip(off[~tie], unit[~tie], S[~tie]))
    assert nearest == Fraction(1, 510)  # a = 254, b = 255: 126.50196
    # what the fp32 quotient and the fp32 product are off by, 3 roundings of 2^-24 at 127 a / (b 2^s) <= 255 / 2^s
    assert 3 * 255 * 2.0 ** -24 < 1 / 510


def code_factor(top):
    f = np.float32(127) / top
    off = np.float64(f) * np.float64(top) - 127.0  # its sign is exact
    down = np.float32(0.5) * top / (top / np.float32(127)) < np.float32(63.5)
    if down and off >= 0:
        f = np.nextafter(f, np.float32(0), dtype=np.float32)
    if not down and off < 0:
        f = np.nextafter(f, np.float32(np.inf), dtype=np.float32)
    return f


def test_the_factor_gives_the_codes_of_two_divisions():
    for e in (-100, -20, 0, 1, 60, 119):
        factor = np.array([code_factor(np.float32(b * 2.0 ** e)) for b in range(128, 256)])
        top = (B * 2.0 ** e).astype(np.float32)
        v = (A * 2.0 ** (e - S)).astype(np.float32)
        want = np.rint(v / (top / np.float32(127)))
        product = v.astype(np.float64) * factor[B - 128].astype(np.float64)  # exact: 8 by 24 bits
        assert np.array_equal(np.rint(product), want)
