"""The 8-bit codes of 16-bit elements, in the steps that csrc/quant8.cuh takes in FP32, against the exact quotient: every
pair of 11-bit significands (FP16's; BF16's are among them) with the element up to nine binary places below the peak, for
every reciprocal that an approximation within one step may give."""
from fractions import Fraction

import numpy as np

F = np.float32
MAGIC = F(12582912.0)                       # 1.5 2^23


def _fma(a, b, c):
    """a b + c in FP32, rounded once (ties to even)."""
    exact = Fraction(float(a)) * Fraction(float(b)) + Fraction(float(c))
    near = F(float(exact))                  # within two steps of it; the nearest of its neighbours
    around = [np.nextafter(near, F(-np.inf)), near, np.nextafter(near, F(np.inf))]
    return min(around, key=lambda v: (abs(Fraction(float(v)) - exact), int(v.view(np.int32)) & 1))


def _inverses(peak):
    """127 (1 + 2^-22) / peak as the kernel forms it from each reciprocal within a step of the exact one."""
    r0 = F(1.0 / float(peak))
    out = set()
    for r in (np.nextafter(r0, F(0)), r0, np.nextafter(r0, F(np.inf))):
        out.add(_fma(r, _fma(-peak, r, F(1.0)), r) * F(127.00003))
    return out


def _exact(v, peak):
    """round(127 v / peak), ties to even, of integers"""
    q, rest = np.divmod(127 * v, peak)
    return q + ((2 * rest > peak) | ((2 * rest == peak) & (q % 2 == 1)))


def test_the_reciprocals_factor():
    assert abs(float(F(127.00003)) / 127.0 - 1 - 2.0 ** -22) < 2.0 ** -28


def test_codes_of_every_pair_of_significands():
    assert _exact(np.array([1, 3, 2, 254]), 254).tolist() == [0, 2, 1, 127]    # 0.5, 1.5: to even
    significands = np.arange(1024, 2048, dtype=np.int64)
    for peak in range(1024, 2048):
        for places in range(10):
            v = significands[significands <= peak] if places == 0 else significands
            want = _exact(v, peak << places)
            x = v.astype(F) * F(2.0 ** -places)
            for inv in _inverses(F(peak)):
                for sign in (1, -1):
                    m = ((sign * x * inv).view(np.uint32) & ~np.uint32(7)).view(F) + MAGIC
                    got = m.view(np.uint32).astype(np.uint8).view(np.int8)
                    assert np.array_equal(got, sign * want), (peak, places)
