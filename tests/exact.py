"""Checks that the elementwise bounds of tests.products leave room beside: at long sums those grow past a lost term.

Exact cases.  Codes, power-of-two scales and small whole x, so that every product and every partial sum is a
multiple of some 2^-j below 2^24 of them: FP32 holds each one, in whatever order they are added, also where an adder
drops the bits below the last it keeps.  The result has to be right to the bit, or for a 16-bit type the right
rounding of it.  One lost, doubled or misplaced term shows.
  NVFP4: codes in halves up to 6, scales 1/2, 1, 2, |x| <= 2, tensor scales powers of two: multiples of 1/4 (before the
  tensor scale), at most 24 n: 96 n < 2^24 of them for n <= 16384 terms.
  INT4: |q - z| <= 15, q <= 15, scales 1/2, 1, 2, |x| <= 2: multiples of 1/2, at most 60 n: 120 n < 2^24 of them.

Error of the norm.  || got - y || / || y || over random operands against the documented figure."""
import numpy as np
import torch


def nvfp4_exact(rng, e, n, k):
    """Codes, scales and tensor scales of e matrices [n][k]."""
    q = rng.integers(0, 256, (e, n, k // 2), dtype=np.uint8)
    s = rng.choice(np.array([0x30, 0x38, 0x40], np.uint8), (e, n, k // 16))
    return q, s, rng.choice(np.array([0.25, 0.5, 1.0, 4.0], np.float32), e)


def int4_exact(rng, n, k, group):
    """Codes, scales (float64) and zero points of a matrix [n][k]."""
    q = rng.integers(0, 256, (n, k // 2), dtype=np.uint8)
    return q, rng.choice([0.5, 1.0, 2.0], (n, k // group)), rng.integers(0, 16, (n, k // group), dtype=np.uint8)


def rows_exact(rng, r, k):
    """Whole numbers -2..2 but zero, which would hide a lost term; float64."""
    return rng.choice([-2.0, -1.0, 1.0, 2.0], (r, k))


def rounded(y, dtype):
    """y (float64, exact in FP32) as the values of dtype."""
    return torch.from_numpy(np.ascontiguousarray(y)).float().to(dtype).double().numpy()


def check_exact(got, y, dtype, what=""):
    want = rounded(y, dtype)
    wrong = np.nonzero(got != want)
    assert not len(wrong[0]), f"{what}: {len(wrong[0])} of {want.size}, first {[int(i[0]) for i in wrong]}: " \
                              f"{got[wrong][0]}, not {want[wrong][0]}"


def norm_error(got, y):
    return float(np.linalg.norm(got - y) / np.linalg.norm(y))


def check_norm(got, y, most, what=""):
    e = norm_error(got, y)
    assert e <= most, f"{what}: error {e:.3g} of the norm, at most {most:.3g}"
