"""The checks of tests.exact reject what a broken sum would give (planted here, in the plain form)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests.exact import check_exact, check_norm, int4_exact, nvfp4_exact, norm_error, rounded, rows_exact
from tests.products import int4_values, nvfp4_values

SIZES = [(16, 16384, 64), (32, 8320, 64), (96, 12416, 32), (208, 16384, 32), (272, 640, 128)]   # N, K, group


def _faults(x, w, unzeroed, group):
    """(what, result) of sums that lose, repeat or misplace something."""
    n, k = w.shape
    one = w.copy()
    one[:, k // 2] = 0.0
    if not one.any():
        raise AssertionError
    yield "one element lost", x @ one.T
    step = w.copy()
    step[:, 128 * (k // 256):128 * (k // 256) + 128] = 0.0
    yield "one step of 128 lost", x @ step.T
    last = w.copy()
    last[:, -128:] = 0.0
    yield "the last step lost", x @ last.T
    for s in (2, 4, 8):
        cut = k // 128 // s * 128
        if cut:
            part = w.copy()
            part[:, cut:2 * cut] = 0.0
            yield f"a slice of {s} lost", x @ part.T
            part[:, cut:2 * cut] = 2 * w[:, cut:2 * cut]
            yield f"a slice of {s} twice", x @ part.T
    yield "zero points taken for 8", x @ unzeroed.T
    yield "groups off by one", x @ np.roll(w, group, axis=1).T


@pytest.mark.parametrize("n,k,group", SIZES)
def test_exact_cases_reject_every_fault(n, k, group):
    rng = np.random.default_rng(k + n)
    q, s, z = int4_exact(rng, n, k, group)
    w, plain = int4_values(q, s, z, group), int4_values(q, s, None, group)
    x = rows_exact(rng, 2, k)
    y = x @ w.T
    assert np.all(np.abs(y) * 2 < 2 ** 24) and np.all(y * 2 == np.round(y * 2))
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        check_exact(rounded(y, dtype), y, dtype)
    for what, bad in _faults(x, w, plain, group):
        with pytest.raises(AssertionError):
            check_exact(rounded(bad, torch.float32), y, torch.float32, what)
    q, s, _ = nvfp4_exact(rng, 1, n, k)
    w = nvfp4_values(q, s)[0]
    y = x @ w.T
    assert np.all(np.abs(y) * 4 < 2 ** 24) and np.all(y * 4 == np.round(y * 4))
    check_exact(rounded(y, torch.float32), y, torch.float32)
    for what, bad in _faults(x, w, w[::-1], 16):
        with pytest.raises(AssertionError):
            check_exact(rounded(bad, torch.float32), y, torch.float32, what)


@pytest.mark.parametrize("n,k,group", SIZES)
def test_error_of_the_norm_rejects_every_fault(n, k, group):
    """The loosest figure that a test asks for is 1e-5; one element of 16384 is 1/128 of the norm."""
    rng = np.random.default_rng(k)
    q = rng.integers(0, 256, (n, k // 2), dtype=np.uint8)
    s, z = rng.uniform(-0.1, 0.1, (n, k // group)), rng.integers(0, 16, (n, k // group), dtype=np.uint8)
    w, plain = int4_values(q, s, z, group), int4_values(q, s, None, group)
    x = rng.standard_normal((2, k))
    y = x @ w.T
    check_norm(y.astype(np.float32).astype(np.float64), y, 2.0 ** -24)
    for what, bad in _faults(x, w, plain, group):
        assert norm_error(bad, y) > 1e-4, what
        with pytest.raises(AssertionError):
            check_norm(bad, y, 1e-5, what)
