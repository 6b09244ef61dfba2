"""Plain float64 forms of the 4-bit products, their random operands and error bounds.

Bounds.  Every product of a code and an activation is exact in FP32 (NVFP4: 6 + 8
significant bits; INT4 codes: 4 + 8 or 4 + 11), so the kernels' only errors are
  * the FP32 summation of n terms, at most n * 2^-24 * sum |terms|, taken with a
    factor 4 for the tensor core's accumulation (which may truncate where a sum
    of its own would round) plus two more operations for the scales.  INT4 sums
    q x and x over a group and takes z times the second from the first, so its
    terms are |s| (q + z) |x|, not |s (q - z) x|, and it rounds twice as often;
  * where activations enter as FP16, those of a row times a power of two that
    brings the row's largest into [2^13, 2^14): an element is off by at most half
    of FP16's smallest step, 2^-25, that is 2^-38 of the row's largest (INT4, half
    of whose elements enter times another 2^-4: 2^-34), so the sum by at most that
    times max|x| * sum |w|;
  * the output's one rounding, eps / 2 of its value.
"""
import numpy as np
import torch

DEV = "cuda:0"
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def nvfp4(rng, *shape):
    """Random codes and scales of matrices [..., N, K]: every code, scales from zero over subnormal to 448."""
    *lead, n, k = shape
    q = rng.integers(0, 256, (*lead, n, k // 2), dtype=np.uint8)
    s = rng.choice(np.array([0x00, 0x01, 0x07, 0x10, 0x20, 0x28, 0x30, 0x33, 0x38, 0x3C, 0x40, 0x7E], np.uint8),
                   (*lead, n, k // 16), p=[.04, .04, .04, .1, .1, .1, .1, .1, .1, .1, .14, .04])
    return q, s


def nvfp4_values(q, s):
    """float64 [..., N, K] of E2M1 codes times E4M3 scales."""
    table = np.array(E2M1 + [-v for v in E2M1])
    code = np.stack([q & 15, q >> 4], axis=-1).reshape(*q.shape[:-1], -1)
    e, m = (s >> 3) & 15, s & 7
    scale = np.where(e > 0, (1 + m / 8) * 2.0 ** (e.astype(np.float64) - 7), m / 8 * 2.0 ** -6)
    return table[code] * np.repeat(scale, 16, axis=-1)


def int4_values(q, scale, zero, group, sign=-1.0):
    """float64 [N, K] of INT4 codes, scale (code - zero); scale float64 [N, K/g], zero [N, K/g] or None."""
    code = np.stack([q & 15, q >> 4], axis=-1).reshape(q.shape[0], -1).astype(np.float64)
    z = 8.0 if zero is None else np.repeat(zero.astype(np.float64), group, axis=1)
    return (code + sign * z) * np.repeat(scale, group, axis=1)


def f64(t):
    return t.detach().double().cpu().numpy()


def bound(y, x, w, out_dtype, fp16_rows=0.0, terms=None, rounds=1):
    """Largest allowed |error| of y = x w^T (x [r][n], w [m][n], all float64).

    fp16_rows: how far FP16 puts an element off, as a share of its row's largest; terms: the weights whose
    magnitudes the kernel sums (default w); rounds: how often it rounds per term."""
    n = x.shape[1]
    w = np.abs(w if terms is None else terms)
    b = 4.0 * (rounds * n + 2) * 2.0 ** -24 * (np.abs(x) @ w.T)
    if fp16_rows:
        b = b + fp16_rows * np.abs(x).max(axis=1, initial=0.0)[:, None] * w.sum(axis=1)[None, :]
    if out_dtype != torch.float32:
        fi = torch.finfo(out_dtype)
        b = b + fi.eps / 2 * (np.abs(y) + b) + fi.tiny * fi.eps
    return b


def check(got, y, b, what=""):
    err = np.abs(got - y)
    assert np.all(np.isfinite(got)), what
    worst = (err / np.maximum(b, 1e-300)).max(initial=0.0)
    assert np.all(err <= b), f"{what}: {worst:.3g} of the bound"
