"""Plain float64 forms of the operators around the 4-bit products, and what their kernels' roundings may do.

A rounding is off by at most half a step: U = 2^-24 of the value in FP32, finfo(type).eps / 2 in 16 bits.  A sum of n
terms in FP32 is off by at most (length of its longest chain of additions) U sum |terms|.
"""
import numpy as np
import torch

DEV = "cuda:0"
U = 2.0 ** -24


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def f64(t):
    return t.detach().double().cpu().numpy()


def half_step(v, dtype):
    """Half a step of `dtype` at v, subnormals included."""
    fi = torch.finfo(dtype)
    return np.maximum(np.abs(v) * fi.eps / 2, fi.tiny * fi.eps / 2)


def within(got, want, tol, what=""):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    fine = np.isfinite(want)
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), what
    err, tol = np.abs(got - want)[fine], np.broadcast_to(tol, want.shape)[fine]
    assert np.all(err <= tol), f"{what}: {np.max(err / np.maximum(tol, 1e-300)):.3g} of the bound"


# ---------------------------------------------------------------------------
# codes
# ---------------------------------------------------------------------------

def codes(v, axis=-1):
    """round(127 v / max |v|), ties to even, and max |v|; exact products of 16-bit numbers in v."""
    peak = np.abs(v).max(axis=axis, keepdims=True)
    with np.errstate(invalid="ignore", divide="ignore"):
        q = np.where(peak > 0, np.rint(127.0 * v / peak), 0.0)
    return q, np.squeeze(peak, axis)


def blocks(v, n=128):
    pad = -v.shape[1] % n
    return np.pad(v, ((0, 0), (0, pad))).reshape(v.shape[0], -1, n)


def checkpoint(v):
    """codes [R][I] and scales [R][blocks] of 128-element blocks; a block that is not finite: 0 and NaN."""
    b = blocks(v)
    bad = ~np.isfinite(b).all(axis=2)
    q, peak = codes(np.where(bad[:, :, None], 0.0, b))
    return q.reshape(v.shape[0], -1)[:, :v.shape[1]], np.where(bad, np.nan, peak / 127.0)


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------
NORM_CHAIN = 8 * 4 + 10 + 3     # a thread's terms, the shuffles and warps, mean and eps


def norm(h, w, eps):
    r = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    return h * w * r[:, None], r


def norm_backward(dy, h, w, r, dsum):
    g, n = dy * w, h * r[:, None]
    c = (g * n).mean(axis=1, keepdims=True)
    dx = r[:, None] * (g - n * c) + dsum
    b_c = (NORM_CHAIN + 3) * U * (np.abs(g * n)).mean(axis=1, keepdims=True)
    b = r[:, None] * (np.abs(n) * b_c + 5 * U * (np.abs(g) + np.abs(n * c))) + 2 * U * np.abs(dx)
    return dx, b, (dy * n).sum(axis=0), (len(dy) + 70) * U * np.abs(dy * n).sum(axis=0)


# ---------------------------------------------------------------------------
# SwiGLU.  sigmoid: the exponential is off by 2 + 1.173 |g| steps of 2^-23 (its documented bound), the addition and the
# division by 3 more; exponentials past FP32's range count as infinite
# ---------------------------------------------------------------------------

def sigmoid(g):
    with np.errstate(over="ignore"):
        return np.where(g >= 0, 1.0 / (1.0 + np.exp(-np.abs(g))), np.exp(-np.abs(g)) / (1.0 + np.exp(-np.abs(g))))


def sigmoid_error(g):
    return (5 + 1.173 * np.abs(g)) * 2 * U


def swiglu(g, u, dtype):
    h = g * sigmoid(g) * u
    b = np.abs(h) * (sigmoid_error(g) + 3 * U) + np.abs(g * u) * 2.0 ** -125
    return h, b + half_step(np.abs(h) + b, dtype)


def swiglu_backward(g, u, d, dtype):
    s = sigmoid(g)
    r, f = sigmoid_error(g), 1.0 + g * (1.0 - s)
    dg, du = d * u * s * f, d * g * s
    bg = np.abs(d * u) * s * (np.abs(f) * (r + 5 * U) + np.abs(g) * (s * r + 2 * U) + 2 * U) + np.abs(d * u) * (1 + np.abs(g)) * 2.0 ** -125
    bu = np.abs(du) * (r + 4 * U) + np.abs(d * g) * 2.0 ** -125
    return dg, bg + half_step(np.abs(dg) + bg, dtype), du, bu + half_step(np.abs(du) + bu, dtype)


# ---------------------------------------------------------------------------
# routing
# ---------------------------------------------------------------------------

def scores(l, score):
    l = np.where(np.isnan(l), -np.inf, l)
    if score == "sigmoid":
        return sigmoid(l)
    m = l.max(axis=1, keepdims=True)
    with np.errstate(invalid="ignore"):
        ex = np.where(m == np.inf, (l == np.inf) * 1.0, np.where(m == -np.inf, 1.0, np.exp(l - np.where(np.isfinite(m), m, 0.0))))
    return ex / ex.sum(axis=1, keepdims=True)


def route(l, k, score="softmax", renorm=True, scale=1.0, bias=None, groups=1, top_groups=1, group_top=1):
    """ids, weights of float64 logits."""
    T, E = l.shape
    s, nan = scores(l, score), np.isnan(l)
    with np.errstate(invalid="ignore"):
        c = l if bias is None else s + bias[None, :]
    c = np.where(nan, np.nan, c)
    lost = np.isnan(c)
    ids = np.empty((T, k), np.int64)
    for t in range(T):
        open_ = np.ones(E, bool)
        if top_groups < groups:
            v = c[t] if group_top == 1 or bias is not None else s[t]
            v = np.where(lost[t], -np.inf, v).reshape(groups, -1)
            with np.errstate(invalid="ignore"):
                value = np.sort(v, axis=1)[:, ::-1][:, :group_top].sum(axis=1)
            value = np.where(np.isnan(value), -np.inf, value)
            best = sorted(range(groups), key=lambda g: (-value[g], g))[:top_groups]
            open_ = np.isin(np.arange(E) // (E // groups), best)
        order = sorted(np.flatnonzero(open_), key=lambda e: (bool(lost[t, e]), 0.0 if lost[t, e] else -c[t, e], e))
        ids[t] = order[:k]
    w = np.take_along_axis(np.where(nan, 0.0, s), ids, axis=1)       # a NaN's score counts as 0
    if score == "softmax" and renorm:
        w = scores(np.take_along_axis(l, ids, axis=1), "softmax")
    elif renorm:
        total = w.sum(axis=1, keepdims=True)
        w = np.where(total > 0, w / np.where(total > 0, total, 1.0), 1.0 / k)
    return ids, scale * w


def tables(ids, E):
    flat = ids.reshape(-1)
    perm = np.argsort(flat, kind="stable")
    inv = np.empty_like(perm)
    inv[perm] = np.arange(len(perm))
    return np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E))]), perm, inv


def route_weights_of(l, ids, score, renorm, scale):
    """The weights as a function of the logits for a fixed choice (torch, float64, differentiable)."""
    at = torch.gather
    if score == "softmax":
        w = torch.softmax(at(l, 1, ids), 1) if renorm else at(torch.softmax(l, 1), 1, ids)
    else:
        w = torch.sigmoid(at(l, 1, ids))
        if renorm:
            w = w / w.sum(1, keepdim=True)
    return scale * w
