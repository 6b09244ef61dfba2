"""Routing on its own against float64: ids and tables equal, weights and gradients within bounds.

Weights are quotients of exponentials (each off by two steps and by half a step of its argument, U |l - max|, whose
largest is what matters) and of a sum of up to E of them, along a chain of E / 32 + 5 additions.
"""
import itertools

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import nvfp4_weight_only_w4a16_gb300 as P
from tests.block_ops import DEV, U, dev, f64, half_step, route, route_weights_of, scores, sigmoid, tables, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    P.build()


def _outs(T, E, k):
    i = lambda *s: torch.full(s, -7, dtype=torch.int32, device=DEV)
    return i(T, k), torch.full((T, k), -7.0, device=DEV), i(E + 1), i(T * k), i(T * k)


def _weights_tol(l, w, E):
    fin = np.where(np.isfinite(l), l, 0.0)
    span = np.minimum(np.ptp(fin, axis=1, keepdims=True), 90.0) + np.minimum(np.abs(fin).max(1, keepdims=True), 90.0)
    return np.abs(w) * (2 * (E / 32 + 16) + 2 * span) * U + 2.0 ** -126


def _check(h, logits, bias, outs, E, k, kw):
    ids, w, off, perm, inv = outs
    l = f64(logits)
    want, ww = route(l, k, bias=None if bias is None else f64(bias), **kw)
    assert np.array_equal(ids.cpu().numpy(), want)
    within(f64(w), ww, _weights_tol(l, ww, E), "weights")
    o, p, v = tables(want, E)
    assert np.array_equal(off.cpu().numpy(), o) and np.array_equal(perm.cpu().numpy(), p) and np.array_equal(inv.cpu().numpy(), v)


SHAPES = [(1, 1, 1, 1, 1), (1, 8, 2, 1, 1), (2, 128, 8, 1, 1), (16, 256, 8, 8, 4), (33, 60, 6, 6, 3), (128, 64, 4, 4, 2),
          (129, 256, 8, 8, 4), (130, 72, 3, 1, 1), (257, 32, 16, 4, 2), (1500, 160, 8, 8, 3), (700, 512, 1, 1, 1),
          (1030, 512, 1, 16, 5), (1100, 384, 12, 32, 7), (40000, 16, 3, 2, 1), (4097, 256, 8, 8, 4),
          (20, 16, 16, 1, 1), (73, 128, 16, 4, 1), (72, 512, 16, 16, 1), (90, 64, 5, 2, 1), (3000, 1, 1, 1, 1), (5000, 8, 8, 2, 2)]


@pytest.mark.parametrize("T,E,k,groups,top", SHAPES)
@pytest.mark.parametrize("score,biased", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
def test_forward(T, E, k, groups, top, score, biased):
    rng = np.random.default_rng(T + E)
    n = 0
    for bf16, renorm in ((False, True), (True, False)):
        group_top = 1 + (n % 2 if E // groups > 1 else 0)
        n += 1
        kw = dict(score=score, renorm=renorm, scale=2.5 if renorm else 1.0, groups=groups, top_groups=top, group_top=group_top)
        h = P.Route(E, k, score=score, renormalize=renorm, scale=kw["scale"], groups=groups, top_groups=top,
                    group_top=group_top, logits_bf16=bf16)
        logits = dev(rng.standard_normal((T, E)).astype(np.float32))
        if bf16:
            logits = logits.to(torch.bfloat16)
        bias = dev((rng.standard_normal(E) * 0.1).astype(np.float32)) if biased else None
        outs = _outs(T, E, k)
        h.nvfp4_route_forward(logits, *outs, bias=bias)
        if T <= 5000:
            _check(h, logits, bias, outs, E, k, kw)
        else:                                          # the tables of its own ids, and some tokens' choice
            o, p, v = tables(outs[0].cpu().numpy().astype(np.int64), E)
            assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(outs[2:], (o, p, v)))
            some = rng.choice(T, 500, replace=False)
            want, ww = route(f64(logits)[some], k, bias=None if bias is None else f64(bias), **kw)
            assert np.array_equal(outs[0].cpu().numpy()[some], want)
            within(f64(outs[1])[some], ww, _weights_tol(f64(logits)[some], ww, E))
        assert h.nvfp4_moe_get_status() == (0, 0)
        h.close()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_neighbours_that_fp32_cannot_tell_apart(score):
    """Biases that make all c alike to 2^-26 and less: the order is that of 64 bits; and exact ties by the thousand."""
    rng = np.random.default_rng(8)
    T, E, k = 300, 64, 8
    base = rng.standard_normal(E).astype(np.float32)
    s = scores(base.astype(np.float64)[None], score)[0]
    bias = (0.5 - s).astype(np.float32)                # c = 0.5 up to bias's rounding
    logits = np.repeat(base[None], T, 0)
    if score == "sigmoid":
        logits = np.nextafter(logits, rng.choice([-9, 9], (T, E)).astype(np.float32))
    for kw in (dict(groups=1, top_groups=1, group_top=1), dict(groups=8, top_groups=3, group_top=2), dict(groups=8, top_groups=3, group_top=1)):
        h = P.Route(E, k, score=score, **kw)
        outs = _outs(T, E, k)
        lg, b = dev(logits), dev(bias)
        h.nvfp4_route_forward(lg, *outs, bias=b)
        _check(h, lg, b, outs, E, k, dict(score=score, **kw))
        tied = dev(rng.integers(-2, 3, (T, E)).astype(np.float32))
        zero = torch.zeros((E,), device=DEV)
        for bb in (None, zero):
            h.nvfp4_route_forward(tied, *outs, bias=bb)
            if score == "sigmoid" or bb is None:       # softmax of equal logits: equal in any order of the sum
                _check(h, tied, bb, outs, E, k, dict(score=score, **kw))
        h.close()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_infinities_nans_and_lowest_values(score, renorm):
    E, k, inf, nan, low = 16, 4, np.inf, np.nan, np.finfo(np.float32).min
    rng = np.random.default_rng(9)
    l = rng.standard_normal((12, E)).astype(np.float32)
    l[0] = -inf
    l[1] = nan
    l[2] = low
    l[3, :14] = -inf
    l[4, 5] = inf
    l[5, [2, 9]] = inf
    l[6, ::2] = nan
    l[7] = 0
    l[8, :13] = nan
    l[9] = 200.0
    l[10] = -200.0
    bias = rng.standard_normal(E).astype(np.float32) * 0.1
    for b in (None, bias, np.where(np.arange(E) % 3 == 0, -inf, bias).astype(np.float32),
              np.where(np.arange(E) % 3 == 0, low, bias).astype(np.float32), np.where(np.arange(E) == 3, nan, bias).astype(np.float32),
              np.where(np.arange(E) == 3, inf, bias).astype(np.float32)):
        for kw in (dict(groups=1, top_groups=1, group_top=1), dict(groups=4, top_groups=2, group_top=2)):
            h = P.Route(E, k, score=score, renormalize=renorm, **kw)
            outs, lg, bb = _outs(12, E, k), dev(l), None if b is None else dev(b)
            h.nvfp4_route_forward(lg, *outs, bias=bb)
            _check(h, lg, bb, outs, E, k, dict(score=score, renorm=renorm, **kw))
            assert h.nvfp4_moe_get_status() == (0, int(np.isnan(l).sum()))
            dl = torch.full_like(lg, 9.0)
            h.nvfp4_route_backward(lg, outs[0], torch.ones((12, k), device=DEV), dl)
            flat = [0, 1, 4, 5] if score == "softmax" else [1]
            assert np.isfinite(f64(dl)).all() and not f64(dl)[flat].any()
            h.close()


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (2, 128, 8), (19, 60, 6), (33, 64, 16), (200, 160, 8), (1021, 256, 8), (130, 512, 16)])
@pytest.mark.parametrize("score,renorm", list(itertools.product(["softmax", "sigmoid"], [False, True])))
@pytest.mark.parametrize("bf16", [False, True])
def test_backward(T, E, k, score, renorm, bf16):
    rng = np.random.default_rng(T * E)
    dt = torch.bfloat16 if bf16 else torch.float32
    h = P.Route(E, k, score=score, renormalize=renorm, scale=1.5, logits_bf16=bf16)
    logits = dev(rng.standard_normal((T, E)).astype(np.float32) * 2).to(dt)
    ids = dev(np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32))
    dw = dev(rng.standard_normal((T, k)).astype(np.float32))
    dl = torch.full((T, E), 9.0, dtype=dt, device=DEV)
    h.nvfp4_route_backward(logits, ids, dw, dl)
    l = logits.double().cpu().requires_grad_()
    (route_weights_of(l, ids.cpu().long(), score, renorm, 1.5) * dw.double().cpu()).sum().backward()
    want = l.grad.numpy()
    # of the score's gradient s (d - sum d s): every score off by the weights' bound, the sums of E terms by their chain
    s, d = scores(f64(logits), score), np.abs(f64(dw)).max(axis=1, keepdims=True) * 1.5
    at = ids.cpu().numpy()
    if renorm:
        chosen = np.zeros_like(s)
        np.put_along_axis(chosen, at.astype(np.int64), np.take_along_axis(s, at.astype(np.int64), 1), 1)
        s = chosen / chosen.sum(axis=1, keepdims=True)
    b = 8 * (E / 32 + 32 + 2 * np.abs(f64(logits)).max(axis=1, keepdims=True)) * U * s * d
    within(f64(dl), want, b + half_step(np.abs(want) + b, dt), "dlogits")
    h.close()


def test_gradient_against_differences():
    rng = np.random.default_rng(1)
    for score, renorm in itertools.product(["softmax", "sigmoid"], [False, True]):
        l = torch.from_numpy(rng.standard_normal((3, 10))).requires_grad_()
        ids = torch.from_numpy(np.argsort(rng.random((3, 10)), axis=1)[:, :4].copy())
        d = torch.from_numpy(rng.standard_normal((3, 4)))
        f = lambda l: (route_weights_of(l, ids, score, renorm, 1.5) * d).sum()
        f(l).backward()
        for i, j in ((0, 0), (1, 4), (2, 9)):
            e = torch.zeros_like(l)
            e[i, j] = 1e-6
            with torch.no_grad():
                assert abs(float(f(l + e) - f(l - e)) / 2e-6 - float(l.grad[i, j])) < 1e-7


def test_ids_that_name_no_expert():
    h = P.Route(8, 3, score="sigmoid", renormalize=False)
    l, dw = torch.zeros((2, 8), device=DEV), torch.ones((2, 3), device=DEV)
    ids = torch.tensor([[8, 1, -1], [2 ** 31 - 1, -2 ** 31, 0]], dtype=torch.int32, device=DEV)
    dl = torch.full((2, 8), 9.0, device=DEV)
    h.nvfp4_route_backward(l, ids, dw, dl)
    want = torch.zeros((2, 8))
    want[0, 1] = want[1, 0] = 0.25
    assert torch.equal(dl.cpu(), want)
    h.close()


@pytest.mark.parametrize("score,renorm", list(itertools.product(["softmax", "sigmoid"], [False, True])))
def test_an_expert_named_twice_counts_twice(score, renorm):
    E, k = 40, 6
    rng = np.random.default_rng(2)
    h = P.Route(E, k, score=score, renormalize=renorm)
    l, dw = dev(rng.standard_normal((50, E)).astype(np.float32)), dev(rng.standard_normal((50, k)).astype(np.float32))
    ids = dev(rng.integers(0, 4, (50, k)).astype(np.int32))
    dl = [torch.empty_like(l) for _ in range(2)]
    for d in dl:
        h.nvfp4_route_backward(l, ids, dw, d)
    assert torch.equal(*dl)
    x = l.double().cpu().requires_grad_()
    (route_weights_of(x, ids.cpu().long(), score, renorm, 1.0) * dw.double().cpu()).sum().backward()
    # k slots whose terms are at most |dw| s, each off by the scores' bound (test_backward), added k times
    within(f64(dl[0]), x.grad.numpy(), 8 * (E / 32 + 40) * U * k * np.abs(f64(dw)).max(axis=1, keepdims=True), "dlogits")
    h.close()


def test_strides_and_no_tokens():
    rng = np.random.default_rng(3)
    for E, bf16, pad in ((64, False, 3), (64, False, 4), (64, True, 8), (60, True, 1), (256, False, 0)):
        T, k, dt = 200, 4, torch.bfloat16 if bf16 else torch.float32
        h = P.Route(E, k, logits_bf16=bf16)
        wide = dev(rng.standard_normal((T, E + pad)).astype(np.float32)).to(dt)
        for o in {0, min(1, pad), pad}:
            view, flat = wide[:, o:o + E], wide[:, o:o + E].contiguous()
            a, b = _outs(T, E, k), _outs(T, E, k)
            h.nvfp4_route_forward(view, *a)
            h.nvfp4_route_forward(flat, *b)
            assert all(torch.equal(x, y) for x, y in zip(a, b))
            dw = torch.ones((T, k), device=DEV)
            grad = torch.full_like(wide, 5.0)
            h.nvfp4_route_backward(view, a[0], dw, grad[:, o:o + E])
            h.nvfp4_route_backward(flat, a[0], dw, flat)          # over the logits
            assert torch.equal(grad[:, o:o + E], flat)
            grad[:, o:o + E] = 5.0
            assert bool((grad == 5.0).all())
        e = _outs(0, E, k)
        h.nvfp4_route_forward(wide[:0, :E], *e)
        assert not bool(e[2].any())
        h.nvfp4_route_backward(wide[:0, :E], e[0], e[1], wide[:0, :E])
        h.close()


@pytest.mark.parametrize("T", [100, 3000])
def test_graph_and_overlapping_calls(T):
    """Captured and replayed with other logits; calls of one handle on four streams at once."""
    E, k = 256, 8
    h = P.Route(E, k, score="sigmoid", groups=8, top_groups=4, group_top=2)
    bias = dev((np.random.default_rng(0).standard_normal(E) * 0.1).astype(np.float32))
    make = lambda seed: dev(np.random.default_rng(seed).standard_normal((T, E)).astype(np.float32))
    logits, outs, dl = make(0), _outs(T, E, k), torch.empty((T, E), device=DEV)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            h.nvfp4_route_forward(logits, *outs, bias=bias)
            h.nvfp4_route_backward(logits, outs[0], outs[1], dl)
    plain = {}
    for seed in range(4):
        a, d = _outs(T, E, k), torch.empty((T, E), device=DEV)
        h.nvfp4_route_forward(make(seed), *a, bias=bias)
        h.nvfp4_route_backward(make(seed), a[0], a[1], d)
        plain[seed] = (*a, d)
    for seed in (1, 2):
        logits.copy_(make(seed))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip((*outs, dl), plain[seed]))
    ls = [make(s) for s in range(4)]
    streams = [torch.cuda.Stream() for _ in ls]
    got = [[_outs(T, E, k) for _ in range(10)] for _ in ls]
    torch.cuda.synchronize()
    for i in range(10):
        for s, l, o in zip(streams, ls, got):
            h.nvfp4_route_forward(l, *o[i], bias=bias, stream=s)
    torch.cuda.synchronize()
    for seed, o in enumerate(got):
        assert all(torch.equal(x, y) for r in o for x, y in zip(r, plain[seed]))
    h.close()
