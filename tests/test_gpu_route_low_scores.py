"""Routing where FP32 scores underflow: sigmoids of very low logits, whose order, groups, weights and gradient are those of
their exact values, and softmax scores of peaked logits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import nvfp4_weight_only_w4a16_gb300 as P
from tests.block_ops import DEV, U, dev, f64, route, route_weights_of, sigmoid, tables, within
from tests.test_gpu_route_alone import _check, _outs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    P.build()


def _low(rng, T, E, lo, hi, bf16):
    l = dev(rng.uniform(lo, hi, (T, E)).astype(np.float32))
    return l.to(torch.bfloat16) if bf16 else l


# all scores flushed to 0 in FP32; some of them; none, next to the border; the lowest that 64 bits hold apart
@pytest.mark.parametrize("lo,hi", [(-150.0, -88.0), (-150.0, -78.0), (-90.0, -86.0), (-88.0, -77.0), (-700.0, -100.0)])
@pytest.mark.parametrize("T,E,k,groups,top", [(40, 64, 4, 8, 3), (300, 256, 8, 8, 4), (33, 60, 6, 6, 3), (130, 512, 8, 16, 5),
                                              (20, 64, 8, 1, 1)])
@pytest.mark.parametrize("group_top", [1, 2])
def test_low_sigmoids_keep_their_order(T, E, k, groups, top, group_top, lo, hi):
    rng = np.random.default_rng(T + E + int(-hi))
    kw = dict(score="sigmoid", groups=groups, top_groups=top, group_top=group_top)
    for bf16 in (False, True):
        h = P.Route(E, k, logits_bf16=bf16, **kw)
        logits = _low(rng, T, E, lo, hi, bf16)
        tiny = (rng.standard_normal(E) * 2.0 ** -126).astype(np.float32)
        for bias in (None, np.zeros(E, np.float32), tiny, (rng.standard_normal(E) * 0.1).astype(np.float32)):
            outs = _outs(T, E, k)
            h.nvfp4_route_forward(logits, *outs, bias=None if bias is None else dev(bias))
            want, _ = route(f64(logits), k, bias=None if bias is None else bias.astype(np.float64), **kw)
            assert np.array_equal(outs[0].cpu().numpy(), want)
            assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(outs[2:], tables(want, E)))
        h.close()


@pytest.mark.parametrize("spread", [10.0, 30.0])
@pytest.mark.parametrize("T,E,groups,top", [(300, 256, 8, 4), (60, 64, 8, 3)])
@pytest.mark.parametrize("biased", [False, True])
def test_peaked_softmax_in_groups(T, E, groups, top, biased, spread):
    """The border is between groups whose scores are far below the token's largest."""
    rng = np.random.default_rng(T)
    kw = dict(score="softmax", groups=groups, top_groups=top, group_top=2)
    h = P.Route(E, 8, **kw)
    logits = dev((rng.standard_normal((T, E)) * spread).astype(np.float32))
    bias = np.zeros(E, np.float32) if biased else None
    outs = _outs(T, E, 8)
    h.nvfp4_route_forward(logits, *outs, bias=dev(bias) if biased else None)
    want, _ = route(f64(logits), 8, bias=bias, **kw)
    assert np.array_equal(outs[0].cpu().numpy(), want)
    h.close()


# Chosen logits that are all below -17.4, the last ones also where FP32's sigmoid is 0; -inf and NaN count as 0.
# Weights: the bound of test_gpu_route_alone (exponentials of l - max and a sum), of which the exact 1 + e^l is less
# than half a rounding.
@pytest.mark.parametrize("lo,hi", [(-150.0, -88.0), (-100.0, -80.0), (-90.0, -60.0), (-30.0, -17.5), (-600.0, -560.0)])
@pytest.mark.parametrize("T,E,k", [(40, 64, 4), (200, 256, 8), (3, 16, 16)])
def test_renormalised_weights_of_low_sigmoids(T, E, k, lo, hi):
    rng = np.random.default_rng(T + int(abs(hi)))
    for bf16 in (False, True):
        h = P.Route(E, k, score="sigmoid", scale=2.5, logits_bf16=bf16)
        logits = _low(rng, T, E, lo, hi, bf16)
        logits[0, 1:] = -np.inf
        logits[1, ::2] = np.nan
        logits[2] = -np.inf
        outs = _outs(T, E, k)
        h.nvfp4_route_forward(logits, *outs)
        _check(h, logits, None, outs, E, k, dict(score="sigmoid", scale=2.5))
        h.close()


# Gradient: of w (d - sum d w), |d| at most the largest dweight: the bound of test_gpu_route_alone's, relative to w.
@pytest.mark.parametrize("lo,hi", [(-150.0, -88.0), (-88.6, -86.0), (-100.0, -80.0), (-90.0, -60.0), (-30.0, -17.5), (-20.0, 2.0)])
@pytest.mark.parametrize("T,E,k", [(40, 64, 4), (200, 256, 8), (3, 16, 16)])
def test_gradient_of_renormalised_low_sigmoids(T, E, k, lo, hi):
    rng = np.random.default_rng(T + int(abs(hi)))
    h = P.Route(E, k, score="sigmoid", scale=1.5)
    logits = _low(rng, T, E, lo, hi, False)
    ids = dev(np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32))
    dw = dev((rng.standard_normal((T, k)) * 100).astype(np.float32))
    dl = torch.full((T, E), 9.0, device=DEV)
    h.nvfp4_route_backward(logits, ids, dw, dl)
    l = logits.double().cpu().requires_grad_()
    (route_weights_of(l, ids.cpu().long(), "sigmoid", True, 1.5) * dw.double().cpu()).sum().backward()
    at, w = ids.cpu().numpy().astype(np.int64), np.zeros((T, E))
    s = np.take_along_axis(sigmoid(f64(logits)), at, 1)
    np.put_along_axis(w, at, s / s.sum(axis=1, keepdims=True), 1)
    d = np.abs(f64(dw)).max(axis=1, keepdims=True) * 1.5
    within(f64(dl), l.grad.numpy(), 8 * (E / 32 + 32 + 2 * np.abs(f64(logits)).max(axis=1, keepdims=True)) * U * w * d + 2.0 ** -120, "dlogits")
    h.close()
