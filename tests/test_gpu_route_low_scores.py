"""Routing where FP32 scores underflow: sigmoids of very low logits, whose order, groups, weights and gradient are those of
their exact values, and softmax scores of peaked logits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import nvfp4_weight_only_w4a16_gb300 as P
from tests.block_ops import DEV, dev, f64, route, tables
from tests.test_gpu_route_alone import _outs

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
