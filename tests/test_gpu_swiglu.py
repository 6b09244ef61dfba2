"""SwiGLU with 8-bit checkpoints against float64: codes equal, scales one rounding off, the rest within the bounds of
block_ops; the backward pass against the formula at the values that the codes stand for."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import nvfp4_weight_only_w4a16_gb300 as P
from tests.block_ops import DEV, U, checkpoint, f64, swiglu, swiglu_backward, within

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def built():
    P.build()


def _rand(rng, shape, dt, scale=1.0):
    return torch.from_numpy(rng.standard_normal(shape) * scale).to(DEV).to(dt)


def _new(R, I, dt):
    return (torch.full((R, I), 7, dtype=dt, device=DEV), torch.full((R, 2, I), 99, dtype=torch.int8, device=DEV),
            torch.full((R, 2, -(-I // 128)), 7.0, device=DEV))


def _check_kept(v, q, s):
    qq, ss = checkpoint(f64(v))
    assert np.array_equal(f64(q), qq)
    within(f64(s), ss, U * np.abs(ss) + 2.0 ** -150, "scales")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("R,I", [(1, 16), (3, 48), (1, 128), (5, 144), (70, 1536), (1, 1552), (257, 272), (9, 16384),
                                 (20000, 32), (4000, 1536)])
def test_forward_and_backward(R, I, dt):
    rng = np.random.default_rng(R * I)
    op = P.SwiGLU(I, act_f16=dt == torch.float16)
    g, u, d = _rand(rng, (R, I), dt, 2.0), _rand(rng, (R, I), dt), _rand(rng, (R, I), dt, 2.0 ** -4)
    h, q, s = _new(R, I, dt)
    op.nvfp4_swiglu_forward(g, u, h, codes=q, scales=s)
    want, b = swiglu(f64(g), f64(u), dt)
    within(f64(h), want, b, "h")
    _check_kept(g, q[:, 0], s[:, 0])
    _check_kept(u, q[:, 1], s[:, 1])
    h2 = torch.empty_like(h)
    op.nvfp4_swiglu_forward(g, u, h2)
    assert torch.equal(h2, h)
    dg, du = (torch.full((R, I), 7, dtype=dt, device=DEV) for _ in range(2))
    op.nvfp4_swiglu_backward(q, s, d, dg, du)
    kept = f64(q) * np.repeat(f64(s), 128, axis=2)[:, :, :I]
    wg, bg, wu, bu = swiglu_backward(kept[:, 0], kept[:, 1], f64(d), dt)
    rel = lambda v: 0.0  # the kept values' own rounding in FP32, half a step, moves the results by:
    k = U * (np.abs(f64(d)) * (1 + np.abs(kept[:, 0])) * (np.abs(kept[:, 1]) * (1.1 + np.abs(kept[:, 0])) + 1.1))
    within(f64(dg), wg, bg + k + rel(wg), "dgate")
    within(f64(du), wu, bu + k, "dup")
    op.close()


@pytest.mark.parametrize("dt", TYPES)
def test_codes_next_to_the_border_of_two(dt):
    rng = np.random.default_rng(2)
    R, I = 600, 256
    v = rng.integers(-254, 255, (R, I)).astype(np.float64)
    v[:, ::128] = 254                                              # peak 254: every odd one is a midpoint
    v *= np.repeat(2.0 ** rng.integers(-5, 6, (R, 2)), 128, axis=1)
    x = torch.from_numpy(v).to(DEV).to(dt)
    near = f64(x) * (1 + rng.choice([-1, 1], (R, I)) * torch.finfo(dt).eps)
    near[:, ::128] = f64(x)[:, ::128]
    near = torch.from_numpy(near).to(DEV).to(dt)
    op = P.SwiGLU(I, act_f16=dt == torch.float16)
    h, q, s = _new(R, I, dt)
    op.nvfp4_swiglu_forward(x, near, h, codes=q, scales=s)
    _check_kept(x, q[:, 0], s[:, 0])
    _check_kept(near, q[:, 1], s[:, 1])
    op.close()


def test_values_out_of_range():
    """Blocks of zeros, of BF16's smallest and largest, infinities and NaNs; far sigmoids."""
    rng = np.random.default_rng(3)
    dt, R, I = torch.bfloat16, 12, 384
    g, u, d = _rand(rng, (R, I), dt), _rand(rng, (R, I), dt), _rand(rng, (R, I), dt)
    g[1, :128] = 0
    u[1, 128:256] = 0
    g[2] *= 2.0 ** -130
    u[2] *= 2.0 ** -120
    g[3] *= 2.0 ** 120
    u[4] *= 2.0 ** 110
    g[5] *= 60.0
    g[6, 200] = float("inf")
    g[7, 3] = float("nan")
    u[8, 383] = float("-inf")
    g[9, 0] = float("-inf")
    op = P.SwiGLU(I)
    h, q, s = _new(R, I, dt)
    op.nvfp4_swiglu_forward(g, u, h, codes=q, scales=s)
    for v, j in ((g, 0), (u, 1)):
        _check_kept(v, q[:, j], s[:, j])
    rows = [0, 1, 2, 4, 5, 10, 11]
    want, b = swiglu(f64(g)[rows], f64(u)[rows], dt)
    keep = np.abs(want) < 3e38
    within(f64(h)[rows][keep], want[keep], b[keep], "h")
    dg, du = torch.empty_like(g), torch.empty_like(g)
    op.nvfp4_swiglu_backward(q, s, d, dg, du)
    bad = np.isnan(f64(s))
    for j in range(3):
        cols = slice(128 * j, 128 * j + 128)
        rows_bad = bad[:, :, j].any(axis=1)
        assert np.isnan(f64(dg)[rows_bad, cols]).all()
        assert np.isfinite(f64(du)[~rows_bad][:, cols]).all()
    r = [0, 1, 5, 10, 11]
    kept = (f64(q) * np.repeat(f64(s), 128, axis=2)[:, :, :I])[r]
    wg, bg, wu, bu = swiglu_backward(kept[:, 0], kept[:, 1], f64(d)[r], dt)
    k = U * (np.abs(f64(d)[r]) * (1 + np.abs(kept[:, 0])) * (np.abs(kept[:, 1]) * (1.1 + np.abs(kept[:, 0])) + 1.1))
    within(f64(dg)[r], wg, bg + k, "dgate")
    within(f64(du)[r], wu, bu + k, "dup")
    op.close()


def test_gradient_against_differences():
    rng = np.random.default_rng(0)
    g, u, d = (rng.standard_normal((2, 8)) * 2 for _ in range(3))
    loss = lambda g, u: (swiglu(g, u, torch.float32)[0] * d).sum()
    dg, _, du, _ = swiglu_backward(g, u, d, torch.float32)
    for i, j in ((0, 0), (0, 5), (1, 7)):
        e = np.zeros_like(g)
        e[i, j] = 1e-6
        assert abs((loss(g + e, u) - loss(g - e, u)) / 2e-6 - dg[i, j]) < 1e-7
        assert abs((loss(g, u + e) - loss(g, u - e)) / 2e-6 - du[i, j]) < 1e-7


def test_strides_in_place_graph_and_no_rows():
    rng = np.random.default_rng(4)
    dt, R, I = torch.bfloat16, 130, 208
    op = P.SwiGLU(I)
    g, u, d = (_rand(rng, (R, I), dt) for _ in range(3))
    h, q, s = _new(R, I, dt)
    op.nvfp4_swiglu_forward(g, u, h, codes=q, scales=s)
    both = torch.zeros((R + 1, 2 * I + 8), dtype=dt, device=DEV)      # halves of one matrix, a row behind them
    both[:R, :I], both[:R, I:2 * I] = g, u
    _, q2, s2 = _new(R, I, dt)
    op.nvfp4_swiglu_forward(both[:R, :I], both[:R, I:2 * I], both[:R, :I], codes=q2, scales=s2)   # h over gate
    assert torch.equal(both[:R, :I], h) and torch.equal(q2, q) and torch.equal(s2, s)
    assert torch.equal(both[:R, I:2 * I], u) and not bool(both[R].any()) and not bool(both[:, 2 * I:].any())
    dg, du = torch.empty_like(g), torch.empty_like(g)
    op.nvfp4_swiglu_backward(q, s, d, dg, du)
    for a in (0, 1):
        o = [torch.empty_like(g), torch.empty_like(g)]
        o[a] = d.clone()
        op.nvfp4_swiglu_backward(q, s, o[a], o[0], o[1])
        assert torch.equal(o[0], dg) and torch.equal(o[1], du)
    e = torch.empty((0, I), dtype=dt, device=DEV)
    op.nvfp4_swiglu_forward(e, e, e)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            op.nvfp4_swiglu_forward(g, u, h, codes=q, scales=s)
            op.nvfp4_swiglu_backward(q, s, d, dg, du)
    for seed in (1, 2):
        g.copy_(_rand(np.random.default_rng(seed), (R, I), dt))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        h2, q2, s2 = _new(R, I, dt)
        a, b = torch.empty_like(g), torch.empty_like(g)
        op.nvfp4_swiglu_forward(g, u, h2, codes=q2, scales=s2)
        op.nvfp4_swiglu_backward(q2, s2, d, a, b)
        assert all(torch.equal(x, y) for x, y in ((h, h2), (q, q2), (s, s2), (dg, a), (du, b)))
    op.close()
