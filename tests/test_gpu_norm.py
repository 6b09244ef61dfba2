"""The RMS norm with the residual's addition, its 8-bit output and its gradient against float64.

Codes are equal; sums are equal to the rounded exact sum; the rest within bounds from the roundings on the way
(block_ops): rstd half of the sum's error and two roundings, y one product more, its scale two, and the type's rounding.
"""
import threading

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import nvfp4_weight_only_w4a16_gb300 as P
from tests.block_ops import DEV, NORM_CHAIN, U, codes, f64, half_step, norm, norm_backward, within

pytestmark = pytest.mark.gpu
EPS = 1e-6
R_ERR = (NORM_CHAIN / 2 + 3) * U


@pytest.fixture(scope="module", autouse=True)
def built():
    P.build()


def _rand(rng, shape, dt, scale=1.0):
    return torch.from_numpy(rng.standard_normal(shape) * scale).to(DEV).to(dt)


def _check(h, x, r, w, eps, sum_, y, q, s, rstd, dt):
    H = f64(x)
    if r is not None:
        H = (f64(x) + f64(r)).astype(np.float32)
        H = f64(torch.from_numpy(H).to(dt))
        assert np.array_equal(f64(sum_), H, equal_nan=True)
    W = f64(w)
    want, rr = norm(H, W, float(np.float32(eps)))
    within(f64(rstd), rr, R_ERR * rr, "rstd")
    if y is not None:
        b = (R_ERR + 2 * U) * np.abs(want)
        within(f64(y), want, b + half_step(np.abs(want) + b, dt), "y")
    if q is not None:
        qq, peak = codes(H * W)
        assert np.array_equal(f64(q), qq)
        within(f64(s), peak * rr / 127.0, (R_ERR + 3 * U) * peak * rr / 127.0 + 2.0 ** -149, "q_scale")


# every split of a row over threads, rows that do not fill it, and the largest
@pytest.mark.parametrize("T,H", [(1, 8), (5, 64), (37, 72), (3, 128), (9, 136), (400, 256), (33, 264), (700, 512), (400, 520),
                                 (1, 1000), (400, 1024), (2, 4096), (400, 4096), (61, 4104), (350, 5120), (17, 8192),
                                 (330, 8192), (1, 16384), (333, 16384)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("residual", [False, True])
def test_forward(T, H, dt, residual):
    rng = np.random.default_rng(T * H)
    n = P.Norm(H, EPS, act_f16=dt == torch.float16)
    x, w = _rand(rng, (T, H), dt), _rand(rng, (H,), dt)
    r = _rand(rng, (T, H), dt, 3.0) if residual else None
    new = lambda d=dt: torch.full((T, H), 7, dtype=d, device=DEV)
    sum_, y, q = new() if residual else None, new(), new(torch.int8)
    s, rstd = (torch.empty((T,), device=DEV) for _ in range(2))
    n.nvfp4_norm_forward(x, w, residual=r, sum=sum_, y=y, q=q, q_scale=s, rstd=rstd)
    _check(n, x, r, w, EPS, sum_, y, q, s, rstd, dt)
    # each output alone is the same
    y2, q2, s2 = new(), new(torch.int8), torch.empty((T,), device=DEV)
    n.nvfp4_norm_forward(x, w, residual=r, sum=sum_, y=y2)
    n.nvfp4_norm_forward(x, w, residual=r, sum=sum_, q=q2, q_scale=s2)
    assert torch.equal(y2, y) and torch.equal(q2, q) and torch.equal(s2, s)
    n.close()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("H", [64, 512, 4096])
def test_codes_next_to_the_border_of_two(dt, H):
    """Rows whose quotients 127 v / peak are exact midpoints, or as near to one as the type allows."""
    rng = np.random.default_rng(H)
    T = 512
    v = rng.integers(-254, 255, (T, H)).astype(np.float64)        # peak 254: every odd one is a midpoint
    v[:, 0] = 254
    v *= 2.0 ** rng.integers(-5, 6, (T, 1))
    x = torch.from_numpy(v).to(DEV).to(dt)
    near = f64(x) * (1 + rng.choice([-1, 1], (T, H)) * torch.finfo(dt).eps)
    near[:, 0] = f64(x)[:, 0]
    w = torch.from_numpy(2.0 ** rng.integers(-3, 4, (H,))).to(DEV).to(dt)
    n = P.Norm(H, EPS, act_f16=dt == torch.float16)
    lin = P.Int8Linear(16, H, 16)
    for rows in (x, torch.from_numpy(near).to(DEV).to(dt)):
        for weight in (torch.ones((H,), dtype=dt, device=DEV), w):
            q, s, rstd = torch.empty((T, H), dtype=torch.int8, device=DEV), *(torch.empty((T,), device=DEV) for _ in range(2))
            n.nvfp4_norm_forward(rows, weight, q=q, q_scale=s, rstd=rstd)
            _check(n, rows, None, weight, EPS, None, None, q, s, rstd, dt)
        lin.nvfp4_int8_quantize(rows, q, s)
        qq, peak = codes(f64(rows))
        assert np.array_equal(f64(q), qq)
        within(f64(s), peak / 127.0, U * peak, "scale")
    assert np.any(np.abs(2 * (127 * f64(x) / np.abs(f64(x)).max(1, keepdims=True)) % 2) == 1)
    n.close()
    lin.close()


@pytest.mark.parametrize("H", [64, 256, 4096])
def test_rows_out_of_range(H):
    """Zeros, rows beyond FP32's squares and products, infinities and NaNs, beside ordinary rows."""
    rng = np.random.default_rng(H + 1)
    dt, T = torch.bfloat16, 11
    x, w = _rand(rng, (T, H), dt), _rand(rng, (H,), dt)
    x[1] = 0
    x[2] *= 1e30
    x[3] *= 1e-25
    x[4, H // 2] = float("inf")
    x[5, 0] = float("nan")
    x[6] *= 2.0 ** 100
    x[7] *= 2.0 ** -100
    x[8] = 0
    x[8, H - 1] = 3e-38
    n = P.Norm(H, EPS)
    y, q = torch.empty_like(x), torch.empty((T, H), dtype=torch.int8, device=DEV)
    s, rstd = (torch.empty((T,), device=DEV) for _ in range(2))
    n.nvfp4_norm_forward(x, w, y=y, q=q, q_scale=s, rstd=rstd)
    ok = [0, 1, 2, 3, 6, 7, 8, 9, 10]
    H64, W = f64(x)[ok], f64(w)
    want, rr = norm(H64, W, float(np.float32(EPS)))
    within(f64(rstd)[ok], rr, R_ERR * rr, "rstd")
    b = (R_ERR + 2 * U) * np.abs(want)
    within(f64(y)[ok], want, b + half_step(np.abs(want) + b, dt) + 2.0 ** -149, "y")
    qq, peak = codes(H64 * W)
    assert np.array_equal(f64(q)[ok], qq)
    within(f64(s)[ok], peak * rr / 127.0, (R_ERR + 3 * U) * peak * rr / 127.0 + 2.0 ** -149, "q_scale")
    for t in (4, 5):
        assert bool(torch.isnan(s[t])) and not bool(q[t].any()) and bool(torch.isnan(y[t]).any())
    assert f64(rstd)[4] == 0 and np.isnan(f64(rstd)[5])
    # eps = 0 and a tiny row
    n0 = P.Norm(H, 0.0)
    n0.nvfp4_norm_forward(x[7:8], w, y=y[:1], rstd=rstd[:1])
    want, rr = norm(f64(x[7:8]), W, 0.0)
    within(f64(rstd[:1]), rr, R_ERR * rr, "rstd without eps")
    b = (R_ERR + 2 * U) * np.abs(want)
    within(f64(y[:1]), want, b + half_step(np.abs(want) + b, dt), "y without eps")
    n.close()
    n0.close()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,H", [(1, 8), (5, 64), (37, 120), (300, 256), (65, 512), (7, 1024), (1000, 2048), (3, 4096),
                                 (2000, 4096), (700, 4104), (350, 8192), (330, 16384)])
@pytest.mark.parametrize("dsum", [False, True])
def test_backward(T, H, dt, dsum):
    rng = np.random.default_rng(T + H)
    n = P.Norm(H, EPS, act_f16=dt == torch.float16)
    h, dy, w = _rand(rng, (T, H), dt, 2.0), _rand(rng, (T, H), dt, 2.0 ** -4), _rand(rng, (H,), dt)
    ds = _rand(rng, (T, H), dt, 2.0 ** -4) if dsum else None
    y, rstd = torch.empty_like(h), torch.empty((T,), device=DEV)
    n.nvfp4_norm_forward(h, w, y=y, rstd=rstd)
    dx, dw = torch.full_like(h, 9), torch.full((H,), 9.0, device=DEV)
    n.nvfp4_norm_backward(dy, h, w, rstd, dx, dweight=dw, dsum=ds)
    want, b, want_w, b_w = norm_backward(f64(dy), f64(h), f64(w), f64(rstd), f64(ds) if dsum else 0.0)
    within(f64(dx), want, b + half_step(np.abs(want) + b, dt), "dx")
    within(f64(dw), want_w, b_w + U * np.abs(want_w), "dweight")
    dx2, dw2 = torch.empty_like(h), torch.empty_like(dw)
    n.nvfp4_norm_backward(dy, h, w, rstd, dx2, dsum=ds)               # without dweight, and twice the same
    assert torch.equal(dx2, dx)
    n.nvfp4_norm_backward(dy, h, w, rstd, dx2, dweight=dw2, dsum=ds)
    assert torch.equal(dw2, dw)
    n.close()


def test_gradient_against_differences():
    """The float64 form that the kernel is held to is the derivative of the float64 forward."""
    rng = np.random.default_rng(0)
    h, dy, w = rng.standard_normal((3, 24)), rng.standard_normal((3, 24)), rng.standard_normal(24)
    loss = lambda h, w: (norm(h, w, EPS)[0] * dy).sum()
    dx, _, dw, _ = norm_backward(dy, h, w, norm(h, w, EPS)[1], 0.0)
    for i, j in ((0, 0), (1, 7), (2, 23)):
        e = np.zeros_like(h)
        e[i, j] = 1e-6
        assert abs((loss(h + e, w) - loss(h - e, w)) / 2e-6 - dx[i, j]) < 1e-7
        assert abs((loss(h, w + e[i]) - loss(h, w - e[i])) / 2e-6 - dw[j]) < 1e-7


def test_strides_in_place_and_rows_left_alone():
    rng = np.random.default_rng(5)
    dt, T, H = torch.bfloat16, 50, 1096
    n = P.Norm(H, EPS)
    x, r, w = _rand(rng, (T, H), dt), _rand(rng, (T, H), dt), _rand(rng, (H,), dt)
    want = [torch.empty_like(x), torch.empty_like(x), torch.empty((T, H), dtype=torch.int8, device=DEV), torch.empty((T,), device=DEV)]
    n.nvfp4_norm_forward(x, w, residual=r, sum=want[0], y=want[1], q=want[2], q_scale=want[3])
    wide = lambda t, ld, d=dt: torch.zeros((T + 2, ld), dtype=d, device=DEV)
    bx, br, by, bq = wide(x, H + 8), wide(r, H + 24), wide(x, H + 16), wide(x, H + 40, torch.int8)
    bx[1:T + 1, :H], br[1:T + 1, 8:H + 8] = x, r
    s = torch.zeros((T,), device=DEV)
    view = lambda b, o=0: b[1:T + 1, o:H + o]
    n.nvfp4_norm_forward(view(bx), w, residual=view(br, 8), sum=view(br, 8), y=view(by, 8), q=view(bq, 16), q_scale=s)
    assert torch.equal(view(br, 8), want[0]) and torch.equal(view(by, 8), want[1]) and torch.equal(view(bq, 16), want[2])
    assert torch.equal(s, want[3])
    for b, o in ((br, 8), (by, 8), (bq, 16)):
        b[1:T + 1, o:H + o] = 0
        assert not bool(b.any())
    xx = x.clone()
    n.nvfp4_norm_forward(xx, w, residual=r, sum=xx, y=by[:T, :H])
    assert torch.equal(xx, want[0])
    n.nvfp4_norm_forward(xx, w, y=xx)                                 # y over x
    assert torch.equal(xx, want[1])
    rstd = torch.empty((T,), device=DEV)
    n.nvfp4_norm_forward(want[0], w, y=want[1], rstd=rstd)
    dx = torch.empty_like(x)
    n.nvfp4_norm_backward(x, want[0], w, rstd, dx, dsum=r)
    for arg in ("dy", "dsum"):
        d = {"dy": x.clone(), "dsum": r.clone()}
        n.nvfp4_norm_backward(d["dy"], want[0], w, rstd, d[arg], dsum=d["dsum"])
        assert torch.equal(d[arg], dx)
    n.close()


def test_no_rows():
    n = P.Norm(64, EPS)
    e, w = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV), torch.ones((64,), dtype=torch.bfloat16, device=DEV)
    f = torch.empty((0,), device=DEV)
    n.nvfp4_norm_forward(e, w, y=e)
    dw = torch.ones((64,), device=DEV)
    n.nvfp4_norm_backward(e, e, w, f, e, dweight=dw)
    assert not bool(dw.any())
    n.close()


def test_streams_graphs_and_threads():
    """Captured and replayed with other rows; calls of two threads on streams of their own."""
    rng = np.random.default_rng(6)
    dt, T, H = torch.bfloat16, 300, 2048
    n, m = P.Norm(H, EPS), P.Norm(H, EPS)
    x, r, w, dy = (_rand(rng, s, dt) for s in ((T, H), (T, H), (H,), (T, H)))
    outs = lambda: [torch.empty_like(x), torch.empty_like(x), torch.empty((T,), device=DEV), torch.empty_like(x), torch.empty((H,), device=DEV)]

    def step(n, x, o, stream=None):
        n.nvfp4_norm_forward(x, w, residual=r, sum=o[0], y=o[1], rstd=o[2], stream=stream)
        n.nvfp4_norm_backward(dy, o[0], w, o[2], o[3], dweight=o[4], dsum=x, stream=stream)

    side = torch.cuda.Stream()
    got, want = outs(), outs()
    with torch.cuda.stream(side):
        step(n, x, got)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step(n, x, got)
    for seed in (1, 2):
        x.copy_(_rand(np.random.default_rng(seed), (T, H), dt))
        torch.cuda.synchronize()
        g.replay()
        step(m, x, want)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    ok = [None, None]

    def work(i, h):
        s = torch.cuda.Stream()
        res = []
        with torch.cuda.stream(s):
            for _ in range(30):
                o = outs()
                step(h, x, o, s)
                res.append(o)
            s.synchronize()
        ok[i] = all(torch.equal(a, b) for o in res for a, b in zip(o, want))

    threads = [threading.Thread(target=work, args=(i, h)) for i, h in enumerate((n, m))]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert ok == [True, True]
    n.close()
    m.close()
