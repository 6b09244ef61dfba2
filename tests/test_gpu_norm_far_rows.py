"""The RMS norm of rows far from 1: the gradient where a square of rstd is outside FP32, and rows without eps whose rstd is."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import nvfp4_weight_only_w4a16_gb300 as P
from tests.block_ops import DEV, U, codes, f64, half_step, norm, norm_backward, within
from tests.test_gpu_norm import R_ERR, _rand

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    P.build()


# every thread layout; the bounds are test_gpu_norm's, which are relative to the terms that are added
@pytest.mark.parametrize("T,H", [(9, 64), (9, 128), (9, 256), (9, 512), (9, 1024), (9, 2048), (300, 4096), (9, 5120), (9, 8192), (9, 16384)])
@pytest.mark.parametrize("power", [-110, -70, -40, 40, 70, 110])
def test_gradient_of_rows_far_from_one(T, H, power):
    rng = np.random.default_rng(T + H)
    n = P.Norm(H, 0.0)
    h, dy, w = _rand(rng, (T, H), BF16, 2.0 ** power), _rand(rng, (T, H), BF16), _rand(rng, (H,), BF16)
    ds = _rand(rng, (T, H), BF16, 2.0 ** -power)
    y, rstd = torch.empty_like(h), torch.empty((T,), device=DEV)
    n.nvfp4_norm_forward(h, w, y=y, rstd=rstd)
    for dsum in (None, ds):
        dx, dw = torch.empty_like(h), torch.empty((H,), device=DEV)
        n.nvfp4_norm_backward(dy, h, w, rstd, dx, dweight=dw, dsum=dsum)
        want, b, want_w, b_w = norm_backward(f64(dy), f64(h), f64(w), f64(rstd), 0.0 if dsum is None else f64(dsum))
        within(f64(dx), want, b + half_step(np.abs(want) + b, BF16), "dx")
        within(f64(dw), want_w, b_w + U * np.abs(want_w), "dweight")
    n.close()


@pytest.mark.parametrize("H", [8, 64, 128, 256, 1024, 4096, 16384])
@pytest.mark.parametrize("T", [7, 400])
def test_zeros_and_the_smallest_rows_without_eps(T, H):
    """eps = 0: a row of zeros is zeros in 16 and in 8 bits, its scale 0; rows whose rstd is beyond FP32 are as the
    others, but for rstd itself, which is infinite."""
    rng = np.random.default_rng(H)
    n = P.Norm(H, 0.0)
    x, w = _rand(rng, (T, H), BF16), _rand(rng, (H,), BF16)
    x[[0, 3]] = 0
    small = rng.integers(1, 20, (2, H)) * rng.choice([-1, 1], (2, H)) * 2.0 ** -133
    x[1:3] = torch.from_numpy(small).to(DEV).to(BF16)
    y, q = torch.full_like(x, 7), torch.full((T, H), 7, dtype=torch.int8, device=DEV)
    s, rstd = (torch.full((T,), 7.0, device=DEV) for _ in range(2))
    n.nvfp4_norm_forward(x, w, y=y, q=q, q_scale=s, rstd=rstd)
    rest = [t for t in range(T) if t not in (0, 3)]
    H64, W = f64(x)[rest], f64(w)
    want, rr = norm(H64, W, 0.0)
    b = (R_ERR + 2 * U) * np.abs(want)
    within(f64(y)[rest], want, b + half_step(np.abs(want) + b, BF16), "y")
    qq, peak = codes(H64 * W)
    assert np.array_equal(f64(q)[rest], qq)
    within(f64(s)[rest], peak * rr / 127.0, (R_ERR + 3 * U) * peak * rr / 127.0 + 2.0 ** -149, "q_scale")
    within(f64(rstd)[rest], np.where(rr > 3.4e38, np.inf, rr), R_ERR * np.where(rr > 3.4e38, 0.0, rr), "rstd")
    assert np.isinf(f64(rstd)[:4]).all()
    assert not bool(y[[0, 3]].any()) and not bool(q[[0, 3]].any()) and not bool(s[[0, 3]].any())
    y2, q2, s2 = torch.full_like(x, 7), torch.full_like(q, 7), torch.full_like(s, 7.0)
    n.nvfp4_norm_forward(x, w, y=y2)
    n.nvfp4_norm_forward(x, w, q=q2, q_scale=s2)
    assert torch.equal(y2, y) and torch.equal(q2, q) and torch.equal(s2, s)
    n.close()


@pytest.mark.parametrize("dt", [BF16, torch.float16])
@pytest.mark.parametrize("H", [8, 64, 72, 128, 256])
def test_rows_do_not_depend_on_their_neighbours(H, dt):
    """Rows that share a warp with zeros, infinities, NaNs or rows out of range are as they are among ordinary ones."""
    rng = np.random.default_rng(H)
    T = 130
    x, w = _rand(rng, (T, H), dt), _rand(rng, (H,), dt)
    among = x.clone()
    odd = rng.choice(T, T // 3, replace=False)
    for i, v in zip(odd, rng.choice([0.0, float("inf"), float("nan"), 2.0 ** -110, 2.0 ** 110], len(odd))):
        among[i] = among[i].float().mul(v).to(dt) if np.isfinite(v) else torch.full((H,), v, dtype=dt, device=DEV)
    rest = torch.from_numpy(np.setdiff1d(np.arange(T), odd)).to(DEV)
    got = []
    for rows in (x, among):
        y, q = torch.empty_like(x), torch.empty((T, H), dtype=torch.int8, device=DEV)
        s, rstd, s2 = (torch.empty((T,), device=DEV) for _ in range(3))
        n, lin = P.Norm(H, 0.0, act_f16=dt == torch.float16), None
        n.nvfp4_norm_forward(rows, w, y=y, q=q, q_scale=s, rstd=rstd)
        out = [y, q, s, rstd]
        if H % 16 == 0:
            lin, q2 = P.Int8Linear(16, H, 16), torch.empty_like(q)
            lin.nvfp4_int8_quantize(rows, q2, s2)
            out += [q2, s2]
            lin.close()
        got.append([t[rest].clone() for t in out])
        n.close()
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("H", [64, 128, 256, 4096])
def test_rows_do_not_depend_on_what_is_asked_of_them(H):
    """Products beyond what codes are formed of in FP32: y and rstd are the same without the codes."""
    rng = np.random.default_rng(H)
    T = 300
    x, w = _rand(rng, (T, H), BF16), _rand(rng, (H,), BF16, 2.0 ** 105)
    n, got = P.Norm(H, 0.0), []
    for codes_too in (False, True):
        y, rstd = torch.empty_like(x), torch.empty((T,), device=DEV)
        q, s = torch.empty((T, H), dtype=torch.int8, device=DEV), torch.empty((T,), device=DEV)
        n.nvfp4_norm_forward(x, w, y=y, rstd=rstd, **(dict(q=q, q_scale=s) if codes_too else {}))
        got.append((y, rstd))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    want, rr = norm(f64(x), f64(w), 0.0)
    qq, peak = codes(f64(x) * f64(w))
    assert np.array_equal(f64(q), qq)
    within(f64(s), peak * rr / 127.0, (R_ERR + 3 * U) * peak * rr / 127.0, "q_scale")
    n.close()
