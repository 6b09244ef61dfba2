"""The RMS norm's gradient of rows far from 1, where a square of rstd is outside FP32."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import nvfp4_weight_only_w4a16_gb300 as P
from tests.block_ops import DEV, U, f64, half_step, norm_backward, within
from tests.test_gpu_norm import _rand

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
