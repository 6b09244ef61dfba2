"""The INT8 linear: equal to the definition to the bit.  The sum of products is exact, so the only roundings are the
stated ones: of the sum and of the scales' product to FP32, of their product with the bias added, and to the type."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import nvfp4_weight_only_w4a16_gb300 as P
from tests.block_ops import DEV, codes, dev, f64

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def built():
    P.build()


def _want(x, w, sx, sw, bias, out):
    """In torch on the GPU: an exact integer sum (float64 products of integers), the stated roundings."""
    acc = (x.double() @ w.double().t()).float()
    y = acc.double() * (sx[:, None] * sw).double()      # exact: 24 + 24 bits
    if bias is not None:
        y = y + bias.double()                           # off by 2^-53 before the rounding to 2^-24
    return y.float().to(TYPES[out])


def _case(seed, N, K, T, bias=True, kind="random"):
    g = torch.Generator(device=DEV).manual_seed(seed)
    ri = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device=DEV, dtype=torch.int32).to(torch.int8)
    if kind == "random":
        x, w = ri(-128, 128, T, K), ri(-128, 128, N, K)
    else:                                               # the largest sums there are: all of one sign, or nearly cancelling
        x, w = torch.full((T, K), -128, dtype=torch.int8, device=DEV), torch.full((N, K), -128, dtype=torch.int8, device=DEV)
        if kind == "cancel":
            w[:, K // 2:] = 127
            x[::2] = 127
            w[:, -1] = ri(-128, 128, N)
    sx = torch.rand((T,), generator=g, device=DEV) * 0.01 + 1e-4
    sw = torch.rand((N,), generator=g, device=DEV) * 0.01 - 0.002
    b = torch.randn((N,), generator=g, device=DEV) if bias else None
    return x, w, sx, sw, b


def _run(N, K, T, out, seed=0, bias=True, kind="random", max_tokens=None):
    x, w, sx, sw, b = _case(seed, N, K, T, bias, kind)
    h = P.Int8Linear(N, K, max_tokens or T, out=out)
    h.nvfp4_int8_pack(w, sw, b)
    y = torch.full((T, N), 7.0, dtype=TYPES[out], device=DEV)
    h.nvfp4_int8_forward(x, sx, y)
    assert h.nvfp4_moe_get_status()[0] == 0
    h.close()
    want = _want(x, w, sx, sw, b, out)
    assert torch.equal(y, want), (f64(y) - f64(want), int((y != want).sum()))


# few tokens: every count; slices, passes, streams and batches of the rows, and rows that fill none
@pytest.mark.parametrize("N,K", [(16, 16), (16, 1024), (272, 256), (48, 48), (1040, 4096), (4096, 4096), (80, 16384),
                                 (2000, 7168), (128, 5136), (12576, 272), (65536, 64), (32768, 528)])
@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16])
def test_few_tokens(N, K, T):
    _run(N, K, T, ("bf16", "f16", "f32")[(N + T) % 3], seed=N + K + T, bias=T % 2 == 0)


# tcgen05: tiles of 64 and 128 and pairs of 192, split and whole, odd numbers of blocks, short and long reductions
@pytest.mark.parametrize("N,K,T", [
    (16, 16, 17), (128, 128, 64), (272, 256, 37), (144, 80, 100), (4096, 4096, 17), (4096, 4096, 64), (4096, 4096, 100),
    (1040, 16384, 33), (4096, 1040, 129), (12576, 4096, 48), (12576, 512, 130), (528, 2064, 1000), (4096, 4096, 1025),
    (2320, 1552, 5000), (16, 4096, 20000), (65536, 256, 200), (144, 272, 40000), (4096, 16384, 600)])
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
def test_more_tokens(N, K, T, out):
    _run(N, K, T, out, seed=N + K + T, bias=(N // 16) % 2 == 0)


@pytest.mark.parametrize("kind", ["largest", "cancel"])
@pytest.mark.parametrize("K", [1024, 1040, 4096, 16384])
@pytest.mark.parametrize("T", [3, 16, 40, 200, 3000])
def test_the_largest_sums_are_exact(K, T, kind):
    _run(400, K, T, "f32", seed=K, bias=False, kind=kind)


def test_scales_that_are_zero_infinite_or_nan():
    for T in (5, 70):
        N, K = 64, 128
        x, w, sx, sw, b = _case(1, N, K, T)
        sw[3] = 0
        sx[0], sx[1], sx[2] = 0, float("nan"), float("inf")
        h = P.Int8Linear(N, K, T, out="f32")
        h.nvfp4_int8_pack(w, sw, None)
        y = torch.empty((T, N), device=DEV)
        h.nvfp4_int8_forward(x, sx, y)
        want = _want(x, w, sx, sw, None, "f32")
        assert torch.equal(torch.isnan(y), torch.isnan(want)) and torch.equal(torch.nan_to_num(y), torch.nan_to_num(want))
        assert bool(torch.isnan(y[1]).all())
        for bad in (float("nan"), float("inf"), -float("inf")):
            sw2 = sw.clone()
            sw2[N - 1] = bad
            with pytest.raises(P.Nvfp4MoeError, match="BAD_SCALE"):
                h.nvfp4_int8_pack(w, sw2, None)
            with pytest.raises(P.Nvfp4MoeError, match="NOT_PACKED"):
                h.nvfp4_int8_forward(x, sx, y)
        h.nvfp4_int8_pack(w, sw, b)
        h.nvfp4_int8_forward(x, sx, y)
        ok = torch.isfinite(sx)
        assert torch.equal(y[ok], _want(x, w, sx, sw, b, "f32")[ok])
        h.close()


@pytest.mark.parametrize("T", [1, 13, 77, 500])
def test_strides_and_rows_left_alone(T):
    N, K = 272, 400
    x, w, sx, sw, b = _case(2, N, K, T)
    h = P.Int8Linear(N, K, 600)
    h.nvfp4_int8_pack(w, sw, b)
    want = torch.empty((T, N), dtype=torch.bfloat16, device=DEV)
    h.nvfp4_int8_forward(x, sx, want)
    xs = torch.full((T + 1, K + 48), 55, dtype=torch.int8, device=DEV)
    xs[:T, 16:K + 16] = x
    ys = torch.zeros((T + 2, N + 24), dtype=torch.bfloat16, device=DEV)
    h.nvfp4_int8_forward(xs[:T, 16:K + 16], sx, ys[1:T + 1, 8:N + 8])
    assert torch.equal(ys[1:T + 1, 8:N + 8], want)
    ys[1:T + 1, 8:N + 8] = 0
    assert not bool(ys.any())
    e = torch.empty((0, K), dtype=torch.int8, device=DEV)
    h.nvfp4_int8_forward(e, sx[:0], ys[:0, :N])
    h.close()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,K", [(1, 16), (3, 1040), (16, 4096), (500, 272), (330, 16384)])
def test_quantize(T, K, dt):
    rng = np.random.default_rng(T + K)
    x = torch.from_numpy(rng.standard_normal((T, K))).to(DEV).to(dt)
    if T > 2:
        x[1] = 0
        x[2, 5] = float("nan")
    h = P.Int8Linear(16, K, 16)
    q, s = torch.full((T, K), 9, dtype=torch.int8, device=DEV), torch.empty((T,), device=DEV)
    h.nvfp4_int8_quantize(x, q, s)
    ok = np.isfinite(f64(x)).all(axis=1)
    qq, peak = codes(f64(x)[ok])
    assert np.array_equal(f64(q)[ok], qq)
    assert np.array_equal(f64(s)[ok], (peak.astype(np.float32) / np.float32(127)).astype(np.float64))
    assert np.isnan(f64(s)[~ok]).all() and not f64(q)[~ok].any()
    h.close()


@pytest.mark.parametrize("T", [5, 60, 300])
def test_graph_overlapping_calls_and_both_paths_alike(T):
    N, K = 1040, 1536
    x, w, sx, sw, b = _case(3, N, K, T)
    h = P.Int8Linear(N, K, T)
    h.nvfp4_int8_pack(w, sw, b)
    out = lambda: torch.empty((T, N), dtype=torch.bfloat16, device=DEV)
    y = out()
    h.nvfp4_int8_forward(x, sx, y)                      # sets the kernels' attributes before the capture
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            h.nvfp4_int8_forward(x, sx, y)
    for seed in (4, 5):
        x2, _, sx2, _, _ = _case(seed, N, K, T)
        x.copy_(x2)
        sx.copy_(sx2)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, _want(x, w, sx, sw, b, "bf16"))
    streams = [torch.cuda.Stream() for _ in range(4 if T <= 64 else 1)]   # above 64 tokens calls share a workspace
    outs = [[out() for _ in range(8)] for _ in streams]
    torch.cuda.synchronize()
    for i in range(8):
        for s, o in zip(streams, outs):
            h.nvfp4_int8_forward(x, sx, o[i], stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(v, y) for o in outs for v in o)
    # the same rows in calls of 16 and fewer
    z = out()
    for t in range(0, T, 16):
        h.nvfp4_int8_forward(x[t:t + 16], sx[t:t + 16], z[t:t + 16])
    assert torch.equal(z, y)
    h.close()


@pytest.mark.parametrize("T,N,K", [(40, 1040, 4096), (100, 4096, 512), (3000, 528, 512)])
def test_bounded_waits(T, N, K):
    """Copies that are never issued: the kernel gives up, says so, and the next call is right."""
    x, w, sx, sw, b = _case(6, N, K, T)
    h = P.Int8Linear(N, K, T)
    h.nvfp4_int8_pack(w, sw, b)
    y = torch.zeros((T, N), dtype=torch.bfloat16, device=DEV)
    h.nvfp4_moe_debug_set_fault(1)
    h.nvfp4_int8_forward(x, sx, y)
    with_status = h.nvfp4_moe_get_status()
    h.nvfp4_moe_debug_set_fault(0)
    assert P.STATUS[with_status[0]] == "NVFP4_MOE_ERR_TIMEOUT"
    h.nvfp4_int8_forward(x, sx, y)
    assert h.nvfp4_moe_get_status()[0] == 0
    assert torch.equal(y, _want(x, w, sx, sw, b, "bf16"))
    h.close()


def test_packed_bytes():
    """[N / 128][K / 16][128][16] bytes q + 128, filled up with q = 0."""
    N, K = 272, 400
    _, w, _, sw, _ = _case(7, N, K, 1)
    h = P.Int8Linear(N, K, 1)
    h.nvfp4_int8_pack(w, sw)
    full = np.zeros((384, 512), np.int64)
    full[:N, :K] = w.cpu().numpy()
    want = (full + 128).astype(np.uint8).reshape(3, 128, 32, 16).transpose(0, 2, 1, 3).reshape(-1)
    assert np.array_equal(h.nvfp4_moe_debug_packed_blob().cpu().numpy(), want)
    h.close()
