"""The INT4 linear with group scales, on the GPU, against float64.

out[t][n] = sum_k s[n][k/g] (q[n][k] - z[n][k/g]) x[t][k] for every group size,
activation type, token count and both symmetric and asymmetric codes, at sizes
from one 16-row group to K beyond what shared memory holds at once.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import nvfp4_weight_only_w4a16_gb300 as P
from tests.products import DEV, bound, check, f64, int4_values

pytestmark = pytest.mark.gpu
CODE = P.STATUS_CODE


class Matrix:
    def __init__(self, N, K, group, zeros, f16, out_f32=False, seed=0, max_tokens=16):
        P.build()
        rng = np.random.default_rng(seed)
        t = torch.float16 if f16 else torch.bfloat16
        q = torch.from_numpy(rng.integers(0, 256, (N, K // 2), dtype=np.uint8)).to(DEV)
        scale = torch.from_numpy(rng.uniform(-0.1, 0.1, (N, K // group))).to(DEV).to(t)
        zero = torch.from_numpy(rng.integers(0, 16, (N, K // group), dtype=np.uint8)).to(DEV) if zeros else None
        self.set_values(q, scale, zero, group)
        self.h = P.Int4Linear(N, K, group, max_tokens=max_tokens, act_f16=f16, out_f32=out_f32)
        self.h.nvfp4_int4_pack(q, scale, zero)
        self.N, self.K, self.act, self.dtype = N, K, t, torch.float32 if out_f32 else t


    def set_values(self, q, scale, zero, group):
        q, scale, zero = q.cpu().numpy(), f64(scale), None if zero is None else zero.cpu().numpy()
        self.w = int4_values(q, scale, zero, group)
        self.terms = int4_values(q, scale, zero, group, sign=1.0)


def rows_of(m, T, seed=1, pad=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn((T, m.K + pad), generator=g, device=DEV).to(m.act)[:, :m.K]


def run(m, x, pad=0, stream=None):
    T = x.shape[0]
    buf = torch.full((T + 2, m.N + pad), float("nan"), dtype=m.dtype, device=DEV)
    m.h.nvfp4_int4_forward(x, buf[1:T + 1, :m.N], stream=stream)
    torch.cuda.synchronize()
    assert bool(torch.isnan(buf[0]).all()) and bool(torch.isnan(buf[-1]).all()), "wrote outside out"
    assert not pad or bool(torch.isnan(buf[:, m.N:]).all()), "wrote between rows"
    return buf[1:T + 1, :m.N]


def verify(m, x, got):
    y = f64(x) @ m.w.T
    check(f64(got), y, bound(y, f64(x), m.w, m.dtype, fp16_rows=2.0 ** -34, terms=m.terms, rounds=2))


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T", [1, 3, 8, 9, 16])
def test_small(T, group, zeros, f16):
    m = Matrix(272, 640, group, zeros, f16)
    x = rows_of(m, T)
    verify(m, x, run(m, x))


@pytest.mark.parametrize("N,K", [(16, 128), (48, 256), (16, 16384), (4112, 128), (80, 4224), (32, 8320)])
@pytest.mark.parametrize("T", [2, 13])
def test_shapes(N, K, T):
    m = Matrix(N, K, 64, True, False, out_f32=True)
    x = rows_of(m, T)
    verify(m, x, run(m, x))


@pytest.mark.parametrize("T,N,K,group,f16", [(16, 4848, 4096, 32, False), (16, 1056, 8320, 32, True), (9, 304, 4224, 64, True),
                                             (16, 208, 16384, 32, False), (8, 272, 16384, 128, False), (10, 16, 2560, 64, True),
                                             (5, 96, 12416, 32, True), (16, 2080, 2176, 128, False)])
@pytest.mark.parametrize("out_f32", [False, True])
def test_rows_that_share_a_cluster(T, N, K, group, f16, out_f32):
    m = Matrix(N, K, group, True, f16, out_f32=out_f32)
    x = rows_of(m, T)
    x *= torch.exp2(torch.arange(K, device=DEV) // 128 % 5 - 2.0).to(m.act)    # slices of different size
    got = run(m, x)
    verify(m, x, got)
    assert torch.equal(got, run(m, x))


def test_wide_matrix():
    m = Matrix(12576, 4096, 128, True, False)
    x = rows_of(m, 2)
    verify(m, x, run(m, x))


def test_rows_apart():
    m = Matrix(144, 384, 32, False, True)
    x = rows_of(m, 5, pad=24)
    verify(m, x, run(m, x, pad=40))


def test_non_finite_rows_stay_in_their_rows():
    m = Matrix(64, 256, 128, True, False, out_f32=True)
    x = rows_of(m, 12)
    clean = run(m, x)
    x[2, 7], x[11, 0] = float("nan"), float("inf")
    got = run(m, x)
    keep = [0, 1, 3, 4, 5, 6, 7, 8, 9, 10]
    assert torch.equal(got[keep], clean[keep])
    assert bool(torch.isnan(got[2]).all()) and not bool(torch.isfinite(got[11]).any())


def test_fp16_results_beyond_its_range_are_infinite():
    m = Matrix(16, 128, 128, False, True)
    x = torch.full((1, 128), 60000.0, dtype=torch.float16, device=DEV)
    x[0, 1::2] = -60000.0
    y = f64(x) @ m.w.T
    got = f64(run(m, x))
    over = np.abs(y) > 65600
    assert over.any() and np.all(np.isinf(got[over])) and np.all(np.sign(got[over]) == np.sign(y[over]))


def test_captured_and_on_two_streams():
    m = Matrix(512, 512, 64, True, False)
    x, out = rows_of(m, 4), torch.empty((4, 512), dtype=m.dtype, device=DEV)
    m.h.nvfp4_int4_forward(x, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.h.nvfp4_int4_forward(x, out)
    x.copy_(rows_of(m, 4, seed=7))
    graph.replay()
    torch.cuda.synchronize()
    verify(m, x, out)
    jobs = [(rows_of(m, T, T), torch.empty((T, 512), dtype=m.dtype, device=DEV), torch.cuda.Stream()) for T in (1, 8, 16)]
    torch.cuda.synchronize()
    for a, b, s in jobs:
        m.h.nvfp4_int4_forward(a, b, stream=s)
    torch.cuda.synchronize()
    for a, b, _ in jobs:
        verify(m, a, b)


@pytest.mark.parametrize("T,K", [(3, 512), (16, 8320)])   # one CTA a slice, and a cluster
def test_bounded_wait_reports_a_timeout(T, K):
    m = Matrix(272, K, 64, True, False)
    x = rows_of(m, T)
    m.h.nvfp4_moe_debug_set_fault(1)
    m.h.nvfp4_int4_forward(x, torch.empty((T, 272), dtype=m.dtype, device=DEV))
    assert P.STATUS[m.h.nvfp4_moe_get_status()[0]] == "NVFP4_MOE_ERR_TIMEOUT"
    m.h.nvfp4_moe_debug_set_fault(0)
    verify(m, x, run(m, x))
    assert m.h.nvfp4_moe_get_status()[0] == 0


def test_packing_again_replaces_the_zero_points():
    m = Matrix(32, 256, 64, True, False)
    rng = np.random.default_rng(5)
    q = torch.from_numpy(rng.integers(0, 256, (32, 128), dtype=np.uint8)).to(DEV)
    scale = torch.from_numpy(rng.uniform(0.01, 0.1, (32, 4))).to(DEV).to(torch.bfloat16)
    m.h.nvfp4_int4_pack(q, scale)
    m.set_values(q, scale, None, 64)
    x = rows_of(m, 3)
    verify(m, x, run(m, x))


def test_refusals():
    m = Matrix(32, 256, 64, False, False, max_tokens=8)
    h, lib = m.h, m.h.lib
    x, out = rows_of(m, 8), torch.empty((8, 32), dtype=m.dtype, device=DEV)
    ptr, st = P.binding._ptr, P.binding._stream()
    inv, shape = CODE["NVFP4_MOE_ERR_INVALID_ARG"], CODE["NVFP4_MOE_ERR_UNSUPPORTED_SHAPE"]
    call = lambda T=8, xp=ptr(x), ldx=256, op=ptr(out), ldo=32: lib.nvfp4_int4_forward(h.h, T, xp, ldx, op, ldo, st)
    assert call() == 0
    assert call(T=0) == shape and call(T=9) == shape
    assert call(xp=None) == inv and call(op=None) == inv
    assert call(ldx=248) == inv and call(ldx=257) == inv and call(ldo=24) == inv
    assert call(xp=P.binding.ctypes.c_void_p(x.data_ptr() + 2)) == inv
    for bad in (x.half(), x.t(), x[:, :128]):
        with pytest.raises(ValueError):
            h.nvfp4_int4_forward(bad, out)
    assert lib.nvfp4_linear_forward(h.h, 4, ptr(x), ptr(out), st) == inv
    assert lib.nvfp4_moe_forward(h.h, ptr(x), 4, 1, ptr(x), ptr(out), st) == inv
    fresh = P.Int4Linear(32, 256, 64)
    with pytest.raises(P.Nvfp4MoeError) as ei:
        fresh.nvfp4_int4_forward(x, out)
    assert ei.value.status == CODE["NVFP4_MOE_ERR_NOT_PACKED"]
    q = torch.zeros((32, 128), dtype=torch.uint8, device=DEV)
    good = torch.ones((32, 4), dtype=torch.bfloat16, device=DEV)
    zero = torch.zeros((32, 4), dtype=torch.uint8, device=DEV)
    for v in (float("nan"), float("inf"), float("-inf")):
        s = good.clone()
        s[31, 3] = v
        with pytest.raises(P.Nvfp4MoeError) as ei:
            fresh.nvfp4_int4_pack(q, s)
        assert ei.value.status == CODE["NVFP4_MOE_ERR_BAD_SCALE"]
    zero[7, 1] = 16
    with pytest.raises(P.Nvfp4MoeError) as ei:
        fresh.nvfp4_int4_pack(q, good, zero)
    assert ei.value.status == CODE["NVFP4_MOE_ERR_BAD_SCALE"]
    with pytest.raises(P.Nvfp4MoeError):
        fresh.nvfp4_int4_forward(x, out)     # still unpacked
