"""Grouped NVFP4 products and their input gradient, on the GPU, against float64.

out[r] = gs_e W_e x[r] and dx[r] = gs_e W_e^T dy[r] for the rows of each expert,
at the row counts and sizes where they can go wrong: no rows, one row, tiles'
edges, matrices that are no multiple of 128 rows, experts without rows, rows
outside every expert, strided rows, non-finite rows beside finite ones.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import nvfp4_weight_only_w4a16_gb300 as P
from tests.products import DEV, bound, check, f64, nvfp4, nvfp4_values

pytestmark = pytest.mark.gpu
FORWARD = [P.PATH_DECODE, P.PATH_PREFILL]
FP16_ROWS = {P.PATH_DECODE: 2.0 ** -38, P.PATH_PREFILL: 0.0}   # the streaming kernel multiplies FP16 rows
CODE = P.STATUS_CODE


class Experts:
    """A packed handle and its float64 matrices."""

    def __init__(self, E, N, K, max_rows, seed=0, out_f32=False):
        P.build()
        rng = np.random.default_rng(seed)
        q, s = nvfp4(rng, E, N, K)
        gs = rng.uniform(0.25, 4.0, E).astype(np.float32)
        self.w = nvfp4_values(q, s) * gs.astype(np.float64)[:, None, None]
        self.h = P.Grouped(E, N, K, max_rows, out_f32=out_f32)
        self.h.nvfp4_grouped_pack(*(torch.from_numpy(a).to(DEV) for a in (q, s, gs)))
        self.E, self.N, self.K = E, N, K
        self.dtype = torch.float32 if out_f32 else torch.bfloat16


def offsets_of(counts, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(counts)]).astype(np.int32), device=DEV)


def rows_of(R, n, seed=1, pad=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    wide = torch.randn((R, n + pad), generator=g, device=DEV)
    wide *= torch.exp2(torch.randint(-6, 7, (R, 1), generator=g, device=DEV).float())  # rows of different size
    return wide.to(torch.bfloat16)[:, :n]


def blank(R, n, dtype, pad=0):
    return torch.full((R, n + pad), float("nan"), dtype=dtype, device=DEV)[:, :n]


def status_ok(h):
    st, _ = h.nvfp4_moe_get_status()
    assert st == 0, (P.STATUS[st], h.lib.nvfp4_moe_last_error(h.h).decode())


def verify(ex, counts, got, x, backward, first=0, fp16_rows=0.0):
    got, x = f64(got), f64(x)
    r = first
    for e, m in enumerate(counts):
        if m:
            w = ex.w[e].T if backward else ex.w[e]
            y = x[r:r + m] @ w.T
            check(got[r:r + m], y, bound(y, x[r:r + m], w, ex.dtype, fp16_rows), f"expert {e}")
        r += m
    assert np.all(np.isnan(got[:first])) and np.all(np.isnan(got[r:])), "wrote rows of no expert"


CASES = [
    (1, 16, 128, [1]),
    (1, 16, 128, [0]),
    (1, 128, 128, [16]),
    (3, 272, 256, [0, 5, 0]),
    (4, 128, 256, [17, 16, 15, 1]),
    (8, 256, 512, [3, 0, 9, 1, 8, 0, 4, 7]),
    (5, 400, 384, [257, 0, 1, 300, 64]),
    (2, 144, 1024, [600, 33]),
    (1, 1040, 4224, [19]),
    (256, 48, 128, [1 if e % 3 else 0 for e in range(255)] + [70]),
    # averages and numbers of feature blocks that lead to each tile of the GEMM, one CTA and two
    (3, 128, 128, [40, 128, 31]),
    (3, 272, 256, [129, 1, 60]),
    (2, 96, 384, [300, 90]),
    (2, 528, 128, [0, 513]),
]


@pytest.mark.parametrize("out_f32", [False, True])
@pytest.mark.parametrize("path", FORWARD)
@pytest.mark.parametrize("E,N,K,counts", CASES)
def test_forward(E, N, K, counts, path, out_f32):
    R = sum(counts) + 3
    ex = Experts(E, N, K, R, out_f32=out_f32)
    ex.h.nvfp4_moe_set_path(path)
    x, out = rows_of(R, K), blank(R, N, ex.dtype)
    ex.h.nvfp4_grouped_forward(x, offsets_of(counts), out)
    status_ok(ex.h)
    verify(ex, counts, out, x, False, fp16_rows=FP16_ROWS[path])


@pytest.mark.parametrize("out_f32", [False, True])
@pytest.mark.parametrize("E,N,K,counts", CASES)
def test_backward(E, N, K, counts, out_f32):
    R = sum(counts) + 3
    ex = Experts(E, N, K, R, out_f32=out_f32)
    dy, dx = rows_of(R, N), blank(R, K, ex.dtype)
    ex.h.nvfp4_grouped_backward(dy, offsets_of(counts), dx)
    status_ok(ex.h)
    verify(ex, counts, dx, dy, True)


@pytest.mark.parametrize("path", FORWARD)
def test_rows_apart_and_a_first_offset(path):
    counts, first = [4, 0, 21], 2
    R = first + sum(counts) + 1
    ex = Experts(3, 144, 256, R)
    ex.h.nvfp4_moe_set_path(path)
    off = offsets_of(counts, first)
    x, out = rows_of(R, 256, pad=40), blank(R, 144, ex.dtype, pad=24)
    ex.h.nvfp4_grouped_forward(x, off, out)
    dy, dx = rows_of(R, 144, pad=8), blank(R, 256, ex.dtype, pad=64)
    ex.h.nvfp4_grouped_backward(dy, off, dx)
    status_ok(ex.h)
    verify(ex, counts, out, x, False, first, fp16_rows=FP16_ROWS[path])
    verify(ex, counts, dx, dy, True, first)
    for t, n in ((out, 144), (dx, 256)):   # the gaps between rows are not written
        whole = torch.as_strided(t, (R, t.stride(0) - n), (t.stride(0), 1), n)[:-1]
        assert bool(torch.isnan(whole).all())


@pytest.mark.parametrize("path", FORWARD)
def test_non_finite_rows_stay_in_their_rows(path):
    counts = [3, 5]
    ex = Experts(2, 128, 256, 9, out_f32=True)
    ex.h.nvfp4_moe_set_path(path)
    off = offsets_of(counts)
    for wi, run in ((256, ex.h.nvfp4_grouped_forward), (128, ex.h.nvfp4_grouped_backward)):
        x = rows_of(9, wi)
        clean = blank(9, 384 - wi, ex.dtype)
        run(x, off, clean)
        x[1, 5], x[4, 0], x[8] = float("nan"), float("inf"), float("nan")   # row 8 belongs to no expert
        got = blank(9, 384 - wi, ex.dtype)
        run(x, off, got)
        keep = [0, 2, 3, 5, 6, 7]
        assert torch.equal(got[keep], clean[keep])
        assert bool(torch.isnan(got[1]).all()) and not bool(torch.isfinite(got[4]).any())
    status_ok(ex.h)


def test_an_infinity_keeps_its_sign_beside_large_values():
    ex = Experts(1, 128, 128, 1, out_f32=True)
    ex.h.nvfp4_moe_set_path(P.PATH_DECODE)
    x = torch.full((1, 128), 3e38, dtype=torch.bfloat16, device=DEV)
    x[0, 1::2] = -3e38
    x[0, 7] = float("inf")
    out = blank(1, 128, ex.dtype)
    ex.h.nvfp4_grouped_forward(x, offsets_of([1]), out)
    got, w = f64(out)[0], ex.w[0][:, 7]
    assert np.all(np.isnan(got[w == 0])) and np.all(got[w > 0] == np.inf) and np.all(got[w < 0] == -np.inf)


@pytest.mark.parametrize("path", FORWARD)
def test_repeatable(path):
    counts = [40, 3, 0, 90]
    ex = Experts(4, 256, 512, 133)
    ex.h.nvfp4_moe_set_path(path)
    x, off = rows_of(133, 512), offsets_of(counts)
    a, b = (ex.h.nvfp4_grouped_forward(x, off, blank(133, 256, ex.dtype)) for _ in range(2))
    assert torch.equal(a, b)


@pytest.mark.parametrize("bad", [[0, 5, 3], [-1, 2, 4], [0, 4, 9], [3, 2, 1]])
def test_bad_offsets_compute_nothing(bad):
    ex = Experts(2, 128, 128, 8)
    off = torch.tensor(bad, dtype=torch.int32, device=DEV)
    x = rows_of(8, 128)
    for path in FORWARD:
        ex.h.nvfp4_moe_set_path(path)
        for run in (ex.h.nvfp4_grouped_forward, ex.h.nvfp4_grouped_backward):
            out = blank(8, 128, ex.dtype)
            run(x, off, out)
            st, _ = ex.h.nvfp4_moe_get_status()
            assert P.STATUS[st] == "NVFP4_MOE_ERR_DEVICE_CHECK"
            assert bool(torch.isnan(out).all())
    status_ok(ex.h)                        # read and cleared


def test_no_rows():
    ex = Experts(2, 128, 256, 4)
    x, out = rows_of(0, 256), blank(0, 128, ex.dtype)
    ex.h.nvfp4_grouped_forward(x, offsets_of([0, 0]), out)
    ex.h.nvfp4_grouped_backward(out, offsets_of([0, 0]), torch.empty_like(x))
    status_ok(ex.h)


@pytest.mark.parametrize("path", FORWARD)
def test_captured_and_replayed_with_other_rows_and_offsets(path):
    ex = Experts(3, 256, 256, 60)
    ex.h.nvfp4_moe_set_path(path)
    x, out, dx = rows_of(60, 256), blank(60, 256, ex.dtype), blank(60, 256, ex.dtype)
    off = offsets_of([20, 20, 20])
    ex.h.nvfp4_grouped_forward(x, off, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ex.h.nvfp4_grouped_forward(x, off, out)
        ex.h.nvfp4_grouped_backward(x, off, dx)
    for seed, counts in ((3, [1, 0, 50]), (4, [0, 0, 0]), (5, [60, 0, 0])):
        x.copy_(rows_of(60, 256, seed))
        off.copy_(offsets_of(counts))
        out.fill_(float("nan"))
        dx.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        verify(ex, counts, out, x, False, fp16_rows=FP16_ROWS[path])
        verify(ex, counts, dx, x, True)
    status_ok(ex.h)


def test_two_streams_share_a_handle():
    ex = Experts(4, 512, 1024, 400)
    jobs = []
    for i, path in enumerate((P.PATH_PREFILL, P.PATH_DECODE) * 3):
        counts = [10 + i, 0, 33 * i, 5]
        R = sum(counts)
        jobs.append((path, counts, rows_of(R, 1024, i), offsets_of(counts), blank(R, 512, ex.dtype), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for path, counts, x, off, out, stream in jobs:
        ex.h.nvfp4_moe_set_path(path)
        ex.h.nvfp4_grouped_forward(x, off, out, stream=stream)
    torch.cuda.synchronize()
    status_ok(ex.h)
    for path, counts, x, off, out, stream in jobs:
        verify(ex, counts, out, x, False, fp16_rows=FP16_ROWS[path])


def test_output_offsets_beyond_32_bits():
    R, ld = 132000, 16384   # element offsets up to 2.16e9
    ex = Experts(1, 16, 128, R)
    x = rows_of(R, 128)
    buf = torch.empty((R, ld), dtype=torch.bfloat16, device=DEV)
    out = buf[:, :16]
    ex.h.nvfp4_grouped_forward(x, offsets_of([R]), out)
    status_ok(ex.h)
    for r in (slice(0, 300), slice(131000, R)):
        y = f64(x[r]) @ ex.w[0].T
        check(f64(out[r]), y, bound(y, f64(x[r]), ex.w[0], ex.dtype))
    ex.h.nvfp4_grouped_backward(out, offsets_of([R]), buf[:, 64:192])
    status_ok(ex.h)
    dy = f64(out[131000:])
    dx = dy @ ex.w[0]
    check(f64(buf[131000:, 64:192]), dx, bound(dx, dy, ex.w[0].T, ex.dtype))


def test_backward_is_the_gradient():
    """<dy, F(x + h) - F(x)> = <dx, h>: the product is linear, so differences are exact up to roundings."""
    counts = [7, 0, 130]
    R = sum(counts)
    ex = Experts(3, 272, 384, R, out_f32=True)
    off = offsets_of(counts)
    x, h, dy = rows_of(R, 384, 1), rows_of(R, 384, 2), rows_of(R, 272, 3)
    xh = (x.float() + h.float()).to(torch.bfloat16)
    y0, y1 = (ex.h.nvfp4_grouped_forward(v, off, blank(R, 272, ex.dtype)) for v in (x, xh))
    dx = ex.h.nvfp4_grouped_backward(dy, off, blank(R, 384, ex.dtype))
    step = f64(xh) - f64(x)
    left, right, slack, r = 0.0, 0.0, 0.0, 0
    left = float(np.sum(f64(dy) * (f64(y1) - f64(y0))))
    right = float(np.sum(f64(dx) * step))
    for e, m in enumerate(counts):
        s = slice(r, r + m)
        w, a = ex.w[e], np.abs(f64(dy)[s])
        for v in (x, xh):
            slack += float(np.sum(a * bound(None, f64(v)[s], w, torch.float32)))
        slack += float(np.sum(np.abs(step[s]) * bound(None, f64(dy)[s], w.T, torch.float32)))
        r += m
    assert abs(left - right) <= slack, (left, right, slack)


def test_bounded_wait_reports_a_timeout():
    ex = Experts(2, 128, 256, 40)
    ex.h.nvfp4_moe_set_path(P.PATH_PREFILL)
    x, off, counts = rows_of(40, 256), offsets_of([30, 10]), [30, 10]
    ex.h.nvfp4_moe_debug_set_fault(1)
    ex.h.nvfp4_grouped_forward(x, off, blank(40, 128, ex.dtype))
    st, _ = ex.h.nvfp4_moe_get_status()
    assert P.STATUS[st] == "NVFP4_MOE_ERR_TIMEOUT"
    ex.h.nvfp4_moe_debug_set_fault(0)
    out = ex.h.nvfp4_grouped_forward(x, off, blank(40, 128, ex.dtype))
    status_ok(ex.h)
    verify(ex, counts, out, x, False)


@pytest.mark.parametrize("path,N,K", [(P.PATH_DECODE, 48, 16384), (P.PATH_PREFILL, 48, 16384), (P.PATH_PREFILL, 16384, 128)])
def test_the_longest_sums(path, N, K):
    counts = [9, 1, 20]
    ex = Experts(3, N, K, 30, out_f32=True)
    ex.h.nvfp4_moe_set_path(path)
    x, dy, off = rows_of(30, K), rows_of(30, N), offsets_of(counts)
    out = ex.h.nvfp4_grouped_forward(x, off, blank(30, N, ex.dtype))
    dx = ex.h.nvfp4_grouped_backward(dy, off, blank(30, K, ex.dtype))
    status_ok(ex.h)
    verify(ex, counts, out, x, False, fp16_rows=FP16_ROWS[path])
    verify(ex, counts, dx, dy, True)


@pytest.mark.parametrize("counts", [[30, 0, 34, 17], [100, 130, 3, 60], [256, 700, 1, 90]])   # each tile of the GEMM
@pytest.mark.parametrize("out_f32", [False, True])
def test_many_units_a_multiprocessor(counts, out_f32):
    """Rings that wrap many times: right, and the same bits each time."""
    ex = Experts(4, 2064, 2048, 1100, out_f32=out_f32)
    ex.h.nvfp4_moe_set_path(P.PATH_PREFILL)
    R = sum(counts)
    off = offsets_of(counts)
    for wi, wo, run, backward in ((2048, 2064, ex.h.nvfp4_grouped_forward, False),
                                  (2064, 2048, ex.h.nvfp4_grouped_backward, True)):
        x = rows_of(R, wi)
        first = run(x, off, blank(R, wo, ex.dtype))
        verify(ex, counts, first, x, backward)
        for _ in range(5):
            assert torch.equal(run(x, off, blank(R, wo, ex.dtype)), first)
    status_ok(ex.h)


@pytest.mark.parametrize("out_f32", [False, True])
def test_narrow_tiles_on_pairs(out_f32):
    """More units than multiprocessors, few rows each: two MMA issuers a pair."""
    counts = [7, 0, 61, 64, 1, 16, 17, 3, 0, 40, 65, 2, 9, 33, 0, 12, 5, 28, 31, 90]
    ex = Experts(20, 1040, 1152, sum(counts), out_f32=out_f32)
    ex.h.nvfp4_moe_set_path(P.PATH_PREFILL)
    off, R = offsets_of(counts), sum(counts)
    for wi, wo, run, backward in ((1152, 1040, ex.h.nvfp4_grouped_forward, False),
                                  (1040, 1152, ex.h.nvfp4_grouped_backward, True)):
        x = rows_of(R, wi)
        first = run(x, off, blank(R, wo, ex.dtype))
        verify(ex, counts, first, x, backward)
        for _ in range(5):
            assert torch.equal(run(x, off, blank(R, wo, ex.dtype)), first)
    status_ok(ex.h)


@pytest.mark.parametrize("E,N,K,counts", [
    (1, 2048, 2048, [1]), (1, 4096, 4096, [33]), (1, 4112, 2176, [70]), (1, 1040, 4224, [300]), (2, 272, 2048, [0, 5]),
    (3, 528, 1152, [64, 1, 129]), (2, 128, 4096, [65, 31]), (1, 144, 640, [513]), (4, 1024, 512, [2, 0, 3, 1])])
@pytest.mark.parametrize("out_f32", [False, True])
def test_clusters_that_share_a_reduction(E, N, K, counts, out_f32):
    """Few units, long sums: each shared by 2 or 4 CTAs."""
    R = sum(counts) + 3
    ex = Experts(E, N, K, R, out_f32=out_f32)
    ex.h.nvfp4_moe_set_path(P.PATH_PREFILL)
    off = offsets_of(counts, 2)
    for wi, wo, run, backward in ((K, N, ex.h.nvfp4_grouped_forward, False), (N, K, ex.h.nvfp4_grouped_backward, True)):
        x = rows_of(R, wi)
        first = run(x, off, blank(R, wo, ex.dtype, pad=8))
        status_ok(ex.h)
        verify(ex, counts, first, x, backward, first=2)
        for _ in range(3):
            assert torch.equal(run(x, off, blank(R, wo, ex.dtype))[2:-1], first[2:-1])
    status_ok(ex.h)


def test_bounded_wait_of_the_streaming_kernel_reports_a_timeout():
    ex = Experts(3, 272, 512, 40)
    ex.h.nvfp4_moe_set_path(P.PATH_DECODE)
    counts = [1, 20, 9]
    x, off = rows_of(30, 512), offsets_of(counts)
    ex.h.nvfp4_moe_debug_set_fault(1)
    ex.h.nvfp4_grouped_forward(x, off, blank(30, 272, ex.dtype))
    assert P.STATUS[ex.h.nvfp4_moe_get_status()[0]] == "NVFP4_MOE_ERR_TIMEOUT"
    ex.h.nvfp4_moe_debug_set_fault(0)
    out = ex.h.nvfp4_grouped_forward(x, off, blank(30, 272, ex.dtype))
    status_ok(ex.h)
    verify(ex, counts, out, x, False, fp16_rows=FP16_ROWS[P.PATH_DECODE])


def test_bounded_waits_of_a_cluster_report_a_timeout():
    ex = Experts(1, 1024, 1024, 40)
    ex.h.nvfp4_moe_set_path(P.PATH_PREFILL)
    x, dy, off = rows_of(40, 1024), rows_of(40, 1024, 5), offsets_of([40])
    ex.h.nvfp4_moe_debug_set_fault(1)
    for run, rows in ((ex.h.nvfp4_grouped_forward, x), (ex.h.nvfp4_grouped_backward, dy)):
        run(rows, off, blank(40, 1024, ex.dtype))
        assert P.STATUS[ex.h.nvfp4_moe_get_status()[0]] == "NVFP4_MOE_ERR_TIMEOUT"
    ex.h.nvfp4_moe_debug_set_fault(0)
    out = ex.h.nvfp4_grouped_forward(x, off, blank(40, 1024, ex.dtype))
    status_ok(ex.h)
    verify(ex, [40], out, x, False)


def test_bounded_waits_of_a_pair_report_a_timeout():
    ex = Experts(2, 272, 256, 200)
    ex.h.nvfp4_moe_set_path(P.PATH_PREFILL)
    x, off, counts = rows_of(200, 256), offsets_of([130, 70]), [130, 70]
    dy = rows_of(200, 272)
    ex.h.nvfp4_moe_debug_set_fault(1)
    for run, rows, n in ((ex.h.nvfp4_grouped_forward, x, 272), (ex.h.nvfp4_grouped_backward, dy, 256)):
        run(rows, off, blank(200, n, ex.dtype))
        assert P.STATUS[ex.h.nvfp4_moe_get_status()[0]] == "NVFP4_MOE_ERR_TIMEOUT"
    ex.h.nvfp4_moe_debug_set_fault(0)
    out = ex.h.nvfp4_grouped_forward(x, off, blank(200, 272, ex.dtype))
    dx = ex.h.nvfp4_grouped_backward(dy, off, blank(200, 256, ex.dtype))
    status_ok(ex.h)
    verify(ex, counts, out, x, False)
    verify(ex, counts, dx, dy, True)


def test_stage_times_count_the_products():
    ex = Experts(2, 128, 256, 40)
    x, off = rows_of(40, 256), offsets_of([30, 10])
    ex.h.nvfp4_moe_set_profiling(True)
    for path in FORWARD:
        ex.h.nvfp4_moe_set_path(path)
        ex.h.nvfp4_grouped_forward(x, off, blank(40, 128, ex.dtype))
    ms, n = ex.h.nvfp4_moe_get_stage_times()
    assert n == 2 and ms[2] > 0 and ms[2] < 1000
    ex.h.nvfp4_moe_set_profiling(False)
    status_ok(ex.h)


def test_refusals():
    ex = Experts(2, 128, 256, 16)
    h, lib = ex.h, ex.h.lib
    x, out, off = rows_of(16, 256), blank(16, 128, ex.dtype), offsets_of([8, 8])
    ptr, st = P.binding._ptr, P.binding._stream()
    inv, shape = CODE["NVFP4_MOE_ERR_INVALID_ARG"], CODE["NVFP4_MOE_ERR_UNSUPPORTED_SHAPE"]
    call = lambda R=16, o=ptr(off), xp=ptr(x), ldx=256, op=ptr(out), ldo=128: \
        lib.nvfp4_grouped_forward(h.h, R, o, xp, ldx, op, ldo, st)
    assert call() == 0
    assert call(R=17) == shape and call(R=-1) == shape
    assert call(o=None) == inv and call(xp=None) == inv and call(op=None) == inv
    assert call(ldx=248) == inv and call(ldx=260) == inv and call(ldo=120) == inv and call(ldo=132) == inv
    assert call(xp=P.binding.ctypes.c_void_p(x.data_ptr() + 2)) == inv
    assert call(op=P.binding.ctypes.c_void_p(out.data_ptr() + 8)) == inv
    with pytest.raises(ValueError):
        h.nvfp4_grouped_forward(x.t(), off, out)
    with pytest.raises(ValueError):
        h.nvfp4_grouped_forward(x, off.long(), out)
    with pytest.raises(ValueError):
        h.nvfp4_grouped_forward(x[:8], off, out)
    with pytest.raises(ValueError):
        h.nvfp4_grouped_forward(x.float(), off, out)
    big = Experts(1, 16, 128, 5000)
    big.h.nvfp4_moe_set_path(P.PATH_DECODE)
    with pytest.raises(P.Nvfp4MoeError) as ei:
        big.h.nvfp4_grouped_forward(rows_of(5000, 128), offsets_of([5000]), blank(5000, 16, big.dtype))
    assert ei.value.status == shape
    fresh = P.Grouped(2, 128, 256, 16)
    with pytest.raises(P.Nvfp4MoeError) as ei:
        fresh.nvfp4_grouped_forward(x, off, out)
    assert ei.value.status == CODE["NVFP4_MOE_ERR_NOT_PACKED"]
    q, s = (torch.zeros((2, 128, n), dtype=torch.uint8, device=DEV) for n in (128, 16))
    for v in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(P.Nvfp4MoeError) as ei:
            fresh.nvfp4_grouped_pack(q, s, torch.tensor([1.0, v], device=DEV))
        assert ei.value.status == CODE["NVFP4_MOE_ERR_BAD_SCALE"]
    # other handles' calls, both ways
    assert lib.nvfp4_linear_forward(h.h, 4, ptr(x), ptr(out), st) == inv
    assert lib.nvfp4_int4_forward(h.h, 4, ptr(x), 256, ptr(out), 128, st) == inv
    assert lib.nvfp4_moe_forward(h.h, ptr(x), 4, 1, ptr(x), ptr(out), st) == inv
    assert lib.nvfp4_moe_set_act_quant(h.h, None, st) == inv
    lin = P.Linear(128, 256, 16)
    assert lib.nvfp4_grouped_forward(lin.h, 16, ptr(off), ptr(x), 256, ptr(out), 128, st) == inv
    assert lib.nvfp4_grouped_backward(lin.h, 16, ptr(off), ptr(x), 256, ptr(out), 128, st) == inv
    lin.close()
    status_ok(h)


def test_packed_bytes_are_the_linears():
    rng = np.random.default_rng(9)
    q, s = nvfp4(rng, 2, 144, 256)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    g = P.Grouped(2, 144, 256, 8)
    g.nvfp4_grouped_pack(t(q), t(s), t(np.ones(2, np.float32)))
    blob = g.nvfp4_moe_debug_packed_blob()
    for e in range(2):
        lin = P.Linear(144, 256, 8)
        lin.nvfp4_linear_pack(t(q[e]), t(s[e]), t(np.ones(1, np.float32)))
        one = lin.nvfp4_moe_debug_packed_blob()
        assert torch.equal(blob[e * one.numel():(e + 1) * one.numel()], one)
        lin.close()
