"""The 4-bit products on the GPU: right to the bit where every sum is exact, and within the documented error of the
norm where it is not (tests.exact says why, test_exact_cpu what these reject)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import nvfp4_weight_only_w4a16_gb300 as P
from tests.exact import check_exact, check_norm, int4_exact, nvfp4_exact, rows_exact
from tests.products import DEV, f64, int4_values, nvfp4, nvfp4_values

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _t(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _product(h, rows, off, n, dtype, backward):
    run = h.nvfp4_grouped_backward if backward else h.nvfp4_grouped_forward
    out = run(rows, off, torch.full((rows.shape[0], n), float("nan"), dtype=dtype, device=DEV))
    assert h.nvfp4_moe_get_status()[0] == 0
    return f64(out)


# few rows: streamed, and as GEMM; the GEMM's tiles of 64, 128 and 256 rows, alone, in pairs, and shared by clusters
GROUPED = [
    (2, 48, 16384, [9, 1], P.PATH_DECODE), (3, 272, 640, [8, 0, 17], P.PATH_DECODE), (1, 1040, 12416, [3], P.PATH_DECODE),
    (2, 48, 16384, [9, 1], P.PATH_PREFILL), (1, 16384, 128, [70], P.PATH_PREFILL), (1, 272, 8320, [200], P.PATH_PREFILL),
    (20, 1040, 1152, [20] * 19 + [64], P.PATH_PREFILL), (10, 1040, 1152, [20] * 10, P.PATH_PREFILL),
    (4, 1040, 4224, [100, 128, 3, 60], P.PATH_PREFILL), (100, 128, 1152, [40] * 100, P.PATH_PREFILL),
    (3, 1040, 4224, [256, 700, 1], P.PATH_PREFILL), (90, 128, 256, [130] * 90, P.PATH_PREFILL)]


@pytest.mark.parametrize("out_f32", [False, True])
@pytest.mark.parametrize("E,N,K,counts,path", GROUPED)
def test_grouped_is_exact(E, N, K, counts, path, out_f32):
    P.build()
    rng = np.random.default_rng(N + K)
    q, s, gs = nvfp4_exact(rng, E, N, K)
    w = nvfp4_values(q, s) * gs.astype(np.float64)[:, None, None]
    R = sum(counts)
    h = P.Grouped(E, N, K, R, out_f32=out_f32)
    h.nvfp4_grouped_pack(_t(q), _t(s), _t(gs))
    h.nvfp4_moe_set_path(path)
    dtype = F32 if out_f32 else BF16
    cuts = np.concatenate([[0], np.cumsum(counts)])
    off = _t(cuts.astype(np.int32))
    for backward in ((False, True) if path == P.PATH_PREFILL else (False,)):
        x = rows_exact(rng, R, N if backward else K)
        got = _product(h, _t(x).to(BF16), off, K if backward else N, dtype, backward)
        for e in range(E):
            r = slice(cuts[e], cuts[e + 1])
            check_exact(got[r], x[r] @ (w[e] if backward else w[e].T), dtype, f"expert {e}, backward {backward}")
    h.close()


@pytest.mark.parametrize("T,N,K,group,zeros,f16,out_f32", [
    (1, 16, 16384, 64, True, False, True), (2, 32, 8320, 64, True, False, True), (5, 96, 12416, 32, True, True, True),
    (16, 208, 16384, 32, True, False, True), (8, 272, 16384, 128, False, False, True), (16, 208, 16384, 32, True, True, False),
    (3, 272, 640, 32, True, False, False), (9, 304, 4224, 64, False, True, False), (16, 4848, 4096, 32, True, False, True),
    (16, 2080, 2176, 128, True, False, False), (13, 1056, 8320, 64, False, True, True), (4, 12576, 1024, 128, True, False, True)])
def test_int4_is_exact(T, N, K, group, zeros, f16, out_f32):
    P.build()
    rng = np.random.default_rng(N + K)
    q, s, z = int4_exact(rng, N, K, group)
    act = F16 if f16 else BF16
    h = P.Int4Linear(N, K, group, act_f16=f16, out_f32=out_f32)
    h.nvfp4_int4_pack(_t(q), _t(s).to(act), _t(z) if zeros else None)
    x = rows_exact(rng, T, K)
    dtype = F32 if out_f32 else act
    out = h.nvfp4_int4_forward(_t(x).to(act), torch.empty((T, N), dtype=dtype, device=DEV))
    assert h.nvfp4_moe_get_status()[0] == 0
    y = x @ int4_values(q, s, z if zeros else None, group).T
    if not f16 or out_f32 or np.abs(y).max() < 65000:
        check_exact(f64(out), y, dtype)
    else:                                    # beyond FP16: infinities, of the right sign
        fits = np.abs(y) < 65000
        assert fits.any()
        check_exact(f64(out)[fits], y[fits], dtype)
    h.close()


@pytest.mark.parametrize("E,N,K,rows,path,forward,backward", [
    (2, 1536, 4096, 8, P.PATH_DECODE, 256, None), (20, 1040, 4096, 60, P.PATH_DECODE, 1024, None),
    (10, 1040, 4096, 20, P.PATH_PREFILL, 2048, 520), (20, 1040, 4096, 20, P.PATH_PREFILL, 2048, 520),
    (20, 1040, 4096, 100, P.PATH_PREFILL, 2048, 520), (20, 1040, 4096, 250, P.PATH_PREFILL, 2048, 520),
    (20, 4096, 1024, 20, P.PATH_PREFILL, 512, 2048), (20, 4096, 1024, 60, P.PATH_PREFILL, 512, 2048),
    (20, 4096, 1024, 250, P.PATH_PREFILL, 512, 2048), (2, 1536, 4096, 8, P.PATH_PREFILL, 1024, 768),
    (2, 1536, 16384, 300, P.PATH_PREFILL, 8192, 768)])
def test_grouped_fp32_results_within_the_documented_error(E, N, K, rows, path, forward, backward):
    """forward, backward: the terms that one accumulator adds: the GEMM has two, or one in each CTA that shares a sum;
    the streaming kernel one in each warp.

    The documented error is 1.2e-9 of the norm per term, here plus an eighth, and 2^-24 for the rounding of the
    result and of the accumulators' sum.  A term's share of one cut at the last of 24 bits, in 16 terms, is 7.5e-9.
    All in one accumulator would be twice the GEMM's."""
    P.build()
    rng = np.random.default_rng(K + rows)
    q, s = nvfp4(rng, E, N, K)
    w = nvfp4_values(q, s)
    h = P.Grouped(E, N, K, E * rows, out_f32=True)
    h.nvfp4_grouped_pack(_t(q), _t(s), torch.ones((E,), device=DEV))
    h.nvfp4_moe_set_path(path)
    off = _t((np.arange(E + 1) * rows).astype(np.int32))
    for back, terms in ((False, forward), (True, backward)):
        if terms is None:
            continue
        x = torch.randn((E * rows, N if back else K), generator=torch.Generator(device=DEV).manual_seed(rows), device=DEV).to(BF16)
        got = _product(h, x, off, K if back else N, F32, back)
        y = np.concatenate([f64(x[e * rows:(e + 1) * rows]) @ (w[e] if back else w[e].T) for e in range(E)])
        check_norm(got, y, 1.35e-9 * terms + 2.0 ** -23, f"backward {back}")
    h.close()


def _normal_codes(rng, N, K, group, zeros):
    """Codes (0..15), scales and zero points of normal weights: about code 8, or over each group's range."""
    w = rng.standard_normal((N, K // group, group))
    if zeros:
        s, z = (w.max(axis=2) - w.min(axis=2)) / 15, np.clip(np.round(-w.min(axis=2) * 15 / np.ptp(w, axis=2)), 0, 15)
    else:
        s, z = np.abs(w).max(axis=2) / 7, np.full((N, K // group), 8.0)
    code = np.clip(np.round(w / s[..., None]) + z[..., None], 0, 15).astype(np.uint8).reshape(N, K)
    return code[:, 0::2] | (code[:, 1::2] << 4), 0.02 * s, z.astype(np.uint8)


@pytest.mark.parametrize("T,N,K,group,zeros", [(1, 4096, 4096, 128, False), (4, 4096, 4096, 64, True), (16, 2048, 8192, 32, True),
                                               (2, 2048, 16384, 64, False), (16, 1024, 16384, 32, True)])
@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("normal,most", [(False, 1.5e-7), (True, 2e-7)])
def test_int4_fp32_results_within_the_documented_error(T, N, K, group, zeros, normal, most, f16):
    """1 to 1.5e-7 of the norm, or half as much again with codes of normal weights, whose sums before the zero points
    come off are larger beside the result.  Codes two bits lower in FP16's subnormals give 2 to 6e-7, and FP16
    activations, whose 3 bits more than BF16's only centred codes keep, 2e-7 without those."""
    P.build()
    rng = np.random.default_rng(K + T)
    act = F16 if f16 else BF16
    if normal:
        q, s, z = _normal_codes(rng, N, K, group, zeros)
    else:
        q, s, z = rng.integers(0, 256, (N, K // 2), dtype=np.uint8), rng.uniform(0.025, 0.075, (N, K // group)), \
            rng.integers(0, 16, (N, K // group), dtype=np.uint8)
    s, z = _t(s).to(act), z if zeros else None
    h = P.Int4Linear(N, K, group, act_f16=f16, out_f32=True)
    h.nvfp4_int4_pack(_t(q), s, None if z is None else _t(z))
    x = torch.randn((T, K), generator=torch.Generator(device=DEV).manual_seed(T), device=DEV).to(act)
    got = h.nvfp4_int4_forward(x, torch.empty((T, N), device=DEV))
    assert h.nvfp4_moe_get_status()[0] == 0
    check_norm(f64(got), f64(x) @ int4_values(q, f64(s), z, group).T, most)
    h.close()
