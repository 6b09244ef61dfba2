"""Calls of the 4-bit products that the documentation allows and that went, or could have gone, wrong."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import nvfp4_weight_only_w4a16_gb300 as P
from tests.products import DEV, nvfp4

pytestmark = pytest.mark.gpu
CODE = P.STATUS_CODE
BF16 = torch.bfloat16


def _t(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _experts(E, N, K, max_rows, out_f32=False, seed=0):
    P.build()
    rng = np.random.default_rng(seed)
    q, s = nvfp4(rng, E, N, K)
    h = P.Grouped(E, N, K, max_rows, out_f32=out_f32)
    h.nvfp4_grouped_pack(_t(q), _t(s), _t(rng.uniform(0.25, 4.0, E).astype(np.float32)))
    return h


def _randn(seed, *shape):
    return torch.randn(shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV)


@pytest.mark.parametrize("path", [P.PATH_DECODE, P.PATH_PREFILL])
def test_offsets_written_by_the_kernel_before(path):
    """The offsets come from a kernel that lets its successor begin early: an INT4 product whose FP32 results are
    the subnormals n 2^-149, that is the integers n.  Each product has to see those of its own predecessor."""
    E, K, R = 15, 512, 48
    h = _experts(E, 256, K, R)
    h.nvfp4_moe_set_path(path)
    rng = np.random.default_rng(1)
    code = np.sort(rng.integers(0, 16, (16, 128), dtype=np.uint8), axis=0)     # ascending: so are the offsets
    lin = P.Int4Linear(16, 128, 128, out_f32=True)
    lin.nvfp4_int4_pack(_t(code[:, 0::2] | (code[:, 1::2] << 4)), torch.full((16, 1), 2.0 ** -49, dtype=BF16, device=DEV),
                        torch.zeros((16, 1), dtype=torch.uint8, device=DEV))
    picks = [[0, 1], [2, 3, 4], [5], [6, 7, 8]]
    sel = torch.zeros((len(picks), 1, 128), dtype=BF16, device=DEV)
    for i, p in enumerate(picks):
        sel[i, 0, p] = 2.0 ** -100
    x = _randn(2, R, K).to(BF16)
    off = torch.empty((1, 16), device=DEV)
    ints = off.view(torch.int32)[0]
    want = []
    for i, p in enumerate(picks):
        lin.nvfp4_int4_forward(sel[i], off)
        assert ints.tolist() == code[:, p].sum(axis=1).tolist()
        out = torch.full((R, 256), float("nan"), dtype=BF16, device=DEV)
        want.append(h.nvfp4_grouped_forward(x, ints, out))
        torch.cuda.synchronize()
    outs = torch.full((50 * len(picks), R, 256), float("nan"), dtype=BF16, device=DEV)
    torch.cuda.synchronize()
    for i in range(outs.shape[0]):
        lin.nvfp4_int4_forward(sel[i % len(picks)], off)
        h.nvfp4_grouped_forward(x, ints, outs[i])
    torch.cuda.synchronize()
    for i in range(outs.shape[0]):
        assert torch.equal(outs[i].view(torch.int16), want[i % len(picks)].view(torch.int16)), i
    for handle in (h, lin):
        assert handle.nvfp4_moe_get_status()[0] == 0
        handle.close()


@pytest.mark.parametrize("path", [P.PATH_DECODE, P.PATH_PREFILL])
def test_a_call_behind_one_that_times_out(path):
    """Every warp of a kernel whose wait has run out leaves it (its copies are held back here), and the call queued
    behind it, which begins early, computes as if nothing had been."""
    N, K = 272, 1152
    h = _experts(3, N, K, 13, out_f32=True)
    h.nvfp4_moe_set_path(path)
    off = _t(np.array([0, 5, 5, 13], np.int32))
    x = _randn(3, 13, K).to(BF16)
    want = h.nvfp4_grouped_forward(x, off, torch.empty((13, N), device=DEV))
    assert h.nvfp4_moe_get_status()[0] == 0
    h.nvfp4_moe_debug_set_fault(1)
    h.nvfp4_grouped_forward(x, off, torch.empty((13, N), device=DEV))
    h.nvfp4_moe_debug_set_fault(0)
    got = h.nvfp4_grouped_forward(x, off, torch.empty((13, N), device=DEV))
    assert P.STATUS[h.nvfp4_moe_get_status()[0]] == "NVFP4_MOE_ERR_TIMEOUT"
    assert h.nvfp4_moe_get_status()[0] == 0
    assert torch.equal(got, want)
    h.close()
