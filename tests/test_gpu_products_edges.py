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


class _Capture:
    """A stream in capture mode, by the driver's own calls: pack, which synchronises, is refused on it."""

    def __init__(self):
        import ctypes
        self.cu, self.ctypes = ctypes.CDLL("libcuda.so.1"), ctypes
        self.stream = torch.cuda.Stream()

    def __enter__(self):
        assert self.cu.cuStreamBeginCapture_v2(self.ctypes.c_void_p(self.stream.cuda_stream), 2) == 0    # relaxed
        return self.stream

    def __exit__(self, *exc):
        graph = self.ctypes.c_void_p()
        self.cu.cuStreamEndCapture(self.ctypes.c_void_p(self.stream.cuda_stream), self.ctypes.byref(graph))
        if graph.value:
            self.cu.cuGraphDestroy(graph)


def _packers():
    """(handle, pack(stream), forward()) of every kind of handle."""
    P.build()
    rng = np.random.default_rng(4)
    q, s = nvfp4(rng, 2, 128, 256)
    gs = torch.ones((2,), device=DEV)
    off = _t(np.array([0, 2, 4], np.int32))
    x, out = _randn(5, 4, 256).to(BF16), torch.empty((4, 128), dtype=BF16, device=DEV)
    g = P.Grouped(2, 128, 256, 4)
    gq, gsc = _t(q), _t(s)
    yield g, lambda st=None: g.nvfp4_grouped_pack(gq, gsc, gs, stream=st), lambda: g.nvfp4_grouped_forward(x, off, out)
    lin = P.Linear(128, 256, 4)
    one = torch.ones((1,), device=DEV)
    yield lin, lambda st=None: lin.nvfp4_linear_pack(gq[0], gsc[0], one, stream=st), lambda: lin.nvfp4_linear_forward(x, out)
    i4 = P.Int4Linear(128, 256, 64)
    scale = torch.full((128, 4), 0.5, dtype=BF16, device=DEV)
    yield i4, lambda st=None: i4.nvfp4_int4_pack(gq[0], scale, stream=st), lambda: i4.nvfp4_int4_forward(x, out)
    moe = P.MoELayer(2, 128, 128, 4, 1)
    q13, s13 = nvfp4(rng, 2, 256, 128)
    q2, s2 = nvfp4(rng, 2, 128, 128)
    gs3, logits = torch.ones((2, 3), device=DEV), torch.zeros((4, 2), device=DEV)
    xm, om = x[:, :128].contiguous(), torch.empty((4, 128), dtype=BF16, device=DEV)
    w = [_t(a) for a in (q13, s13, q2, s2)]
    yield moe, lambda st=None: moe.nvfp4_moe_pack(*w, gs3, stream=st), lambda: moe.nvfp4_moe_forward(logits, xm, 1, om)


@pytest.mark.parametrize("kind", range(4), ids=["grouped", "linear", "int4", "layer"])
def test_a_refused_call_does_not_fail_the_next(kind):
    """CUDA keeps the last error until it is asked for: one call's must not come back as another's."""
    h, pack, forward = list(_packers())[kind]
    with _Capture() as stream:
        with pytest.raises(P.Nvfp4MoeError):
            pack(stream)
    pack()
    forward()
    assert h.nvfp4_moe_get_status()[0] == 0


@pytest.mark.parametrize("kind", range(4), ids=["grouped", "linear", "int4", "layer"])
def test_a_pack_that_fails_leaves_the_handle_unpacked(kind):
    h, pack, forward = list(_packers())[kind]
    pack()
    forward()
    torch.cuda.synchronize()
    with _Capture() as stream:
        with pytest.raises(P.Nvfp4MoeError) as ei:
            pack(stream)
        assert ei.value.status == CODE["NVFP4_MOE_ERR_CUDA"]
    with pytest.raises(P.Nvfp4MoeError) as ei:
        forward()
    assert ei.value.status == CODE["NVFP4_MOE_ERR_NOT_PACKED"]


def _int4(N, K, group, zeros, f16, out_f32, seed=0):
    """A packed INT4 handle and its codes less their zero points and scales, in float64."""
    P.build()
    rng = np.random.default_rng(seed)
    t = torch.float16 if f16 else BF16
    q = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    scale = torch.from_numpy(rng.uniform(-0.1, 0.1, (N, K // group))).to(t)
    scale[0, 0] = 0.0
    zero = rng.integers(0, 16, (N, K // group), dtype=np.uint8)
    h = P.Int4Linear(N, K, group, act_f16=f16, out_f32=out_f32)
    h.nvfp4_int4_pack(_t(q), scale.to(DEV), _t(zero) if zeros else None)
    code = np.stack([q & 15, q >> 4], axis=-1).reshape(N, K).astype(np.float64)
    z = np.repeat(zero.astype(np.float64), group, axis=1) if zeros else 8.0
    return h, (code - z) * np.repeat(scale.double().numpy(), group, axis=1)


@pytest.mark.parametrize("T,N,K,group,zeros,f16,out_f32", [
    (1, 48, 128, 128, False, False, True), (5, 272, 640, 32, True, True, False), (8, 80, 512, 64, True, False, False),
    (16, 144, 1024, 64, False, True, True), (3, 64, 384, 32, False, False, False), (10, 80, 640, 128, True, True, True),
    (16, 208, 8320, 32, True, False, True),      # clusters: each CTA has a slice of the token
    (12, 48, 16384, 64, False, True, False)])
def test_int4_infinities_keep_their_sign(T, N, K, group, zeros, f16, out_f32):
    """A token's infinities give what the definition gives: s (q - z) x is an infinity of the term's sign, NaN where
    s (q - z) is zero or two terms' signs differ.  Tokens without any are as they were, bit for bit."""
    h, w = _int4(N, K, group, zeros, f16, out_f32)
    x = _randn(6, T, K).to(torch.float16 if f16 else BF16)
    new = lambda: torch.empty((T, N), dtype=torch.float32 if out_f32 else x.dtype, device=DEV)
    clean = h.nvfp4_int4_forward(x, new())
    rng = np.random.default_rng(7)
    inf = float("inf")
    marks = [[(0, inf)], [(K - 1, -inf)], [(K // 2 + 3, inf), (K // 3, inf)], [(5, inf), (K - 9, -inf)],
             [(K // 2, inf), (K // 2 + 1, -inf)], [(17, float("nan"))], [(K - 2, inf), (1, float("nan"))]]
    hit = {}
    for i, t in enumerate(rng.permutation(T)[:max(1, T - 1)]):
        for k, v in marks[i % len(marks)]:
            x[t, k] = v
        hit[t] = True
    got = h.nvfp4_int4_forward(x, new())
    assert h.nvfp4_moe_get_status()[0] == 0
    xs = x.double().cpu().numpy()
    for t in range(T):
        if t not in hit:
            assert torch.equal(got[t], clean[t])
            continue
        k = np.nonzero(~np.isfinite(xs[t]))[0]
        with np.errstate(invalid="ignore"):
            want = (w[:, k] * xs[t, k]).sum(axis=1)
        np.testing.assert_array_equal(got[t].double().cpu().numpy(), want)
    h.close()


@pytest.mark.parametrize("K,most", [(4096, 8), (7168, 5), (8192, 4), (12288, 2), (16384, 2)])
def test_the_default_path_streams_one_tile_an_expert(K, most):
    """Where an expert's rows no longer fit the streaming kernel's one pass over the matrix, the GEMM takes over.  The
    two add in different orders, so the bits of an FP32 result tell which one ran."""
    E, N = 4, 256
    h = _experts(E, N, K, E * 8 + 4, out_f32=True, seed=K)
    for R, path in ((E * most, P.PATH_DECODE), (E * most + 4, P.PATH_PREFILL), (E * 8 + 4, P.PATH_PREFILL)):
        off = _t((np.arange(E + 1) * R // E).astype(np.int32))
        x = _randn(R, R, K).to(BF16)
        got = {}
        for p in (P.PATH_AUTO, P.PATH_DECODE, P.PATH_PREFILL):
            h.nvfp4_moe_set_path(p)
            got[p] = h.nvfp4_grouped_forward(x, off, torch.empty((R, N), device=DEV))
        assert not torch.equal(got[P.PATH_DECODE], got[P.PATH_PREFILL])
        assert torch.equal(got[P.PATH_AUTO], got[path]), (R, path)
    assert h.nvfp4_moe_get_status()[0] == 0
    h.close()
