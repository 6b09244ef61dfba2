"""The operators around the products at their largest: rows further apart than 32 bits reach, more tokens than the INT8
workspace holds, the most tokens of a route call.  Whole results are compared for equality, with those of small calls, which
are tested against plain forms elsewhere, or with their definition."""
import pytest

torch = pytest.importorskip("torch")

import nvfp4_weight_only_w4a16_gb300 as P
from tests.block_ops import DEV, U, f64, half_step, norm_backward, within
from tests.test_gpu_int8 import _run

pytestmark = pytest.mark.gpu
FAR = 1 << 24          # the largest row stride; 150 rows of it are beyond 2^31 elements
ROWS = 150


@pytest.fixture(scope="module", autouse=True)
def built():
    P.build()


def _far(shape, dtype, fill=None):
    """Rows FAR elements apart."""
    m = torch.empty((shape[0], FAR), dtype=dtype, device=DEV)[:, :shape[1]]
    m.copy_(fill) if fill is not None else m.fill_(7)
    return m


def _rand(*s, dtype=torch.bfloat16):
    return torch.randn(s, device=DEV, generator=torch.Generator(DEV).manual_seed(sum(s))).to(dtype)


@pytest.mark.parametrize("H", [64, 4096])
def test_norm_of_rows_far_apart(H):
    n = P.Norm(H)
    x, r, w, dy = _rand(ROWS, H), _rand(ROWS, H) * 2, _rand(H), _rand(ROWS, H) * 3
    got = []
    for far in (False, True):
        new = (lambda d, f=None: _far((ROWS, H), d, f)) if far else \
              (lambda d, f=None: f if f is not None else torch.empty((ROWS, H), dtype=d, device=DEV))
        bf = torch.bfloat16
        s, y, q = new(bf), new(bf), new(torch.int8)
        qs, rstd, dw = torch.empty(ROWS, device=DEV), torch.empty(ROWS, device=DEV), torch.empty(H, device=DEV)
        n.nvfp4_norm_forward(new(bf, x), w, residual=new(bf, r), sum=s, y=y, q=q, q_scale=qs, rstd=rstd)
        dx = new(bf)
        n.nvfp4_norm_backward(new(bf, dy), s, w, rstd, dx, dweight=dw)
        got.append([t.clone() for t in (s, y, q, qs, rstd, dx, dw)])
        del s, y, q, dx
        torch.cuda.empty_cache()
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert n.nvfp4_moe_get_status()[0] == 0
    n.close()


# every thread layout with more rows than its CTAs hold at a time, and a last turn that few of them have
@pytest.mark.parametrize("T,H", [(40003, 8), (30001, 64), (15001, 128), (12345, 256), (9001, 512), (5001, 1024), (2501, 2048),
                                 (1501, 5120), (1001, 8192)])
def test_norm_gradient_of_many_rows(T, H):
    n = P.Norm(H)
    h, dy, w = _rand(T, H) * 2, _rand(T, H) * 2.0 ** -4, _rand(H)
    y, rstd = torch.empty_like(h), torch.empty((T,), device=DEV)
    n.nvfp4_norm_forward(h, w, y=y, rstd=rstd)
    dx, dw = torch.empty_like(h), torch.empty((H,), device=DEV)
    n.nvfp4_norm_backward(dy, h, w, rstd, dx, dweight=dw)
    want, b, want_w, b_w = norm_backward(f64(dy), f64(h), f64(w), f64(rstd), 0.0)
    within(f64(dx), want, b + half_step(abs(want) + b, torch.bfloat16), "dx")
    within(f64(dw), want_w, b_w + U * abs(want_w), "dweight")
    dw2 = torch.empty_like(dw)
    n.nvfp4_norm_backward(dy, h, w, rstd, dx, dweight=dw2)
    assert torch.equal(dw2, dw)
    n.close()


def test_swiglu_of_rows_far_apart():
    I = 272
    n = P.SwiGLU(I)
    g, u, dh = _rand(ROWS, I), _rand(ROWS, I) * 2, _rand(ROWS, I) * 3
    got = []
    for far in (False, True):
        new = (lambda f=None: _far((ROWS, I), torch.bfloat16, f)) if far else \
              (lambda f=None: f if f is not None else torch.empty((ROWS, I), dtype=torch.bfloat16, device=DEV))
        h, dg, du = new(), new(), new()
        codes = torch.empty((ROWS, 2, I), dtype=torch.int8, device=DEV)
        scales = torch.empty((ROWS, 2, n.blocks), device=DEV)
        n.nvfp4_swiglu_forward(new(g), new(u), h, codes, scales)
        n.nvfp4_swiglu_backward(codes, scales, new(dh), dg, du)
        got.append([t.clone() for t in (h, codes, scales, dg, du)])
        del h, dg, du
        torch.cuda.empty_cache()
    assert all(torch.equal(a, b) for a, b in zip(*got))
    n.close()


def test_swiglu_codes_beyond_32_bits():
    R, I, S = (1 << 32) // (2 * 16384) + 70, 16384, 40     # the codes of the last rows lie behind 2^32 bytes
    n = P.SwiGLU(I)
    blk = _rand(64, I)
    g = blk.repeat((R + 63) // 64, 1)[:R].contiguous()
    h = torch.empty_like(g)
    codes = torch.empty((R, 2, I), dtype=torch.int8, device=DEV)
    scales = torch.empty((R, 2, n.blocks), device=DEV)
    n.nvfp4_swiglu_forward(g, g, h, codes, scales)
    dg, du = torch.empty_like(g), torch.empty_like(g)
    n.nvfp4_swiglu_backward(codes, scales, g, dg, du)
    for at in (0, R // 2, R - S):
        few = [t[at:at + S] for t in (g, h, codes, scales, dg, du)]
        h2, c2, s2, dg2, du2 = (torch.empty_like(t) for t in few[1:])
        n.nvfp4_swiglu_forward(few[0], few[0], h2, c2, s2)
        n.nvfp4_swiglu_backward(c2, s2, few[0], dg2, du2)
        assert all(torch.equal(a, b) for a, b in zip(few[1:], (h2, c2, s2, dg2, du2))), at
    n.close()


@pytest.mark.parametrize("T,E", [(ROWS, 256), (ROWS, 64)])
def test_route_of_rows_far_apart(T, E):
    k = 4
    h = P.Route(E, k, score="sigmoid")
    near = _rand(T, E, dtype=torch.float32)
    dw = _rand(T, k, dtype=torch.float32)
    got = []
    for logits, dl in ((near, torch.empty_like(near)), (_far((T, E), torch.float32, near), _far((T, E), torch.float32))):
        ids, w = torch.empty((T, k), dtype=torch.int32, device=DEV), torch.empty((T, k), device=DEV)
        off = torch.empty(E + 1, dtype=torch.int32, device=DEV)
        perm, inv = (torch.empty(T * k, dtype=torch.int32, device=DEV) for _ in range(2))
        h.nvfp4_route_forward(logits, ids, w, off, perm, inv)
        h.nvfp4_route_backward(logits, ids, dw, dl)
        got.append([t.clone() for t in (ids, w, off, perm, inv, dl)])
    assert all(torch.equal(a, b) for a, b in zip(*got))
    h.close()


@pytest.mark.parametrize("E,k", [(512, 1), (256, 8), (8, 8), (1, 1)])
def test_route_of_the_most_tokens(E, k):
    T = 1 << 20
    h = P.Route(E, k, logits_bf16=True)
    logits = _rand(T, E)
    ids, w = torch.empty((T, k), dtype=torch.int32, device=DEV), torch.empty((T, k), device=DEV)
    off = torch.empty(E + 1, dtype=torch.int32, device=DEV)
    perm, inv = (torch.empty(T * k, dtype=torch.int32, device=DEV) for _ in range(2))
    h.nvfp4_route_forward(logits, ids, w, off, perm, inv)
    flat = ids.flatten().long()
    want = torch.sort(flat, stable=True).indices
    assert torch.equal(perm.long(), want)
    assert torch.equal(inv.long()[want], torch.arange(T * k, device=DEV))
    assert torch.equal(off.long(), torch.cat([flat.new_zeros(1), torch.bincount(flat, minlength=E).cumsum(0)]))
    for at in (0, T // 2 - 3, T - 60):                      # and the choice is a small call's
        few = logits[at:at + 60]
        i2, w2 = torch.empty((60, k), dtype=torch.int32, device=DEV), torch.empty((60, k), device=DEV)
        p2, v2 = (torch.empty(60 * k, dtype=torch.int32, device=DEV) for _ in range(2))
        h.nvfp4_route_forward(few, i2, w2, torch.empty_like(off), p2, v2)
        assert torch.equal(i2, ids[at:at + 60]) and torch.equal(w2, w[at:at + 60]), at
    h.close()


# K 16384: the workspace holds 8064 tokens; a last stretch of 1, 5, 60 and 130 tokens, and a third one
@pytest.mark.parametrize("T", [8064, 8065, 8069, 8124, 8194, 16129])
@pytest.mark.parametrize("N", [16, 400])
def test_int8_of_more_tokens_than_the_workspace_holds(N, T):
    _run(N, 16384, T, ("bf16", "f32")[T % 2], seed=T, bias=T % 2 == 0)


@pytest.mark.parametrize("T", [9, 40, 150])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_int8_of_rows_far_apart(T, out):
    N, K = 272, 528
    g = torch.Generator(DEV).manual_seed(T)
    ri = lambda *s: torch.randint(-128, 128, s, generator=g, device=DEV, dtype=torch.int32).to(torch.int8)
    x, w, sx, sw = ri(T, K), ri(N, K), torch.rand(T, generator=g, device=DEV), torch.rand(N, generator=g, device=DEV)
    h = P.Int8Linear(N, K, T, out=out)
    h.nvfp4_int8_pack(w, sw)
    dt = torch.float32 if out == "f32" else torch.bfloat16
    near, far = torch.empty((T, N), dtype=dt, device=DEV), _far((T, N), dt)
    h.nvfp4_int8_forward(x, sx, near)
    h.nvfp4_int8_forward(_far((T, K), torch.int8, x), sx, far)
    assert torch.equal(near, far)
    assert h.nvfp4_moe_get_status()[0] == 0
    h.close()
