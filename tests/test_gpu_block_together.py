"""The operators around the 4-bit products used together, on the GPU: a block of a model, forward and backward --
norm with the residual, routing, the experts' gate, up and down products, SwiGLU with 8-bit checkpoints, the weighted sum
-- and beside it the norm's 8-bit output into an INT8 linear.

Each operator is held to the float64 form of its own actual inputs (its own bounds, tests/block_ops.py and
tests/products.py), so that what is tested here is that they fit: what one writes is what the next reads, without a copy or
a wait between them, in a captured graph too.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import nvfp4_weight_only_w4a16_gb300 as P
from tests import block_ops as B
from tests.products import bound, check, nvfp4_values
from tests.test_gpu_int8 import _want
from tests.test_gpu_route_alone import _weights_tol

pytestmark = pytest.mark.gpu
DEV, dev, f64, BF16 = B.DEV, B.dev, B.f64, torch.bfloat16
EPS = 1e-6


class Block:
    """E experts of H x I, top-k of T tokens, and an INT8 projection to N; every buffer there from the start."""

    def __init__(self, T, E=16, H=512, I=272, k=4, N=208, seed=0):
        P.build()
        rng = np.random.default_rng(seed)
        self.T, self.E, self.H, self.I, self.k, self.N = T, E, H, I, k, N
        R = T * k
        self.norm = P.Norm(H, EPS)
        self.route = P.Route(E, k, score="sigmoid", groups=4, top_groups=2, group_top=2, scale=1.5)
        self.act = P.SwiGLU(I)
        self.proj = P.Int8Linear(N, H, T, out="f32")
        wq = rng.integers(-127, 128, (N, H)).astype(np.int8)
        self.wq, self.sw = dev(wq), dev(rng.uniform(1e-4, 1e-3, N).astype(np.float32))
        self.proj.nvfp4_int8_pack(self.wq, self.sw)
        Ip = -(-I // 128) * 128           # the grouped products' reduction is in multiples of 128: zeros in the rest
        self.Ip = Ip
        self.mats, self.w = {}, {}
        for name, n, kk in (("gate", I, H), ("up", I, H), ("down", H, Ip)):
            q = rng.integers(0, 256, (E, n, kk // 2), dtype=np.uint8)
            s = rng.choice(np.array([0x28, 0x30, 0x33, 0x38], np.uint8), (E, n, kk // 16))
            g = np.full(E, 0.02, np.float32)
            h = P.Grouped(E, n, kk, R)
            h.nvfp4_grouped_pack(dev(q), dev(s), dev(g))
            self.mats[name], self.w[name] = h, nvfp4_values(q, s) * g.astype(np.float64)[:, None, None]
        new = lambda *s, d=BF16: torch.zeros(s, dtype=d, device=DEV)
        i32, f32 = torch.int32, torch.float32
        self.x, self.res, self.weight = new(T, H), new(T, H), (1 + 0.1 * torch.randn(H, device=DEV)).to(BF16)
        self.router = (torch.randn(E, H, device=DEV) * 0.05).to(BF16)
        self.bias = torch.randn(E, device=DEV) * 0.05
        self.sum, self.y, self.q, self.qs, self.rstd = new(T, H), new(T, H), new(T, H, d=torch.int8), new(T, d=f32), new(T, d=f32)
        self.logits, self.ids, self.wts = new(T, E, d=f32), new(T, k, d=i32), new(T, k, d=f32)
        self.off, self.perm, self.inv = new(E + 1, d=i32), new(R, d=i32), new(R, d=i32)
        self.gu, self.h = new(R, 2 * I), new(R, Ip)
        self.codes, self.scales = new(R, 2, I, d=torch.int8), new(R, 2, -(-I // 128), d=f32)
        self.yd, self.out, self.z = new(R, H), new(T, H), new(T, N, d=f32)
        self.dout, self.drow, self.dh = new(T, H), new(R, H), new(R, Ip)
        self.dgu, self.da, self.db = new(R, 2 * I), new(R, H), new(R, H)
        self.dw, self.dl, self.dsum, self.dx, self.dweight = new(T, k, d=f32), new(T, E, d=f32), new(T, H), new(T, H), new(H, d=f32)

    def fill(self, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        for t in (self.x, self.res, self.dout):
            t.copy_(torch.randn(t.shape, generator=g, device=DEV))

    def run(self):
        I, T, k = self.I, self.T, self.k
        self.norm.nvfp4_norm_forward(self.x, self.weight, residual=self.res, sum=self.sum, y=self.y, q=self.q, q_scale=self.qs,
                                     rstd=self.rstd)
        self.proj.nvfp4_int8_forward(self.q, self.qs, self.z)
        torch.matmul(self.y.float(), self.router.float().t(), out=self.logits)
        self.route.nvfp4_route_forward(self.logits, self.ids, self.wts, self.off, self.perm, self.inv, bias=self.bias)
        token = self.perm.long() // k
        rows = self.y[token]
        gate, up, h = self.gu[:, :I], self.gu[:, I:], self.h[:, :I]
        self.mats["gate"].nvfp4_grouped_forward(rows, self.off, gate)
        self.mats["up"].nvfp4_grouped_forward(rows, self.off, up)
        self.act.nvfp4_swiglu_forward(gate, up, h, codes=self.codes, scales=self.scales)
        self.mats["down"].nvfp4_grouped_forward(self.h, self.off, self.yd)
        back = self.yd[self.inv.long()].view(T, k, -1).float()          # the rows in the tokens' order
        self.out.copy_((self.wts[:, :, None] * back).sum(dim=1))
        # backward of sum(dout * out), to the block's input, the norm's weight and the router's logits
        self.dw.copy_((back * self.dout.float()[:, None]).sum(dim=2))
        self.route.nvfp4_route_backward(self.logits, self.ids, self.dw, self.dl)
        self.drow.copy_(self.wts.flatten()[self.perm.long()][:, None] * self.dout[token].float())
        self.mats["down"].nvfp4_grouped_backward(self.drow, self.off, self.dh)
        dgate, dup = self.dgu[:, :I], self.dgu[:, I:]
        self.act.nvfp4_swiglu_backward(self.codes, self.scales, self.dh[:, :I], dgate, dup)
        self.mats["gate"].nvfp4_grouped_backward(dgate, self.off, self.da)
        self.mats["up"].nvfp4_grouped_backward(dup, self.off, self.db)
        dy = (self.da.float() + self.db.float())[self.inv.long()].view(T, k, -1).sum(dim=1) + self.dl @ self.router.float()
        self.norm.nvfp4_norm_backward(dy.to(BF16), self.sum, self.weight, self.rstd, self.dx, dweight=self.dweight,
                                      dsum=self.dout)
        self.dy = dy.to(BF16)
        self.rows = rows

    def results(self):
        return [t.clone() for t in (self.sum, self.y, self.q, self.qs, self.z, self.ids, self.wts, self.off, self.perm, self.inv,
                                    self.h, self.codes, self.scales, self.out, self.dl, self.dgu, self.dx, self.dweight)]

    def status_ok(self):
        for h in (self.norm, self.route, self.act, self.proj, *self.mats.values()):
            assert h.nvfp4_moe_get_status() == (0, 0)


def _products(off, x, w, got, what, fp16=2.0 ** -38):
    for e in range(len(off) - 1):
        s = slice(off[e], off[e + 1])
        if off[e + 1] > off[e]:
            y = x[s] @ w[e].T
            check(got[s], y, bound(y, x[s], w[e], BF16, fp16), f"{what}, expert {e}")


@pytest.mark.parametrize("T", [1, 13, 300])
def test_a_block_forward_and_backward(T):
    b = Block(T)
    b.fill(T)
    b.run()
    b.status_ok()
    I, E, k = b.I, b.E, b.k
    h = f64((b.x.float() + b.res.float()).to(BF16))
    assert np.array_equal(f64(b.sum), h)
    want, r = B.norm(h, f64(b.weight), float(np.float32(EPS)))
    tol = (B.NORM_CHAIN / 2 + 5) * B.U * np.abs(want)
    B.within(f64(b.y), want, tol + B.half_step(np.abs(want) + tol, BF16), "y")
    assert np.array_equal(f64(b.q), B.codes(h * f64(b.weight))[0])
    assert torch.equal(b.z, _want(b.q, b.wq, b.qs, b.sw, None, "f32"))
    ids, w = B.route(f64(b.logits), k, score="sigmoid", scale=1.5, bias=f64(b.bias), groups=4, top_groups=2, group_top=2)
    assert np.array_equal(b.ids.cpu().numpy(), ids)
    B.within(f64(b.wts), w, _weights_tol(f64(b.logits), w, E), "weights")
    o, p, v = B.tables(ids, E)
    assert all(np.array_equal(t.cpu().numpy(), a) for t, a in ((b.off, o), (b.perm, p), (b.inv, v)))
    gate, up = b.gu[:, :I], b.gu[:, I:]
    _products(o, f64(b.rows), b.w["gate"], f64(gate), "gate")
    _products(o, f64(b.rows), b.w["up"], f64(up), "up")
    hh, tol = B.swiglu(f64(gate), f64(up), BF16)
    B.within(f64(b.h[:, :I]), hh, tol, "h")
    assert not bool(b.h[:, I:].any())
    _products(o, f64(b.h), b.w["down"], f64(b.yd), "down")
    for j, t in enumerate((gate, up)):
        q, s = B.checkpoint(f64(t))
        assert np.array_equal(f64(b.codes[:, j]), q)
        B.within(f64(b.scales[:, j]), s, B.U * s + 2.0 ** -150, "scales")
    # backward
    wt = {n: np.swapaxes(m, 1, 2) for n, m in b.w.items()}
    _products(o, f64(b.drow), wt["down"], f64(b.dh), "down's gradient", 0.0)
    kept = f64(b.codes) * np.repeat(f64(b.scales), 128, axis=2)[:, :, :I]
    d = f64(b.dh[:, :I])
    dg, tg, du, tu = B.swiglu_backward(kept[:, 0], kept[:, 1], d, BF16)
    more = B.U * np.abs(d) * (1 + np.abs(kept[:, 0])) * (np.abs(kept[:, 1]) * (1.1 + np.abs(kept[:, 0])) + 1.1)
    B.within(f64(b.dgu[:, :I]), dg, tg + more, "dgate")
    B.within(f64(b.dgu[:, I:]), du, tu + more, "dup")
    _products(o, f64(b.dgu[:, :I]), wt["gate"], f64(b.da), "gate's gradient", 0.0)
    _products(o, f64(b.dgu[:, I:]), wt["up"], f64(b.db), "up's gradient", 0.0)
    dx, tx, dw, tw = B.norm_backward(f64(b.dy), h, f64(b.weight), f64(b.rstd), f64(b.dout))
    B.within(f64(b.dx), dx, tx + B.half_step(np.abs(dx) + tx, BF16), "dx")
    B.within(f64(b.dweight), dw, tw + B.U * np.abs(dw), "dweight")


@pytest.mark.parametrize("T", [13, 300])
def test_captured_and_replayed_with_other_tokens(T):
    """One graph of the whole block on another stream; replays equal calls one after the other, each waited for."""
    b = Block(T, seed=1)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b.fill(0)
        b.run()
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            b.run()
    for seed in (1, 2, 3):
        b.fill(seed)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = b.results()
        b.run()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, b.results()))
    b.status_ok()


def test_calls_that_feed_each_other_without_a_wait():
    """Each launch may begin before the last one's end: what it reads of it, and overwrites under it, has to wait."""
    T, H = 500, 1024
    rng = np.random.default_rng(3)
    P.build()
    norm, act = P.Norm(H, EPS), P.SwiGLU(H)
    lin = [P.Int8Linear(H, H, T) for _ in range(2)]
    for l in lin:
        l.nvfp4_int8_pack(dev(rng.integers(-127, 128, (H, H)).astype(np.int8)), dev(rng.uniform(1e-3, 2e-3, H).astype(np.float32)))
    x0 = dev(rng.standard_normal((T, H)).astype(np.float32)).to(BF16)
    w = torch.ones((H,), dtype=BF16, device=DEV)
    e = lambda d=BF16: torch.empty((T, H), dtype=d, device=DEV)
    q, s, r, y, u, dw = e(torch.int8), torch.empty((T,), device=DEV), torch.empty((T,), device=DEV), e(), e(), torch.empty((H,), device=DEV)
    codes, scales = torch.empty((T, 2, H), dtype=torch.int8, device=DEV), torch.empty((T, 2, H // 128), device=DEV)

    def chain(wait, n):
        x = x0.clone()
        seen = []
        for _ in range(4):
            norm.nvfp4_norm_forward(x, w, residual=x0, sum=x, q=q, q_scale=s, rstd=r)
            wait()
            lin[0].nvfp4_int8_forward(q[:n], s[:n], y[:n])
            wait()
            lin[1].nvfp4_int8_forward(q[:n], s[:n], u[:n])
            wait()
            act.nvfp4_swiglu_forward(y, u, y, codes=codes, scales=scales)
            wait()
            act.nvfp4_swiglu_backward(codes, scales, y, y, u)
            wait()
            norm.nvfp4_norm_backward(y, x, w, r, y, dweight=dw, dsum=u)
            wait()
            lin[0].nvfp4_int8_quantize(y, q, s)
            wait()
            x.copy_(y)
            seen += [x.clone(), q.clone(), s.clone(), dw.clone()]
        torch.cuda.synchronize()
        return seen

    for n in (500, 60, 9):
        y.zero_(), u.zero_()
        want = chain(torch.cuda.synchronize, n)
        assert all(bool(torch.isfinite(t.float()).all()) for t in want)
        for _ in range(8):
            y.zero_(), u.zero_()
            assert all(torch.equal(a, b) for a, b in zip(chain(lambda: None, n), want))
    for h in (norm, act, *lin):
        assert h.nvfp4_moe_get_status() == (0, 0)
        h.close()
