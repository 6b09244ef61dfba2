"""The 4-bit products used together, on the GPU: an MoE layer with its input
gradient built from the grouped products, and an INT4 linear behind it.

Bounds.  Each product against its own actual inputs: products.bound.  The layer
against the layer's own bars (test_gpu_parity).  The gradient end to end against
float64: the roundings that lie on its way, each at most half a step (BF16 2^-8
of the value) plus the products' FP32 summation, carried through the absolute
values of everything behind them; second-order terms are covered by 2% on top.
"""
import threading

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle as O
import nvfp4_weight_only_w4a16_gb300 as P
from synth import CONFIGS, make_inputs
from tests.products import DEV, bound, check, f64, int4_values, nvfp4_values
from tests.test_gpu_parity import assert_layer_close

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _t(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


class Layer:
    """gate, up and down as grouped handles, beside the whole layer's."""

    def __init__(self, cfg, weights, max_tokens):
        P.build()
        E, H, I, k = cfg.num_experts, cfg.hidden, cfg.inter, cfg.top_k
        self.moe = P.MoELayer(E, H, I, max_tokens, k, out_f32=True)
        P.upload_layer(self.moe, weights, DEV)
        rows = max_tokens * k
        mats = {"gate": (weights.w13_q[:, :I], weights.w13_s[:, :I], 0, I, H),
                "up": (weights.w13_q[:, I:], weights.w13_s[:, I:], 1, I, H),
                "down": (weights.w2_q, weights.w2_s, 2, H, I)}
        self.w = {}
        for name, (q, s, g, n, kk) in mats.items():
            h = P.Grouped(E, n, kk, rows, out_f32=True)
            gs = np.ascontiguousarray(weights.gscale[:, g], dtype=np.float32)
            h.nvfp4_grouped_pack(_t(q), _t(s), _t(gs))
            setattr(self, name, h)
            self.w[name] = nvfp4_values(q, s) * gs.astype(np.float64)[:, None, None]
        self.cfg = cfg

    def route(self, logits):
        T, k = logits.shape[0], self.cfg.top_k
        _, w, off, perm = self.moe.nvfp4_moe_debug_route(logits, T, k)
        perm = perm.long()
        return w.flatten()[perm][:, None], off, perm // k

    def forward(self, x, route):
        w, off, token = route
        rows, I, H = x[token], self.cfg.inter, self.cfg.hidden
        new = lambda n: torch.empty((rows.shape[0], n), device=DEV)
        g = self.gate.nvfp4_grouped_forward(rows, off, new(I))
        u = self.up.nvfp4_grouped_forward(rows, off, new(I))
        h = (torch.nn.functional.silu(g) * u).to(BF16)
        y = self.down.nvfp4_grouped_forward(h, off, new(H))
        out = torch.zeros((x.shape[0], H), device=DEV).index_add_(0, token, w * y)
        return out, (rows, g, u, h, y)

    def backward(self, dout, route, saved):
        w, off, token = route
        rows, g, u, _, _ = saved
        new = lambda n: torch.empty((rows.shape[0], n), device=DEV)
        dy = (w * dout[token]).to(BF16)
        dh = self.down.nvfp4_grouped_backward(dy, off, new(self.cfg.inter))
        s = torch.sigmoid(g)
        dg, du = (dh * u * s * (1 + g * (1 - s))).to(BF16), (dh * g * s).to(BF16)
        da = self.gate.nvfp4_grouped_backward(dg, off, new(self.cfg.hidden))
        db = self.up.nvfp4_grouped_backward(du, off, new(self.cfg.hidden))
        return torch.zeros_like(dout).index_add_(0, token, da + db), (dy, dh, dg, du, da, db)

    def status_ok(self):
        for h in (self.gate, self.up, self.down):
            assert h.nvfp4_moe_get_status()[0] == 0


@pytest.fixture(scope="module")
def tiny():
    cfg = CONFIGS["tiny"]
    return Layer(cfg, make_inputs(cfg).weights, 300)


def _products(off, x, w, got, what, fp16_rows=2.0 ** -38):
    off, x, got = off.cpu().numpy(), f64(x), f64(got)
    for e in range(len(off) - 1):
        s = slice(off[e], off[e + 1])
        if off[e + 1] > off[e]:
            y = x[s] @ w[e].T
            check(got[s], y, bound(y, x[s], w[e], torch.float32, fp16_rows), f"{what}, expert {e}")


@pytest.mark.parametrize("T", [1, 16, 300])   # streamed, streamed, tcgen05 GEMM
def test_layer_and_its_input_gradient(tiny, T):
    cfg = tiny.cfg.with_tokens(T)
    inp = make_inputs(cfg)
    x = _t(inp.x_bits.view(np.int16)).view(BF16)
    logits = _t(inp.logits)
    route = tiny.route(logits)
    out, saved = tiny.forward(x, route)
    whole = torch.empty_like(out)
    tiny.moe.nvfp4_moe_forward(logits, x, cfg.top_k, whole)
    torch.cuda.synchronize()
    ref = O.moe_forward(inp.logits, inp.x_bits, inp.weights, cfg.top_k)
    assert_layer_close(f64(out), ref, bf16_out=False)
    assert_layer_close(f64(out), f64(whole), bf16_out=False)
    w, off, token = route
    rows, g, u, h, y = saved
    _products(off, rows, tiny.w["gate"], g, "gate")
    _products(off, rows, tiny.w["up"], u, "up")
    _products(off, h, tiny.w["down"], y, "down")

    dout = torch.randn(out.shape, generator=torch.Generator(device=DEV).manual_seed(T), device=DEV)
    dx, (dy, dh, dg, du, da, db) = tiny.backward(dout, route, saved)
    tiny.status_ok()
    wt = {n: np.swapaxes(m, 1, 2) for n, m in tiny.w.items()}
    _products(off, dy, wt["down"], dh, "down's gradient", 0.0)
    _products(off, dg, wt["gate"], da, "gate's gradient", 0.0)
    _products(off, du, wt["up"], db, "up's gradient", 0.0)

    # end to end, in float64, with the bound of what the roundings do to it
    half, f32 = 2.0 ** -8, 2.0 ** -24
    offs, tok, ww = off.cpu().numpy(), token.cpu().numpy(), f64(w)
    X, D = f64(x), f64(dout)
    ref, tol = np.zeros_like(D), np.zeros_like(D)
    for e in range(cfg.num_experts):
        t = tok[offs[e]:offs[e + 1]]
        if not len(t):
            continue
        Wg, Wu, Wd = (tiny.w[n][e] for n in ("gate", "up", "down"))
        xr = X[t]
        g, u = xr @ Wg.T, xr @ Wu.T
        bg, bu = (bound(None, xr, m, torch.float32, 2.0 ** -38) for m in (Wg, Wu))
        dy = ww[offs[e]:offs[e + 1]] * D[t]
        bdy = (half + 2 * f32) * np.abs(dy)
        dh = dy @ Wd
        bdh = bdy @ np.abs(Wd) + bound(None, dy, Wd.T, torch.float32)
        s = 1 / (1 + np.exp(-g))
        p1 = s * (1 + g * (1 - s))          # the derivative of silu; its own is at most 1/2, silu's at most 1.1
        dg, du = dh * u * p1, dh * g * s
        flops = 16 * f32                     # of the elementwise FP32 arithmetic, relative to |dh u| (1 + |g|)
        bdg = bdh * np.abs(u * p1) + np.abs(dh) * (bu * np.abs(p1) + np.abs(u) * bg) + flops * np.abs(dh * u) * (1 + np.abs(g)) \
            + half * np.abs(dg)
        bdu = bdh * np.abs(g * s) + np.abs(dh) * 1.1 * bg + flops * np.abs(dh * g) + half * np.abs(du)
        d = dg @ Wg + du @ Wu
        b = bdg @ np.abs(Wg) + bdu @ np.abs(Wu) + bound(None, dg, Wg.T, torch.float32) + bound(None, du, Wu.T, torch.float32) \
            + f32 * np.abs(d)
        np.add.at(ref, t, d)
        np.add.at(tol, t, b)
    tol += cfg.top_k * f32 * np.abs(ref)
    check(f64(dx), ref, 1.02 * tol, "gradient of the layer's input")


def test_captured_layer_with_an_int4_linear_behind(tiny):
    """Forward, INT4 linear and backward in one graph on another stream, replayed with other tokens and routes."""
    cfg, T, N = tiny.cfg, 12, 208
    rng = np.random.default_rng(3)
    q = rng.integers(0, 256, (N, cfg.hidden // 2), dtype=np.uint8)
    scale = torch.from_numpy(rng.uniform(-0.1, 0.1, (N, cfg.hidden // 64))).to(DEV).to(BF16)
    zero = rng.integers(0, 16, (N, cfg.hidden // 64), dtype=np.uint8)
    head = P.Int4Linear(N, cfg.hidden, 64, out_f32=True)
    head.nvfp4_int4_pack(_t(q), scale, _t(zero))
    x, logits = torch.zeros((T, cfg.hidden), dtype=BF16, device=DEV), torch.zeros((T, cfg.num_experts), device=DEV)
    dout = torch.ones((T, cfg.hidden), device=DEV)
    z, mid = torch.empty((T, N), device=DEV), torch.empty((T, cfg.hidden), dtype=BF16, device=DEV)
    kept = {}

    def step():
        route = tiny.route(logits)
        out, saved = tiny.forward(x, route)
        mid.copy_(out)
        head.nvfp4_int4_forward(mid, z)
        kept["dx"], _ = tiny.backward(dout, route, saved)

    def fill(seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        x.copy_(torch.randn(x.shape, generator=g, device=DEV))
        logits.copy_(torch.randn(logits.shape, generator=g, device=DEV))

    torch.use_deterministic_algorithms(True, warn_only=True)   # index_add_ sums in one order
    try:
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            fill(0)
            step()
            stream.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                step()
            captured = kept["dx"]
            for seed in (1, 2, 3):
                fill(seed)
                graph.replay()
                stream.synchronize()
                got = z.clone(), captured.clone(), mid.clone()
                step()
                stream.synchronize()
                assert all(torch.equal(a, b) for a, b in zip(got, (z, kept["dx"], mid)))
                m = f64(mid)
                y = m @ int4_values(q, f64(scale), zero, 64).T
                check(f64(z), y, bound(y, m, int4_values(q, f64(scale), zero, 64), torch.float32, 2.0 ** -34,
                                       terms=int4_values(q, f64(scale), zero, 64, sign=1.0), rounds=2))
    finally:
        torch.use_deterministic_algorithms(False)
    tiny.status_ok()
    head.close()


@pytest.mark.parametrize("R,path", [(24, P.PATH_DECODE), (24, P.PATH_PREFILL), (500, P.PATH_PREFILL)])
def test_products_that_feed_each_other_without_a_kernel_between(R, path):
    """A launch may begin before the last one's end: what it reads of it, and overwrites under it, has to wait."""
    P.build()
    rng = np.random.default_rng(R)
    E, n, k = 4, 512, 1024
    pack = lambda N, K: tuple(_t(rng.integers(0, 256, (E, N, K // d), dtype=np.uint8) & m) for d, m in ((2, 255), (16, 0x27)))
    a, b = P.Grouped(E, n, k, R), P.Grouped(E, k, n, R)
    gs = torch.full((E,), 0.02, device=DEV)
    a.nvfp4_grouped_pack(*pack(n, k), gs)
    b.nvfp4_grouped_pack(*pack(k, n), gs)
    lin = P.Int4Linear(k, k, 128)
    lin.nvfp4_int4_pack(_t(rng.integers(0, 256, (k, k // 2), dtype=np.uint8)),
                        torch.from_numpy(rng.uniform(-0.01, 0.01, (k, k // 128))).to(DEV).to(BF16))
    for h in (a, b):
        h.nvfp4_moe_set_path(path)
    cuts = np.sort(rng.integers(0, R + 1, E - 1))
    off = _t(np.concatenate([[0], cuts, [R]]).astype(np.int32))
    x0 = torch.from_numpy(rng.standard_normal((R, k))).to(DEV).to(BF16)
    x, y, z = x0.clone(), torch.empty((R, n), dtype=BF16, device=DEV), torch.empty((R, k), dtype=BF16, device=DEV)

    def chain(sync):
        wait = torch.cuda.synchronize if sync else (lambda: None)
        x.copy_(x0)
        seen = []
        for _ in range(6):
            a.nvfp4_grouped_forward(x, off, y)
            wait()
            b.nvfp4_grouped_forward(y, off, z)
            wait()
            b.nvfp4_grouped_backward(z, off, y)
            wait()
            a.nvfp4_grouped_backward(y, off, x)      # overwrites the first product's input
            wait()
            lin.nvfp4_int4_forward(x[:16], z[:16])
            wait()
            x[:16].copy_(z[:16])
            seen.append(x.clone())
        torch.cuda.synchronize()
        return seen

    want = chain(True)
    assert bool(torch.isfinite(want[-1]).all()) and bool((want[-1] != 0).any())
    for _ in range(10):
        assert all(torch.equal(u, v) for u, v in zip(chain(False), want))
    for h in (a, b, lin):
        assert h.nvfp4_moe_get_status()[0] == 0
        h.close()


def test_host_threads_share_handles():
    """Calls on one handle from several host threads, each on a stream of its own: as if made one after the other."""
    P.build()
    rng = np.random.default_rng(8)
    E, n, k = 4, 512, 1024
    g = P.Grouped(E, n, k, 200)
    g.nvfp4_grouped_pack(_t(rng.integers(0, 256, (E, n, k // 2), dtype=np.uint8)),
                         _t(rng.integers(0, 0x40, (E, n, k // 16), dtype=np.uint8)), torch.full((E,), 0.02, device=DEV))
    lin = P.Int4Linear(n, k, 64)
    lin.nvfp4_int4_pack(_t(rng.integers(0, 256, (n, k // 2), dtype=np.uint8)),
                        torch.from_numpy(rng.uniform(-0.01, 0.01, (n, k // 64))).to(DEV).to(BF16))
    off = [_t(np.array(o, np.int32)) for o in ([0, 3, 3, 20, 24], [0, 100, 100, 130, 200])]
    xs = [torch.from_numpy(rng.standard_normal((r, k))).to(DEV).to(BF16) for r in (24, 200, 13)]
    dy = torch.from_numpy(rng.standard_normal((200, n))).to(DEV).to(BF16)
    new = lambda r, c: torch.empty((r, c), dtype=BF16, device=DEV)
    jobs = [lambda s: g.nvfp4_grouped_forward(xs[0], off[0], new(24, n), stream=s),
            lambda s: g.nvfp4_grouped_forward(xs[1], off[1], new(200, n), stream=s),
            lambda s: g.nvfp4_grouped_backward(dy, off[1], new(200, k), stream=s),
            lambda s: lin.nvfp4_int4_forward(xs[2], new(13, n), stream=s)]
    want = [j(None) for j in jobs]
    torch.cuda.synchronize()
    got = [None] * len(jobs)

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            outs = [jobs[i](s) for _ in range(50)]
            s.synchronize()
        got[i] = all(torch.equal(o, want[i]) for o in outs)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert got == [True] * len(jobs)
    for h in (g, lin):
        assert h.nvfp4_moe_get_status()[0] == 0
        h.close()
