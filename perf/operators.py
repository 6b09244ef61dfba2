"""The 4-bit weight-only products outside the fused MoE layer, as measured cases.

Three operators:
  grouped_forward   y[r]  = g_e W_e   x[r]   for the rows r of expert e (rows sorted by expert, ragged counts)
  grouped_backward  dx[r] = g_e W_e^T dy[r]  its input gradient (the 4-bit weights are frozen)
  int4_linear       y[t]  = sum_k s[n, k // g] (q[n, k] - z[n, k // g]) x[t, k]
W_e is NVFP4: E2M1 codes, one E4M3 scale per 16 elements of a row, one FP32 scale g_e per expert.

`run` computes them in elementary FP32 torch operations, or with `own` set through the framework's calls.
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _grouped(name, op, experts, n, k, rows, zipf, spare=0, f32_out=False):
    return {"name": name, "op": op, "experts": experts, "n": n, "k": k, "rows": rows, "zipf": zipf, "spare": spare,
            "f32_out": f32_out}


def _int4(name, n, k, tokens, group, zeros, fp16, f32_out=False):
    return {"name": name, "op": "int4_linear", "n": n, "k": k, "tokens": tokens, "group": group, "zeros": zeros,
            "fp16": fp16, "f32_out": f32_out}


def listed():
    return [
        # 16 tokens x top-2 of the tiny layer's down products: latency alone
        _grouped("forward_tiny", "grouped_forward", 8, 256, 512, 32, 0.0),
        # one decode step of two tokens x top-8: the down products of the few experts it touches
        _grouped("forward_mtp_down", "grouped_forward", 128, 4096, 1536, 16, 0.0),
        # eight streams x two tokens x top-8: the gate (or up) product, most experts touched by a row or two
        _grouped("forward_c16_gate", "grouped_forward", 128, 1536, 4096, 128, 0.0),
        # a 1024-token prefill piece, mild imbalance: every expert, tens of rows each
        _grouped("forward_1k_gate", "grouped_forward", 128, 1536, 4096, 8192, 0.5),
        # a 16K-token prefill over 256 experts of Zipf popularity: hundreds of rows on average, thousands at the top
        _grouped("forward_16k_down", "grouped_forward", 256, 4096, 1536, 131072, 1.1),
        # odd sizes: a matrix that is no multiple of 128 rows, an odd row count, rows behind the last expert
        _grouped("backward_odd", "grouped_backward", 8, 272, 256, 37, 0.7, spare=5),
        # tuning adapters beside frozen experts: the gradient through the down products of 1024 tokens
        _grouped("backward_1k_down", "grouped_backward", 128, 4096, 1536, 8192, 0.5),
        # and through the gate products of 16K tokens
        _grouped("backward_16k_gate", "grouped_backward", 256, 1536, 4096, 131072, 1.1),
        # one token through a square projection: latency and bandwidth at their smallest
        _int4("int4_one_token", 4096, 4096, 1, 128, False, False),
        # a fused attention in-projection at a two-token step, asymmetric codes
        _int4("int4_in_proj_mtp", 12576, 4096, 2, 128, True, False),
        # a batch of 16 in FP16 with fine groups
        _int4("int4_batch16_g32", 8192, 8192, 16, 32, True, True),
        # an output head over a large vocabulary, unrounded logits
        _int4("int4_head", 131072, 4096, 4, 64, False, False, f32_out=True),
    ]


_MAX_WEIGHTS = 256 * 4096 * 1536       # the largest listed case's weights and products
_MAX_PRODUCTS = 131072 * 4096 * 1536


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["grouped_forward", "grouped_backward", "int4_linear"])
    if op == "int4_linear":
        while True:
            n, k = 16 * _log(rng, 1, 8192), 128 * _log(rng, 1, 128)
            if n * k <= 131072 * 4096:
                break
        return {"op": op, "n": n, "k": k, "tokens": _log(rng, 1, 16), "group": rng.choice([32, 64, 128]),
                "zeros": rng.random() < 0.5, "fp16": rng.random() < 0.5, "f32_out": rng.random() < 0.3}
    while True:
        e, n, k = _log(rng, 1, 256), 16 * _log(rng, 1, 256), 128 * _log(rng, 1, 32)
        rows = _log(rng, 1, 131072)
        if e * n * k <= _MAX_WEIGHTS and rows * n * k <= _MAX_PRODUCTS:
            break
    return {"op": op, "experts": e, "n": n, "k": k, "rows": rows, "zipf": round(rng.uniform(0.0, 1.2), 3),
            "spare": rng.choice([0, 0, 3, 40]), "f32_out": rng.random() < 0.3}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _popularity(case):
    ranks = torch.arange(1, case["experts"] + 1, dtype=torch.float64)
    p = ranks ** -case["zipf"]
    return p / p.sum()


def _encode_nvfp4(w):
    """FP32 [N][K] -> E2M1 codes [N][K/2] (element 2j in the low nibble), E4M3 scale bytes [N][K/16], tensor scale."""
    n, k = w.shape
    g = w.abs().amax() / (6.0 * 448.0)
    blocks = w.view(n, k // 16, 16)
    s = (blocks.abs().amax(dim=2) / 6.0 / g).to(torch.float8_e4m3fn)
    step = s.float() * g
    inv = torch.where(step > 0, 1.0 / step, torch.zeros_like(step))
    v = (blocks * inv.unsqueeze(2)).view(n, k)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
    code = torch.bucketize(v.abs(), edges).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
    return code[:, 0::2] | (code[:, 1::2] << 4), s.view(torch.uint8), g


def _grouped_inputs(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    e, n, k, rows = case["experts"], case["n"], case["k"], case["rows"]
    p = _popularity(case)[torch.randperm(e, generator=host)]
    counts = torch.bincount(torch.multinomial(p, rows, replacement=True, generator=host), minlength=e)
    w_q = torch.empty((e, n, k // 2), dtype=torch.uint8, device=DEV)
    w_s = torch.empty((e, n, k // 16), dtype=torch.uint8, device=DEV)
    gscale = torch.empty((e,), dtype=torch.float32, device=DEV)
    for i in range(e):
        w_q[i], w_s[i], gscale[i] = _encode_nvfp4(torch.randn((n, k), generator=gen, device=DEV) * 0.02)
    wide = k if case["op"] == "grouped_forward" else n
    x = torch.randn((rows + case["spare"], wide), generator=gen, device=DEV).to(torch.bfloat16)
    if case["op"] == "grouped_backward":
        x *= 2.0 ** -8                     # gradients are small next to activations
    offsets = torch.zeros((e + 1,), dtype=torch.int32)
    offsets[1:] = torch.cumsum(counts, 0)
    return w_q, w_s, gscale, x, offsets.to(DEV), offsets.tolist()


def _int4_inputs(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    n, k, g = case["n"], case["k"], case["group"]
    t = torch.float16 if case["fp16"] else torch.bfloat16
    w = torch.randn((n, k // g, g), generator=gen, device=DEV) * 0.02
    if case["zeros"]:                      # asymmetric: codes 0..15 over the group's range
        lo, hi = w.amin(dim=2), w.amax(dim=2)
        scale = ((hi - lo) / 15.0).to(t)
        zero = torch.round(-lo / scale.float()).clamp_(0, 15)
    else:                                  # symmetric about code 8
        scale = (w.abs().amax(dim=2) / 7.0).to(t)
        zero = torch.full_like(scale, 8.0, dtype=torch.float32)
    code = (torch.round(w / scale.float().unsqueeze(2)) + zero.unsqueeze(2)).clamp_(0, 15).to(torch.uint8).view(n, k)
    w_q = code[:, 0::2] | (code[:, 1::2] << 4)
    x = torch.randn((case["tokens"], k), generator=gen, device=DEV).to(t)
    return w_q, scale, zero.to(torch.uint8) if case["zeros"] else None, x


def prepare(case, seed):
    s = {"case": case}
    if case["op"] == "int4_linear":
        w_q, scale, zero, x = _int4_inputs(case, seed)
        t = torch.float32 if case["f32_out"] else x.dtype
        s.update(x=x, out=torch.zeros((case["tokens"], case["n"]), dtype=t, device=DEV))
        if own:
            import nvfp4_weight_only_w4a16_gb300 as fw
            s["linear"] = fw.Int4Linear(case["n"], case["k"], case["group"], act_f16=case["fp16"],
                                        out_f32=case["f32_out"])
            s["linear"].nvfp4_int4_pack(w_q, scale, zero)
        else:
            s.update(w_q=w_q, scale=scale, zero=zero)
        return s
    w_q, w_s, gscale, x, offsets, bounds = _grouped_inputs(case, seed)
    wide = case["n"] if case["op"] == "grouped_forward" else case["k"]
    t = torch.float32 if case["f32_out"] else torch.bfloat16
    s.update(x=x, offsets=offsets, out=torch.zeros((x.shape[0], wide), dtype=t, device=DEV))
    if own:
        import nvfp4_weight_only_w4a16_gb300 as fw
        s["experts"] = fw.Grouped(case["experts"], case["n"], case["k"], x.shape[0], out_f32=case["f32_out"])
        s["experts"].nvfp4_grouped_pack(w_q, w_s, gscale)
    else:
        s.update(w_q=w_q, w_s=w_s, gscale=gscale, bounds=bounds,
                 table=torch.tensor(E2M1, dtype=torch.float32, device=DEV))
    return s


# ---------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------

def _codes(w_q):
    return torch.stack((w_q & 15, w_q >> 4), dim=-1).flatten(-2)


def _run_grouped(s, forward):
    x, out = s["x"], s["out"]
    for e in range(s["case"]["experts"]):
        r0, r1 = s["bounds"][e], s["bounds"][e + 1]
        if r0 == r1:
            continue
        w = s["table"][_codes(s["w_q"][e]).int()]
        n, k = w.shape
        w = (w.view(n, k // 16, 16) * s["w_s"][e].view(torch.float8_e4m3fn).float().unsqueeze(2)).view(n, k)
        out[r0:r1] = s["gscale"][e] * (x[r0:r1].float() @ (w.t() if forward else w))
    return out


def _run_int4(s):
    case = s["case"]
    n, k, g = case["n"], case["k"], case["group"]
    q = _codes(s["w_q"]).float().view(n, k // g, g)
    zero = 8.0 if s["zero"] is None else s["zero"].float().unsqueeze(2)
    w = ((q - zero) * s["scale"].float().unsqueeze(2)).view(n, k)
    s["out"].copy_(s["x"].float() @ w.t())
    return s["out"]


def run(state):
    op = state["case"]["op"]
    if op == "int4_linear":
        if own:
            return state["linear"].nvfp4_int4_forward(state["x"], state["out"])
        return _run_int4(state)
    if own:
        if op == "grouped_forward":
            return state["experts"].nvfp4_grouped_forward(state["x"], state["offsets"], state["out"])
        return state["experts"].nvfp4_grouped_backward(state["x"], state["offsets"], state["out"])
    return _run_grouped(state, op == "grouped_forward")


# ---------------------------------------------------------------------------
# what a pass cannot do without, and its exact result
# ---------------------------------------------------------------------------

def work(case):
    n, k = case["n"], case["k"]
    if case["op"] == "int4_linear":
        t, groups = case["tokens"], n * (k // case["group"])
        out = 4 if case["f32_out"] else 2
        return {"bytes": n * k / 2 + groups * (3 if case["zeros"] else 2) + 2 * t * k + out * t * n,
                "flops": 2 * t * n * k}
    rows, p = case["rows"], _popularity(case)
    touched = float((1.0 - (1.0 - p) ** rows).sum())
    inner, outer = (k, n) if case["op"] == "grouped_forward" else (n, k)
    out = 4 if case["f32_out"] else 2
    return {"bytes": touched * n * k * 9 / 16 + rows * (2 * inner + out * outer) + 4 * (case["experts"] + 1),
            "flops": 2 * rows * n * k}


def _value_e2m1(code):
    """(-1)^s * 2^(e-1) * (1 + m/2) for e > 0, (-1)^s * m/2 for e = 0."""
    c = code.to(torch.int64)
    e, m = (c >> 1) & 3, (c & 1).double()
    mag = torch.where(e > 0, (1.0 + 0.5 * m) * (2.0 ** (e - 1).double()), 0.5 * m)
    return torch.where((c & 8) != 0, -mag, mag)


def _value_e4m3(byte):
    """2^(e-7) * (1 + m/8) for e > 0, 2^-6 * m/8 for e = 0 (the encoder makes no negative or NaN scale)."""
    b = byte.to(torch.int64)
    e, m = (b >> 3) & 15, (b & 7).double()
    return torch.where(e > 0, (1.0 + m / 8.0) * (2.0 ** (e - 7).double()), m / 8.0 * 2.0 ** -6)


def exact(case, seed):
    if 2.0 * case["n"] * case["k"] * case.get("rows", case.get("tokens")) > 4e12:
        return None                        # FP64 runs at about a TFLOP/s
    if case["op"] == "int4_linear":
        w_q, scale, zero, x = _int4_inputs(case, seed)
        y = torch.empty((case["tokens"], case["n"]), dtype=torch.float64, device=DEV)
        for a in range(0, case["n"], 4096):
            q = w_q[a:a + 4096]
            codes = torch.empty((q.shape[0], case["k"]), dtype=torch.float64, device=DEV)
            codes[:, 0::2], codes[:, 1::2] = (q % 16).double(), (q // 16).double()
            if zero is None:
                codes -= 8.0
            else:
                codes -= zero[a:a + 4096].double().repeat_interleave(case["group"], dim=1)
            codes *= scale[a:a + 4096].double().repeat_interleave(case["group"], dim=1)
            y[:, a:a + 4096] = x.double() @ codes.T
        return y
    w_q, w_s, gscale, x, _, bounds = _grouped_inputs(case, seed)
    forward = case["op"] == "grouped_forward"
    y = torch.zeros((x.shape[0], case["n"] if forward else case["k"]), dtype=torch.float64, device=DEV)
    for e in range(case["experts"]):
        rows = slice(bounds[e], bounds[e + 1])
        if rows.start == rows.stop:
            continue
        w = torch.empty((case["n"], case["k"]), dtype=torch.float64, device=DEV)
        w[:, 0::2], w[:, 1::2] = _value_e2m1(w_q[e] % 16), _value_e2m1(w_q[e] // 16)
        w *= _value_e4m3(w_s[e]).repeat_interleave(16, dim=1) * gscale[e].double()
        y[rows] = x[rows].double() @ (w.T if forward else w)
    return y
