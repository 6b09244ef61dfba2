"""What stands around the 4-bit products in a block of the model, as measured cases.

Four operators:
  route        scores = softmax or sigmoid of a token's logits; the top-k of scores + bias, within the best groups of
               experts where there are groups; the chosen scores, renormalised, as weights; and the tables that the
               grouped products and the combination read.  Backward: the weights' gradient to the logits.
  norm         h = x + residual; y = w h / sqrt(mean(h^2) + eps), in 16 bits and in 8 with a scale a token.
               Backward: the gradients of h and of w.
  swiglu       h = silu(gate) up, with gate and up kept for the backward pass in 8 bits, a scale for every 128
               elements of a row.  Backward, from those: the gradients of gate and up.
  int8_linear  y[t][n] = sx[t] sw[n] sum_k xq[t][k] wq[n][k] + bias[n], the sum exact.  Where a case says `dynamic`, x
               comes in 16 bits and is quantised first.

`run` computes them in elementary torch operations, or with `own` set through the framework's calls.  8-bit codes are
integers, returned as such with their scales beside them.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 128     # elements of a row that share a checkpoint's scale


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _route(name, op, tokens, experts, k, score, bias, groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0,
           bf16=False):
    return {"name": name, "op": op, "tokens": tokens, "experts": experts, "k": k, "score": score, "bias": bias,
            "groups": groups, "top_groups": top_groups, "group_top": group_top, "renorm": renorm, "scale": scale,
            "bf16": bf16}


def _norm(name, op, tokens, hidden, residual, y, q, fp16=False):
    return {"name": name, "op": op, "tokens": tokens, "hidden": hidden, "residual": residual, "y": y, "q": q,
            "fp16": fp16}


def _swiglu(name, op, rows, inter, fp16=False):
    return {"name": name, "op": op, "rows": rows, "inter": inter, "fp16": fp16}


def _int8(name, n, k, tokens, dynamic, bias, out):
    return {"name": name, "op": "int8_linear", "n": n, "k": k, "tokens": tokens, "dynamic": dynamic, "bias": bias,
            "out": out}


def listed():
    return [
        # one decode step of two tokens: 128 experts, top-8, the layer's own rule; latency alone
        _route("route_mtp", "route_forward", 2, 128, 8, "softmax", False),
        # a prefill of 16384 tokens over 256 experts in 8 groups, balanced by a bias
        _route("route_16k_groups", "route_forward", 16384, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5),
        # tuning the router on an odd batch: all scores take part in each weight's gradient
        _route("route_backward", "route_backward", 8191, 256, 8, "softmax", False, renorm=False, bf16=True),
        # one decode step of two tokens: the residual added, normalised, and straight into an 8-bit product
        _norm("norm_mtp_int8", "norm_forward", 2, 4096, True, False, True),
        # a prefill of 16384 tokens whose result goes to 16-bit products (router, experts) and to 8-bit ones
        _norm("norm_16k", "norm_forward", 16384, 4096, True, True, True),
        # its gradient on an odd batch, the residual branch's added
        _norm("norm_backward", "norm_backward", 8191, 4096, True, False, False),
        # eight streams x two tokens x top-8 rows of the experts
        _swiglu("swiglu_c16", "swiglu_forward", 128, 1536),
        # 16384 tokens x top-8 rows
        _swiglu("swiglu_16k", "swiglu_forward", 131072, 1536),
        _swiglu("swiglu_backward_16k", "swiglu_backward", 131072, 1536),
        # a square projection, one token
        _int8("int8_decode", 4096, 4096, 1, False, False, "bf16"),
        # the fused input projection, eight streams x two tokens, from 16-bit activations
        _int8("int8_in_proj_c16", 12576, 4096, 16, True, True, "bf16"),
        # the same at a prefill of 16384 tokens
        _int8("int8_in_proj_16k", 12576, 4096, 16384, False, False, "bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    case = _drawn(rng)
    del case["name"]
    return case


def _drawn(rng):
    op = rng.choice(["route_forward", "route_forward", "route_backward", "norm_forward", "norm_forward", "norm_backward",
                     "swiglu_forward", "swiglu_backward", "int8_linear", "int8_linear", "int8_linear"])
    if op.startswith("route"):
        while True:
            e, t = rng.choice([8, 16, 60, 64, 72, 128, 160, 256, 384, 512]), _log(rng, 1, 32768)
            if e * t <= 16384 * 256:
                break
        groups = rng.choice([g for g in (1, 1, 2, 4, 6, 8, 16) if e % g == 0 and e // g >= 2])
        top = groups if groups == 1 else rng.randint(1, groups - 1)
        return _route("", op, t, e, rng.randint(1, min(16, top * (e // groups))), rng.choice(["softmax", "sigmoid"]),
                      rng.random() < 0.5, groups, top, rng.choice([1, 2]), rng.random() < 0.6, rng.choice([1.0, 2.5]),
                      rng.random() < 0.4)
    if op.startswith("norm"):
        while True:
            h, t = 8 * _log(rng, 8, 2048), _log(rng, 1, 65536)
            if h * t <= (16384 if op == "norm_forward" else 8191) * 4096:
                break
        q = rng.random() < 0.6
        return _norm("", op, t, h, rng.random() < 0.7, not q or rng.random() < 0.4, q, rng.random() < 0.3)
    if op.startswith("swiglu"):
        while True:
            i, r = 16 * _log(rng, 4, 1024), _log(rng, 1, 262144)
            if i * r <= 131072 * 1536:
                break
        return _swiglu("", op, r, i, rng.random() < 0.3)
    while True:
        n, k, t = 16 * _log(rng, 1, 8192), 16 * _log(rng, 4, 1024), _log(rng, 1, 32768)
        if n * k <= 131072 * 4096 and t * n * k <= 16384 * 12576 * 4096 and t * max(n, k) <= 1 << 28:
            break
    return _int8("", n, k, t, rng.random() < 0.4, rng.random() < 0.4, rng.choice(["bf16", "f16", "f32"]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _act(case):
    return torch.float16 if case["fp16"] else torch.bfloat16


def _out_type(case):
    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[case["out"]]


def _route_inputs(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    t, e, k = case["tokens"], case["experts"], case["k"]
    popular = torch.randn((e,), generator=gen, device=DEV) * 0.5
    logits = torch.randn((t, e), generator=gen, device=DEV) + popular
    if case["bf16"]:
        logits = logits.to(torch.bfloat16)
    # a balancing bias works against what is popular
    bias = -0.1 * popular + 0.01 * torch.randn((e,), generator=gen, device=DEV) if case["bias"] else None
    dweights = torch.randn((t, k), generator=gen, device=DEV) * 2.0 ** -8
    # the choice that a backward pass is given: any k different experts a token
    ids = torch.rand((t, e), generator=gen, device=DEV).argsort(dim=1)[:, :k].to(torch.int32).contiguous()
    return logits, bias, dweights, ids


def _norm_inputs(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    t, h, dt = case["tokens"], case["hidden"], _act(case)
    x = torch.randn((t, h), generator=gen, device=DEV).to(dt)
    residual = (torch.randn((t, h), generator=gen, device=DEV) * 3.0).to(dt)
    weight = (1.0 + 0.2 * torch.randn((h,), generator=gen, device=DEV)).to(dt)
    return x, residual, weight, gen


def _swiglu_inputs(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    r, i, dt = case["rows"], case["inter"], _act(case)
    gate, up, dh = ((torch.randn((r, i), generator=gen, device=DEV) * s).to(dt) for s in (1.5, 1.0, 2.0 ** -8))
    return gate, up, dh


def _int8_inputs(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    n, k, t = case["n"], case["k"], case["tokens"]
    w = torch.randn((n, k), generator=gen, device=DEV)
    w_scale = w.abs().amax(dim=1) / 127.0
    w_q = torch.round(w / w_scale[:, None]).to(torch.int8)
    del w
    w_scale *= 0.02
    x = torch.randn((t, k), generator=gen, device=DEV).to(torch.bfloat16)
    x_q = x_scale = None
    if not case["dynamic"]:
        x_scale = x.float().abs().amax(dim=1) / 127.0
        x_q = torch.round(x.float() / x_scale[:, None]).to(torch.int8)
    bias = torch.randn((n,), generator=gen, device=DEV) * 0.1 if case["bias"] else None
    return w_q, w_scale, bias, x, x_q, x_scale


EPS = 1e-6


def prepare(case, seed):
    s = {"case": case}
    op = case["op"]
    if own:
        import nvfp4_weight_only_w4a16_gb300 as fw
    new = lambda shape, dt: torch.zeros(shape, dtype=dt, device=DEV)
    if op.startswith("route"):
        logits, bias, dweights, ids = _route_inputs(case, seed)
        t, e, k = case["tokens"], case["experts"], case["k"]
        s.update(logits=logits, bias=bias)
        if op == "route_backward":
            s.update(ids=ids, dweights=dweights, dlogits=new((t, e), logits.dtype))
        else:
            i32 = torch.int32
            s.update(ids=new((t, k), i32), weights=new((t, k), torch.float32), offsets=new((e + 1,), i32),
                     perm=new((t * k,), i32), inv=new((t * k,), i32))
        if own:
            s["route"] = fw.Route(e, k, score=case["score"], renormalize=case["renorm"], scale=case["scale"],
                                  groups=case["groups"], top_groups=case["top_groups"], group_top=case["group_top"],
                                  logits_bf16=case["bf16"])
    elif op.startswith("norm"):
        x, residual, weight, gen = _norm_inputs(case, seed)
        t, h, dt = case["tokens"], case["hidden"], _act(case)
        s.update(x=x, residual=residual if case["residual"] else None, weight=weight)
        if op == "norm_forward":
            s.update(sum=new((t, h), dt) if case["residual"] else None, y=new((t, h), dt) if case["y"] else None,
                     q=new((t, h), torch.int8) if case["q"] else None,
                     q_scale=new((t,), torch.float32) if case["q"] else None, rstd=new((t,), torch.float32))
        else:   # x is the forward's sum, whose 1 / sqrt(..) the forward has left
            s["rstd"] = torch.rsqrt(x.float().square().mean(dim=1) + EPS)
            s["dy"] = (torch.randn((t, h), generator=gen, device=DEV) * 2.0 ** -8).to(dt)
            s["residual"] = (residual * 2.0 ** -8).to(dt) if case["residual"] else None
            s.update(dx=new((t, h), dt), dweight=new((h,), torch.float32))
        if own:
            s["norm"] = fw.Norm(h, EPS, act_f16=case["fp16"])
    elif op.startswith("swiglu"):
        gate, up, dh = _swiglu_inputs(case, seed)
        r, i, dt = case["rows"], case["inter"], _act(case)
        s.update(codes=new((r, 2, i), torch.int8), scales=new((r, 2, -(-i // BLOCK)), torch.float32))
        if op == "swiglu_forward":
            s.update(gate=gate, up=up, h=new((r, i), dt))
        else:
            for j, v in enumerate((gate, up)):
                q, scale = _checkpoint(v)
                s["codes"][:, j], s["scales"][:, j] = q, scale
            s.update(dh=dh, dgate=new((r, i), dt), dup=new((r, i), dt))
        if own:
            s["swiglu"] = fw.SwiGLU(i, act_f16=case["fp16"])
    else:
        w_q, w_scale, bias, x, x_q, x_scale = _int8_inputs(case, seed)
        t, n, k = case["tokens"], case["n"], case["k"]
        s.update(out=new((t, n), _out_type(case)))
        if case["dynamic"]:
            s.update(x=x, x_q=new((t, k), torch.int8), x_scale=new((t,), torch.float32))
        else:
            s.update(x_q=x_q, x_scale=x_scale)
        if own:
            s["linear"] = fw.Int8Linear(n, k, t, out=case["out"])
            s["linear"].nvfp4_int8_pack(w_q, w_scale, bias)
        else:
            s.update(w_q=w_q, w_scale=w_scale, bias=bias)
    return s


# ---------------------------------------------------------------------------
# the operators, plain
# ---------------------------------------------------------------------------

def _scores(case, logits, dt):
    l = logits.to(dt)
    if case["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    ex = torch.exp(l - l.amax(dim=1, keepdim=True))
    return ex / ex.sum(dim=1, keepdim=True)


def _route_forward(s):
    case, logits = s["case"], s["logits"]
    t, e, k, g = case["tokens"], case["experts"], case["k"], case["groups"]
    score = _scores(case, logits, torch.float64)      # in 64 bits: which of two experts is ahead may be close
    # both scores increase with the logit, so without a bias the logits order the experts
    choice = logits.double() if s["bias"] is None else score + s["bias"].double()
    if case["top_groups"] < g:
        # one member a group: as for the experts; two: the sum of their scores and biases
        rated = choice if case["group_top"] == 1 or s["bias"] is not None else score
        best = torch.sort(rated.view(t, g, e // g), dim=2, descending=True)[0][:, :, :case["group_top"]].sum(dim=2)
        kept = torch.sort(best, dim=1, descending=True, stable=True)[1][:, :case["top_groups"]]
        out = torch.ones((t, g), dtype=torch.bool, device=DEV).scatter_(1, kept, False)
        choice = choice.masked_fill(out.repeat_interleave(e // g, dim=1), -math.inf)
    ids = torch.sort(choice, dim=1, descending=True, stable=True)[1][:, :k]
    w = torch.gather(score, 1, ids)
    if case["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    s["weights"].copy_(w * case["scale"])
    s["ids"].copy_(ids)
    flat = ids.reshape(-1)
    perm = torch.sort(flat, stable=True)[1]
    s["perm"].copy_(perm)
    s["inv"][perm] = torch.arange(t * k, dtype=torch.int32, device=DEV)
    s["offsets"][1:] = torch.cumsum(torch.bincount(flat, minlength=e), 0)
    return {n: s[n] for n in ("ids", "weights", "offsets", "perm", "inv")}


def _route_backward(s):
    case, ids = s["case"], s["ids"].long()
    score = _scores(case, s["logits"], torch.float32)
    chosen, dw = torch.gather(score, 1, ids), s["dweights"] * case["scale"]
    if case["renorm"]:
        total = chosen.sum(dim=1, keepdim=True)
        ds = (dw - (dw * chosen).sum(dim=1, keepdim=True) / total) / total
    else:
        ds = dw
    dscore = torch.zeros_like(score).scatter_(1, ids, ds)
    if case["score"] == "sigmoid":
        dl = dscore * score * (1.0 - score)
    else:
        dl = score * (dscore - (dscore * score).sum(dim=1, keepdim=True))
    s["dlogits"].copy_(dl)
    return s["dlogits"]


def _to_int8(p, peak):
    """round(127 p / peak) of values in 64 bits; zeros where the peak is zero."""
    return torch.round(torch.where(peak > 0, 127.0 * p / peak, torch.zeros_like(p)))


def _norm_forward(s):
    case, h = s["case"], s["x"]
    if case["residual"]:
        h = (h.float() + s["residual"].float()).to(h.dtype)
        s["sum"].copy_(h)
    rstd = torch.rsqrt(h.float().square().mean(dim=1) + EPS)
    s["rstd"].copy_(rstd)
    if case["y"]:
        s["y"].copy_(h.float() * rstd[:, None] * s["weight"].float())
    if case["q"]:
        p = h.double() * s["weight"].double()          # in 64 bits: a code may lie next to the border of two
        peak = p.abs().amax(dim=1)
        s["q"].copy_(_to_int8(p, peak[:, None]))
        s["q_scale"].copy_(peak * rstd / 127.0)
    return {n: s[n] for n in ("sum", "y", "q", "q_scale", "rstd") if s[n] is not None}


def _norm_backward(s):
    x, dy, r = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    g = dy * s["weight"].float()
    dx = r * g - x * (r ** 3 / x.shape[1]) * (g * x).sum(dim=1, keepdim=True)
    if s["case"]["residual"]:
        dx = dx + s["residual"].float()
    s["dx"].copy_(dx)
    s["dweight"].copy_((dy * x * r).sum(dim=0))
    return s["dx"], s["dweight"]


def _blocks(v):
    """[R][I] as [R][blocks][128], the last block filled up with zeros."""
    r, i = v.shape
    return torch.nn.functional.pad(v, (0, -i % BLOCK)).view(r, -1, BLOCK)


def _checkpoint(v):
    b = _blocks(v.float())
    peak = b.abs().amax(dim=2)
    # 127 v is exact in 32 bits; the quotient is taken in 64, for codes next to the border of two
    q = torch.round(torch.where(peak[:, :, None] > 0, (127.0 * b).double() / peak[:, :, None].double(), 0.0))
    return q.to(torch.int8).view(v.shape[0], -1)[:, :v.shape[1]], peak / 127.0


def _swiglu_forward(s):
    g, u = s["gate"].float(), s["up"].float()
    s["h"].copy_(g / (1.0 + torch.exp(-g)) * u)
    s["codes"][:, 0], s["scales"][:, 0] = _checkpoint(s["gate"])
    s["codes"][:, 1], s["scales"][:, 1] = _checkpoint(s["up"])
    return s["h"], s["codes"], s["scales"]


def _kept(s, j):
    i = s["case"]["inter"]
    return s["codes"][:, j].float() * s["scales"][:, j].repeat_interleave(BLOCK, dim=1)[:, :i]


def _swiglu_backward(s):
    g, u, dh = _kept(s, 0), _kept(s, 1), s["dh"].float()
    sig = 1.0 / (1.0 + torch.exp(-g))
    s["dgate"].copy_(dh * u * sig * (1.0 + g * (1.0 - sig)))
    s["dup"].copy_(dh * g * sig)
    return s["dgate"], s["dup"]


def _int8_linear(s):
    if s["case"]["dynamic"]:
        x = s["x"].float()
        peak = x.abs().amax(dim=1)
        s["x_q"].copy_(_to_int8(x.double(), peak[:, None].double()))
        s["x_scale"].copy_(peak / 127.0)
    y = s["x_q"].float() @ s["w_q"].float().t()
    y = y * s["x_scale"][:, None] * s["w_scale"]
    if s["bias"] is not None:
        y = y + s["bias"]
    s["out"].copy_(y)
    return [s["out"]] + ([s["x_q"], s["x_scale"]] if s["case"]["dynamic"] else [])


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"route_forward": _route_forward, "route_backward": _route_backward, "norm_forward": _norm_forward,
                "norm_backward": _norm_backward, "swiglu_forward": _swiglu_forward,
                "swiglu_backward": _swiglu_backward, "int8_linear": _int8_linear}[op](s)
    if op == "route_forward":
        s["route"].nvfp4_route_forward(s["logits"], s["ids"], s["weights"], s["offsets"], s["perm"], s["inv"],
                                       bias=s["bias"])
        return {n: s[n] for n in ("ids", "weights", "offsets", "perm", "inv")}
    if op == "route_backward":
        return s["route"].nvfp4_route_backward(s["logits"], s["ids"], s["dweights"], s["dlogits"])
    if op == "norm_forward":
        s["norm"].nvfp4_norm_forward(s["x"], s["weight"], residual=s["residual"], sum=s["sum"], y=s["y"], q=s["q"],
                                     q_scale=s["q_scale"], rstd=s["rstd"])
        return {n: s[n] for n in ("sum", "y", "q", "q_scale", "rstd") if s[n] is not None}
    if op == "norm_backward":
        s["norm"].nvfp4_norm_backward(s["dy"], s["x"], s["weight"], s["rstd"], s["dx"], dweight=s["dweight"],
                                      dsum=s["residual"])
        return s["dx"], s["dweight"]
    if op == "swiglu_forward":
        s["swiglu"].nvfp4_swiglu_forward(s["gate"], s["up"], s["h"], codes=s["codes"], scales=s["scales"])
        return s["h"], s["codes"], s["scales"]
    if op == "swiglu_backward":
        s["swiglu"].nvfp4_swiglu_backward(s["codes"], s["scales"], s["dh"], s["dgate"], s["dup"])
        return s["dgate"], s["dup"]
    if s["case"]["dynamic"]:
        s["linear"].nvfp4_int8_quantize(s["x"], s["x_q"], s["x_scale"])
    s["linear"].nvfp4_int8_forward(s["x_q"], s["x_scale"], s["out"])
    return [s["out"]] + ([s["x_q"], s["x_scale"]] if s["case"]["dynamic"] else [])


# ---------------------------------------------------------------------------
# what a pass cannot do without, and its exact result
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op.startswith("route"):
        t, e, k, b = case["tokens"], case["experts"], case["k"], 2 if case["bf16"] else 4
        if op == "route_backward":
            return {"bytes": t * (2 * e * b + 8 * k), "flops": 8 * t * e}
        return {"bytes": t * (e * b + 16 * k) + 4 * (e + 1) + (4 * e if case["bias"] else 0), "flops": 8 * t * e}
    if op.startswith("norm"):
        t, h = case["tokens"], case["hidden"]
        if op == "norm_backward":
            return {"bytes": t * (h * (6 + (2 if case["residual"] else 0)) + 4) + 6 * h, "flops": 10 * t * h}
        return {"bytes": t * (h * (2 + (4 if case["residual"] else 0) + (2 if case["y"] else 0) + (1 if case["q"] else 0))
                              + (8 if case["q"] else 4)) + 2 * h, "flops": 6 * t * h}
    if op.startswith("swiglu"):
        r, i = case["rows"], case["inter"]
        return {"bytes": r * (8 * i + 8 * -(-i // BLOCK)), "flops": 10 * r * i}
    t, n, k = case["tokens"], case["n"], case["k"]
    return {"bytes": n * k + t * k * (3 if case["dynamic"] else 1) + t * n * (4 if case["out"] == "f32" else 2)
            + 4 * n * (2 if case["bias"] else 1) + 4 * t, "flops": 2 * t * n * k}


def _exact_scores(case, logits):
    """Row by row of exponents in 64 bits: sigmoid as 1 / (1 + e^-l) by the sign of l, softmax by log-sum-exp."""
    l = logits.double()
    if case["score"] == "sigmoid":
        z = torch.exp(-l.abs())
        return torch.where(l >= 0, 1.0 / (1.0 + z), z / (1.0 + z))
    top = l.max(dim=1, keepdim=True)[0]
    return torch.exp(l - top - torch.log(torch.exp(l - top).sum(dim=1, keepdim=True)))


def _exact_route(case, seed):
    logits, bias, dweights, ids = _route_inputs(case, seed)
    score = _exact_scores(case, logits)
    if case["op"] == "route_forward":
        t, e, g = case["tokens"], case["experts"], case["groups"]
        key = logits.double() if bias is None else score + bias.double()
        if case["top_groups"] < g:
            rated = (key if case["group_top"] == 1 or bias is not None else score).view(t, g, e // g)
            first, at = rated.max(dim=2)
            best = first
            if case["group_top"] == 2:
                best = first + rated.scatter(2, at.unsqueeze(2), -math.inf).amax(dim=2)
            ahead = (best[:, None, :] > best[:, :, None]).sum(dim=2)      # groups ahead of each, ties apart
            first_tied = torch.tril(best[:, None, :] == best[:, :, None], diagonal=-1).sum(dim=2)
            lost = (ahead + first_tied) >= case["top_groups"]
            key = torch.where(lost.repeat_interleave(e // g, dim=1), -math.inf, key)
        order = torch.argsort(-key, dim=1, stable=True)[:, :case["k"]]
        w = score.take_along_dim(order, dim=1)
        if case["renorm"]:
            w /= w.sum(dim=1, keepdim=True)
        return {"ids": None, "weights": case["scale"] * w, "offsets": None, "perm": None, "inv": None}
    at = ids.long()
    up = torch.zeros_like(score)
    up.scatter_(1, at, case["scale"] * dweights.double())
    mask = torch.zeros_like(score)
    mask.scatter_(1, at, 1.0)
    if case["renorm"]:                  # w_j = s_j / S: dw_j / ds_i = (delta_ij - w_j) / S
        share = score * mask
        total = share.sum(dim=1, keepdim=True)
        up = mask * (up - (up * share / total).sum(dim=1, keepdim=True)) / total
    if case["score"] == "sigmoid":
        z = torch.exp(-logits.double().abs())
        return up * z / (1.0 + z) ** 2
    return score * up - score * (score * up).sum(dim=1, keepdim=True)


def _exact_norm(case, seed):
    x, residual, weight, gen = _norm_inputs(case, seed)
    w = weight.double()
    if case["op"] == "norm_forward":
        h = x.double()
        if case["residual"]:
            h = (h + residual.double()).to(x.dtype).double()        # the sum is kept in 16 bits
        rms = (torch.linalg.vector_norm(h, dim=1) ** 2 / case["hidden"] + EPS).sqrt()
        y = h / rms[:, None] * w
        res = {"sum": h if case["residual"] else None, "y": y if case["y"] else None, "q": None,
               "q_scale": y.abs().max(dim=1)[0] / 127.0 if case["q"] else None, "rstd": 1.0 / rms}
        return {n: v for n, v in res.items() if v is not None}
    t, hidden = case["tokens"], case["hidden"]
    r = torch.rsqrt(x.float().square().mean(dim=1) + EPS).double()      # an input of the backward pass
    dy = (torch.randn((t, hidden), generator=gen, device=DEV) * 2.0 ** -8).to(x.dtype).double()
    n = x.double() * r[:, None]
    dn = dy * w
    dx = r[:, None] * (dn - n * torch.einsum("th,th->t", dn, n)[:, None] / hidden)
    if case["residual"]:
        dx += (residual * 2.0 ** -8).to(x.dtype).double()
    return dx, torch.einsum("th,th->h", dy, n)


def _exact_swiglu(case, seed):
    gate, up, dh = _swiglu_inputs(case, seed)
    if case["op"] == "swiglu_forward":
        peaks = torch.stack([torch.stack([c.abs().amax(dim=1) for c in v.double().split(BLOCK, dim=1)], dim=1)
                             for v in (gate, up)], dim=1)
        h = torch.empty(gate.shape, dtype=torch.float64, device=DEV)
        for a in range(0, case["rows"], 8192):
            g = gate[a:a + 8192].double()
            h[a:a + 8192] = g * torch.special.expit(g) * up[a:a + 8192].double()
        return h, None, peaks / 127.0
    dg, du = (torch.empty(gate.shape, dtype=torch.float64, device=DEV) for _ in range(2))
    for a in range(0, case["rows"], 8192):
        kept = []
        for v in (gate, up):
            q, scale = _checkpoint(v[a:a + 8192])                      # inputs of the backward pass
            kept.append(q.double() * scale.double().repeat_interleave(BLOCK, dim=1)[:, :case["inter"]])
        g, u = kept
        d, s = dh[a:a + 8192].double(), torch.special.expit(g)
        dg[a:a + 8192] = d * u * (s + g * s * torch.special.expit(-g))
        du[a:a + 8192] = d * g * s
    return dg, du


def _exact_int8(case, seed):
    w_q, w_scale, bias, x, x_q, x_scale = _int8_inputs(case, seed)
    first = None
    if case["dynamic"]:
        first = x.double().abs().max(dim=1)[0] / 127.0
        x_q = torch.round(x.double() / first[:, None])                 # the codes that the product is of
        x_scale = first
    y = torch.empty((case["tokens"], case["n"]), dtype=torch.float64, device=DEV)
    for a in range(0, case["n"], 4096):
        part = x_q.double() @ w_q[a:a + 4096].double().T
        y[:, a:a + 4096] = part * x_scale.double()[:, None] * w_scale[a:a + 4096].double()
        if bias is not None:
            y[:, a:a + 4096] += bias[a:a + 4096].double()
    return [y] + ([None, first] if case["dynamic"] else [])


def exact(case, seed):
    op = case["op"]
    if op == "int8_linear":
        if 2.0 * case["tokens"] * case["n"] * case["k"] > 4e12:
            return None                 # FP64 runs at about a TFLOP/s
        return _exact_int8(case, seed)
    return (_exact_route if op.startswith("route") else _exact_norm if op.startswith("norm") else _exact_swiglu)(case, seed)
