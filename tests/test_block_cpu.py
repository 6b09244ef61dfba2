"""Host-side checks, without a GPU, of the operators around the 4-bit products: refusals, declarations, devices."""
import ctypes
import types

import pytest

import nvfp4_weight_only_w4a16_gb300 as P
from nvfp4_weight_only_w4a16_gb300.binding import Int8Config, NormConfig, RouteConfig, SwiGLUConfig

INV, SHAPE = "NVFP4_MOE_ERR_INVALID_ARG", "NVFP4_MOE_ERR_UNSUPPORTED_SHAPE"
GOOD = {
    "int8": (Int8Config, dict(out_features=272, in_features=256, max_tokens=64, out_dtype=0, device=0)),
    "route": (RouteConfig, dict(num_experts=64, top_k=4, groups=8, top_groups=2, group_top=2, score=0, renormalize=1,
                                scale=1.0, logits_dtype=0, device=0)),
    "norm": (NormConfig, dict(hidden=4096, eps=1e-6, act_dtype=0, device=0)),
    "swiglu": (SwiGLUConfig, dict(inter=1536, act_dtype=0, device=0)),
}


@pytest.fixture(scope="module")
def lib():
    P.build()
    return P.load_library()


def _create(lib, op, **kw):
    cls, base = GOOD[op]
    h = ctypes.c_void_p()
    return P.STATUS[getattr(lib, f"nvfp4_{op}_create")(ctypes.byref(cls(**{**base, **kw})), ctypes.byref(h))], h.value


@pytest.mark.parametrize("op,kw", [
    ("int8", dict(out_features=0)), ("int8", dict(out_features=24)), ("int8", dict(out_features=(1 << 20) + 16)),
    ("int8", dict(in_features=0)), ("int8", dict(in_features=8)), ("int8", dict(in_features=16400)),
    ("int8", dict(max_tokens=0)), ("int8", dict(max_tokens=(1 << 20) + 1)),
    ("route", dict(num_experts=0)), ("route", dict(num_experts=520)), ("route", dict(top_k=0)), ("route", dict(top_k=17)),
    ("route", dict(num_experts=8, groups=4, top_groups=1, top_k=3)), ("route", dict(groups=0)), ("route", dict(groups=7)),
    ("route", dict(groups=64)), ("route", dict(top_groups=0)), ("route", dict(top_groups=9)), ("route", dict(group_top=0)),
    ("route", dict(group_top=3)), ("route", dict(num_experts=8, groups=8, top_groups=4)),
    ("norm", dict(hidden=0)), ("norm", dict(hidden=12)), ("norm", dict(hidden=16392)),
    ("swiglu", dict(inter=0)), ("swiglu", dict(inter=24)), ("swiglu", dict(inter=16400)),
])
def test_shapes_that_are_refused(lib, op, kw):
    assert _create(lib, op, **kw) == (SHAPE, None)


@pytest.mark.parametrize("op,kw", [
    ("int8", dict(out_dtype=3)), ("int8", dict(out_dtype=-1)), ("int8", dict(device=-1)), ("int8", dict(device=4096)),
    ("route", dict(score=2)), ("route", dict(renormalize=2)), ("route", dict(scale=float("nan"))),
    ("route", dict(scale=float("inf"))), ("route", dict(logits_dtype=2)), ("route", dict(device=4096)),
    ("norm", dict(eps=-1.0)), ("norm", dict(eps=float("nan"))), ("norm", dict(eps=float("inf"))), ("norm", dict(act_dtype=2)),
    ("norm", dict(device=-1)), ("swiglu", dict(act_dtype=2)), ("swiglu", dict(device=4096)),
])
def test_arguments_that_are_refused(lib, op, kw):
    assert _create(lib, op, **kw) == (INV, None)


def test_nulls(lib):
    for op in GOOD:
        h = ctypes.c_void_p()
        create = getattr(lib, f"nvfp4_{op}_create")
        assert P.STATUS[create(None, ctypes.byref(h))] == INV
        assert P.STATUS[create(ctypes.byref(GOOD[op][0](**GOOD[op][1])), None)] == INV
    for name in P.header_functions():
        if name.split("_")[1] in GOOD and not name.endswith("create"):
            fn = getattr(lib, name)
            assert P.STATUS[fn(*[None if t is ctypes.c_void_p else 1 for t in fn.argtypes])] == INV, name


def test_the_header_declares_them(lib):
    names = P.header_functions()
    for n in ("int8_create", "int8_pack", "int8_quantize", "int8_forward", "route_create", "route_forward", "route_backward",
              "norm_create", "norm_forward", "norm_backward", "swiglu_create", "swiglu_forward", "swiglu_backward"):
        assert f"nvfp4_{n}" in names and hasattr(lib, f"nvfp4_{n}")


def test_plain_forms_against_values_worked_by_hand():
    np = pytest.importorskip("numpy")
    pytest.importorskip("torch")
    from tests.block_ops import checkpoint, codes, route, tables
    q, peak = codes(np.array([[254.0, 1.0, 3.0, -5.0, 0.5]]))
    assert q.tolist() == [[127, 0, 2, -2, 0]] and peak.tolist() == [254.0]      # 0.5, 1.5, -2.5: to even
    q, s = checkpoint(np.array([[0.0] * 128 + [np.inf, 1.0], [254.0] + [1.0] * 127 + [-2.0, 1.0]]))
    assert not q[0].any() and s[0, 0] == 0 and np.isnan(s[0, 1]) and q[1, 128:].tolist() == [-127, 64] and s[1, 0] == 2.0
    l = np.array([[1.0, 3.0, 2.0, 3.0, np.nan, -np.inf]])
    assert route(l, 3)[0].tolist() == [[1, 3, 2]]
    assert route(l, 6)[0].tolist() == [[1, 3, 2, 0, 5, 4]]
    ids, w = route(l, 2, score="sigmoid", bias=np.array([9.0, 0, 0, 0, 9.0, 8.0]))
    assert ids.tolist() == [[0, 5]] and np.allclose(w, [[1, 0]])
    assert route(l, 2, groups=3, top_groups=1)[0].tolist() == [[1, 0]]
    assert route(l, 2, groups=3, top_groups=1, group_top=2, bias=np.zeros(6), score="sigmoid")[0].tolist() == [[3, 2]]
    o, p, v = tables(np.array([[2, 0], [0, 1]]), 3)
    assert o.tolist() == [0, 2, 3, 4] and p.tolist() == [1, 2, 3, 0] and v.tolist() == [3, 0, 1, 2]


class Placed:
    """A CPU tensor that says it is on cuda:`device`."""

    def __init__(self, t, device):
        self._t, self._device = t, device

    def __getattr__(self, name):
        return getattr(self._t, name)

    def get_device(self):
        return self._device


def test_tensors_on_another_device_and_of_other_shapes_are_refused():
    torch = pytest.importorskip("torch")
    B, F, I8, I32 = torch.bfloat16, torch.float32, torch.int8, torch.int32
    reached = []

    def call(*a):
        reached.append(a)
        return 0

    def handle(cls, **fields):
        h = object.__new__(cls)
        h.lib = types.SimpleNamespace(**{n: call for n in P.header_functions()})
        h.h, h.device, h._int8, h._int32, h._f32, h._act, h._out = None, 1, I8, I32, F, B, B
        h._logits, h._x_types, h._current_stream = F, {B: 0}, lambda device: 0
        for k, v in fields.items():
            setattr(h, k, v)
        return h

    z = lambda shape, dt: torch.zeros(shape, dtype=dt)
    route, norm = handle(P.Route, E=8, k=2), handle(P.Norm, H=64)
    swiglu, lin = handle(P.SwiGLU, I=144, blocks=2), handle(P.Int8Linear, N=32, K=64)
    m = lambda dt, n=64: z((3, n), dt)
    calls = [
        (route.nvfp4_route_forward, dict(logits=z((3, 8), F), ids=z((3, 2), I32), weights=z((3, 2), F), offsets=z(9, I32),
                                         perm=z(6, I32), inv=z(6, I32), bias=z(8, F))),
        (route.nvfp4_route_backward, dict(logits=z((3, 8), F), ids=z((3, 2), I32), dweights=z((3, 2), F), dlogits=z((3, 8), F))),
        (norm.nvfp4_norm_forward, dict(x=m(B), weight=z(64, B), residual=m(B), sum=m(B), y=m(B), q=m(I8), q_scale=z(3, F), rstd=z(3, F))),
        (norm.nvfp4_norm_backward, dict(dy=m(B), sum=m(B), weight=z(64, B), rstd=z(3, F), dx=m(B), dweight=z(64, F), dsum=m(B))),
        (swiglu.nvfp4_swiglu_forward, dict(gate=m(B, 144), up=m(B, 144), out=m(B, 144), codes=z((3, 2, 144), I8), scales=z((3, 2, 2), F))),
        (swiglu.nvfp4_swiglu_backward, dict(codes=z((3, 2, 144), I8), scales=z((3, 2, 2), F), dh=m(B, 144), dgate=m(B, 144), dup=m(B, 144))),
        (lin.nvfp4_int8_pack, dict(w=z((32, 64), I8), w_scale=z(32, F), bias=z(32, F))),
        (lin.nvfp4_int8_quantize, dict(x=m(B), q=m(I8), q_scale=z(3, F))),
        (lin.nvfp4_int8_forward, dict(x=m(I8), x_scale=z(3, F), out=m(B, 32))),
    ]
    on = lambda t, d: Placed(t, d)
    for fn, kw in calls:
        fn(**{n: on(t, 1) for n, t in kw.items()})
    assert len(reached) == len(calls)
    del reached[:]
    for fn, kw in calls:
        for name, t in kw.items():
            others = [on(t, 0), on(t, -1), on(t.to(torch.float64), 1), on(torch.zeros((*t.shape[:-1], t.shape[-1] + 1), dtype=t.dtype), 1)]
            if t.dim() > 1:
                others.append(on(torch.zeros((t.shape[0] + 1, *t.shape[1:]), dtype=t.dtype), 1))
                others.append(on(torch.zeros((*t.shape[:-1], 2 * t.shape[-1]), dtype=t.dtype)[..., ::2], 1))
            for other in others:
                with pytest.raises(ValueError):
                    fn(**{n: other if n == name else on(v, 1) for n, v in kw.items()})
    assert not reached
