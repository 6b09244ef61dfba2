"""Calls of the operators around the products that are refused on the host: nothing is launched, nothing written, and the
handle works afterwards.  All pointers are to memory of ours, larger than any of these calls would touch."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import nvfp4_weight_only_w4a16_gb300 as P

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INV, SHAPE, UNPACKED = "NVFP4_MOE_ERR_INVALID_ARG", "NVFP4_MOE_ERR_UNSUPPORTED_SHAPE", "NVFP4_MOE_ERR_NOT_PACKED"


@pytest.fixture(scope="module")
def room():
    P.build()
    return torch.zeros(1 << 22, dtype=torch.uint8, device=DEV)


def _refused(room, fn, base, changes):
    """base: the call's arguments, in order; changes: {argument: [(value, status), ..]}; p(k) below is 1 << 16 bytes each."""
    lib = P.load_library()
    for name, values in changes.items():
        for value, status in values:
            args = {**base, name: value}
            got = getattr(lib, fn)(*args.values())
            assert P.STATUS[got] == status, (fn, name, value, P.STATUS[got])
    torch.cuda.synchronize()
    assert not bool(room.any())


def _at(room):
    first = room.data_ptr()
    return lambda k, off=0: first + (k << 16) + off


def _rows(p, k, ld, align=16, cols=None):
    """What is refused of a matrix's pointer and stride."""
    return [(None, INV), (p(k, align // 2), INV)], [(cols - 8, INV), (ld + align // 4, INV), ((1 << 24) + 16, INV), (0, INV), (-ld, INV)]


def test_norm(room):
    p, H, T = _at(room), 64, 3
    n, lin = P.Norm(H), P.Int8Linear(16, H, 16)
    fwd = dict(h=n.h, T=T, x=p(0), ldx=H, res=p(1), ldr=H, w=p(2), sum=p(3), lds=H, y=p(4), ldy=H, q=p(5), ldq=H, qs=p(6), rstd=p(7), st=None)
    ch = dict(h=[(None, INV), (lin.h, INV)], T=[(-1, SHAPE), ((1 << 20) + 1, SHAPE)], w=[(None, INV), (p(2, 8), INV)],
              qs=[(None, INV), (p(6, 2), INV)], rstd=[(p(7, 2), INV)])
    for name, ld, k in (("x", "ldx", 0), ("res", "ldr", 1), ("sum", "lds", 3), ("y", "ldy", 4)):
        ptr, strides = _rows(p, k, H, cols=H)
        ch[name] = ptr if name in ("x", "sum") else ptr[1:]
        ch[ld] = strides
    ch["q"], ch["ldq"] = [(p(5, 4), INV)], [(H - 8, INV), (H + 4, INV), ((1 << 24) + 8, INV)]
    _refused(room, "nvfp4_norm_forward", fwd, ch)
    _refused(room, "nvfp4_norm_forward", {**fwd, "res": None}, dict(sum=[(p(3), INV)]))
    _refused(room, "nvfp4_norm_forward", {**fwd, "y": None}, dict(q=[(None, INV)]))
    back = dict(h=n.h, T=T, dy=p(0), ldd=H, sum=p(1), lds=H, w=p(2), rstd=p(3), dsum=p(4), ldr=H, dx=p(5), ldx=H, dw=p(6), st=None)
    ch = dict(h=[(None, INV), (lin.h, INV)], T=[(-1, SHAPE), ((1 << 20) + 1, SHAPE)], w=[(None, INV), (p(2, 8), INV)],
              rstd=[(None, INV), (p(3, 2), INV)], dw=[(p(6, 8), INV)])
    for name, ld, k in (("dy", "ldd", 0), ("sum", "lds", 1), ("dsum", "ldr", 4), ("dx", "ldx", 5)):
        ptr, strides = _rows(p, k, H, cols=H)
        ch[name] = ptr[1:] if name == "dsum" else ptr
        ch[ld] = strides
    _refused(room, "nvfp4_norm_backward", back, ch)
    q = dict(h=lin.h, T=T, x=p(0), dt=0, ldx=H, q=p(1), ldq=H, qs=p(2), st=None)
    ptr, strides = _rows(p, 0, H, cols=H)
    _refused(room, "nvfp4_int8_quantize", q, dict(h=[(None, INV), (n.h, INV)], T=[(-1, SHAPE), ((1 << 20) + 1, SHAPE)], x=ptr,
                                                  dt=[(2, INV), (-1, INV)], ldx=strides, q=[(None, INV), (p(1, 4), INV)],
                                                  ldq=[(H - 8, INV), (H + 4, INV)], qs=[(None, INV), (p(2, 2), INV)]))
    n.close()
    lin.close()


def test_swiglu(room):
    p, I, R = _at(room), 144, 3
    a, n = P.SwiGLU(I), P.Norm(64)
    fwd = dict(h=a.h, R=R, g=p(0), ldg=I, u=p(1), ldu=I, o=p(2), ldo=I, c=p(3), s=p(4), st=None)
    back = dict(h=a.h, R=R, c=p(0), s=p(1), d=p(2), ldd=I, g=p(3), ldg=I, u=p(4), ldu=I, st=None)
    common = dict(h=[(None, INV), (n.h, INV)], R=[(-1, SHAPE), ((1 << 24) + 1, SHAPE)])
    for fn, base, rows in (("nvfp4_swiglu_forward", fwd, (("g", "ldg", 0), ("u", "ldu", 1), ("o", "ldo", 2))),
                           ("nvfp4_swiglu_backward", back, (("d", "ldd", 2), ("g", "ldg", 3), ("u", "ldu", 4)))):
        ch = dict(common, c=[(None, INV), (base["c"] + 8, INV)], s=[(None, INV), (base["s"] + 2, INV)])
        for name, ld, k in rows:
            ch[name], ch[ld] = _rows(p, k, I, cols=I)
        _refused(room, fn, base, ch)
    a.close()
    n.close()


def test_route(room):
    p, E, k, T = _at(room), 16, 4, 3
    r, n = P.Route(E, k), P.Norm(64)
    fwd = dict(h=r.h, T=T, l=p(0), ld=E, b=p(1), ids=p(2), w=p(3), off=p(4), perm=p(5), inv=p(6), st=None)
    out = {name: [(None, INV), (fwd[name] + 2, INV)] for name in ("ids", "w", "off", "perm", "inv")}
    common = dict(h=[(None, INV), (n.h, INV)], T=[(-1, SHAPE), ((1 << 20) + 1, SHAPE)], l=[(None, INV), (p(0, 2), INV)],
                  ld=[(E - 1, INV), ((1 << 24) + 1, INV)])
    _refused(room, "nvfp4_route_forward", fwd, dict(common, b=[(p(1, 2), INV)], **out))
    back = dict(h=r.h, T=T, l=p(0), ld=E, ids=p(1), dw=p(2), dl=p(3), ldd=E, st=None)
    _refused(room, "nvfp4_route_backward", back, dict(common, ids=[(None, INV), (p(1, 2), INV)], dw=[(None, INV), (p(2, 2), INV)],
                                                      dl=[(None, INV), (p(3, 2), INV)], ldd=[(E - 1, INV), ((1 << 24) + 1, INV)]))
    r.close()
    n.close()


def test_int8(room):
    p, N, K, T = _at(room), 32, 64, 3
    lin, other = P.Int8Linear(N, K, 20), P.Int4Linear(32, 128, 32)
    fwd = dict(h=lin.h, T=T, x=p(0), ldx=K, xs=p(1), o=p(2), ldo=N, st=None)
    _refused(room, "nvfp4_int8_forward", fwd, dict(T=[(T, UNPACKED)]))
    pack = dict(h=lin.h, w=p(3), ws=p(4), b=p(5), st=None)
    _refused(room, "nvfp4_int8_pack", pack, dict(h=[(None, INV), (other.h, INV)], w=[(None, INV), (p(3, 8), INV)],
                                                 ws=[(None, INV), (p(4, 2), INV)], b=[(p(5, 2), INV)]))
    lin.nvfp4_int8_pack(torch.zeros((N, K), dtype=torch.int8, device=DEV), torch.zeros((N,), device=DEV))
    x, xs = _rows(p, 0, K, cols=K)
    o, os = _rows(p, 2, N, cols=N)
    _refused(room, "nvfp4_int8_forward", fwd, dict(h=[(None, INV), (other.h, INV)], T=[(-1, SHAPE), (21, SHAPE)], x=x,
                                                   ldx=xs + [(K + 8, INV)], xs=[(None, INV), (p(1, 2), INV)], o=o, ldo=os))
    assert P.STATUS[P.load_library().nvfp4_int4_forward(lin.h, 1, p(0), 128, p(1), 32, None)] == INV
    y = torch.ones((T, N), dtype=torch.bfloat16, device=DEV)
    lin.nvfp4_int8_forward(torch.ones((T, K), dtype=torch.int8, device=DEV), torch.ones((T,), device=DEV), y)
    assert not bool(y.any())
    lin.close()
    other.close()


def test_other_calls_refuse_these_handles(room):
    p = _at(room)
    lib = P.load_library()
    handles = [P.Norm(64), P.Route(16, 4), P.SwiGLU(16), P.Int8Linear(16, 16, 16)]
    for h in handles:
        assert P.STATUS[lib.nvfp4_moe_forward(h.h, p(0), 1, 1, p(1), p(2), None)] == INV
        assert P.STATUS[lib.nvfp4_linear_forward(h.h, 1, p(0), p(1), None)] == INV
        assert P.STATUS[lib.nvfp4_grouped_forward(h.h, 1, p(0), p(1), 128, p(2), 128, None)] == INV
        assert P.STATUS[lib.nvfp4_int4_forward(h.h, 1, p(0), 128, p(1), 128, None)] == INV
        assert P.STATUS[lib.nvfp4_moe_set_scoring(h.h, 0, 1, 1.0, None, None)] == INV
        assert P.STATUS[lib.nvfp4_moe_debug_packed_blob(h.h, p(0), 1 << 16, None)] == UNPACKED
        n = ctypes.c_uint32(7)
        assert P.STATUS[lib.nvfp4_moe_get_status(h.h, ctypes.byref(n))] == "NVFP4_MOE_OK" and n.value == 0
        h.close()
    assert not bool(room.any())


def test_views_that_do_not_start_on_16_bytes_are_refused():
    P.build()
    x = torch.zeros((4, 80), dtype=torch.bfloat16, device=DEV)
    n, w = P.Norm(64), torch.zeros((64,), dtype=torch.bfloat16, device=DEV)
    for view in (x[:, 1:65], torch.zeros((4, 66), dtype=torch.bfloat16, device=DEV)[:, :64]):
        with pytest.raises(P.Nvfp4MoeError, match="INVALID_ARG"):
            n.nvfp4_norm_forward(view, w, y=torch.empty((4, 64), dtype=torch.bfloat16, device=DEV))
    n.close()
