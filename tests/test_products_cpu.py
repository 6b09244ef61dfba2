"""Host-side checks of the grouped and INT4 products that need no GPU."""
import ctypes

import numpy as np
import pytest

import nvfp4_weight_only_w4a16_gb300 as P
from nvfp4_weight_only_w4a16_gb300.binding import GroupedConfig, Int4Config

CODE = P.STATUS_CODE


@pytest.fixture(scope="module")
def lib():
    P.build()
    return P.load_library()


def _create(fn, cfg):
    h = ctypes.c_void_p()
    return P.STATUS[fn(ctypes.byref(cfg), ctypes.byref(h))], h.value


def _grouped(**kw):
    return GroupedConfig(**{**dict(num_experts=8, out_features=272, in_features=256, max_rows=64, out_dtype=0, device=0),
                            **kw})


def _int4(**kw):
    return Int4Config(**{**dict(out_features=272, in_features=256, group_size=64, max_tokens=16, act_dtype=0, out_f32=0,
                                device=0), **kw})


@pytest.mark.parametrize("kw", [
    dict(num_experts=0), dict(num_experts=257), dict(out_features=0), dict(out_features=24), dict(out_features=16400),
    dict(in_features=64), dict(in_features=192), dict(in_features=16512), dict(max_rows=0), dict(max_rows=(1 << 24) + 1),
])
def test_grouped_create_rejects_bad_shapes(lib, kw):
    assert _create(lib.nvfp4_grouped_create, _grouped(**kw)) == ("NVFP4_MOE_ERR_UNSUPPORTED_SHAPE", None)


@pytest.mark.parametrize("kw", [
    dict(out_features=0), dict(out_features=40), dict(out_features=(1 << 20) + 16), dict(in_features=64),
    dict(in_features=200), dict(in_features=16512), dict(group_size=16), dict(group_size=48), dict(group_size=256),
    dict(max_tokens=0), dict(max_tokens=17),
])
def test_int4_create_rejects_bad_shapes(lib, kw):
    assert _create(lib.nvfp4_int4_create, _int4(**kw)) == ("NVFP4_MOE_ERR_UNSUPPORTED_SHAPE", None)


def test_create_rejects_bad_types_devices_and_nulls(lib):
    inv = "NVFP4_MOE_ERR_INVALID_ARG"
    for kw in (dict(out_dtype=2), dict(device=-1), dict(device=4096)):
        assert _create(lib.nvfp4_grouped_create, _grouped(**kw)) == (inv, None)
    for kw in (dict(act_dtype=2), dict(out_f32=2), dict(device=-1), dict(device=4096)):
        assert _create(lib.nvfp4_int4_create, _int4(**kw)) == (inv, None)
    for fn in (lib.nvfp4_grouped_create, lib.nvfp4_int4_create):
        h = ctypes.c_void_p()
        assert P.STATUS[fn(None, ctypes.byref(h))] == inv
    assert P.STATUS[lib.nvfp4_grouped_create(ctypes.byref(_grouped()), None)] == inv
    assert P.STATUS[lib.nvfp4_int4_create(ctypes.byref(_int4()), None)] == inv


def test_null_handles(lib):
    inv = CODE["NVFP4_MOE_ERR_INVALID_ARG"]
    assert lib.nvfp4_grouped_pack(None, None, None, None, None) == inv
    assert lib.nvfp4_grouped_forward(None, 1, None, None, 128, None, 16, None) == inv
    assert lib.nvfp4_grouped_backward(None, 1, None, None, 16, None, 128, None) == inv
    assert lib.nvfp4_int4_pack(None, None, None, None, None) == inv
    assert lib.nvfp4_int4_forward(None, 1, None, 128, None, 16, None) == inv


def test_header_declares_the_products(lib):
    names = P.header_functions()
    for n in ("grouped_create", "grouped_pack", "grouped_forward", "grouped_backward", "int4_create", "int4_pack",
              "int4_forward"):
        assert f"nvfp4_{n}" in names and hasattr(lib, f"nvfp4_{n}")


def test_plain_forms_decode_the_formats():
    """The tests' own float64 decoders against values worked by hand."""
    torch = pytest.importorskip("torch")
    from tests.products import int4_values, nvfp4_values
    q = np.arange(16, dtype=np.uint8).reshape(1, 16)[:, ::2] | (np.arange(16, dtype=np.uint8).reshape(1, 16)[:, 1::2] << 4)
    s = np.array([[0x38]], np.uint8)                       # 1.0
    assert nvfp4_values(q, s).tolist() == [[0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6]]
    every = np.arange(127, dtype=np.uint8)                 # every finite positive E4M3 value
    want = torch.from_numpy(every).view(torch.float8_e4m3fn).double().numpy()
    ones = np.full((127, 8), 0x22, np.uint8)               # code 2: 1.0
    assert np.array_equal(nvfp4_values(ones, every.reshape(127, 1))[:, 0], want)
    w = int4_values(np.array([[0x0F, 0x80]], np.uint8), np.array([[2.0, 0.5]]), np.array([[1, 3]], np.uint8), 2)
    assert w.tolist() == [[28.0, -2.0, -1.5, 2.5]]
