"""ctypes binding of libnvfp4moe.so: argument marshalling only.

Every function here turns torch tensors into device pointers and sizes and
calls the C entry point of the same name; all arithmetic of the layer runs in
the library's CUDA kernels.  There is no fallback: if the library cannot be
loaded, or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import os
import re

from .build import LIB, ROOT

STATUS = {
    0: "NVFP4_MOE_OK", 1: "NVFP4_MOE_ERR_INVALID_ARG", 2: "NVFP4_MOE_ERR_UNSUPPORTED_SHAPE",
    3: "NVFP4_MOE_ERR_NOT_PACKED", 4: "NVFP4_MOE_ERR_WORKSPACE", 5: "NVFP4_MOE_ERR_CUDA",
    6: "NVFP4_MOE_ERR_TIMEOUT", 7: "NVFP4_MOE_ERR_BAD_SCALE", 8: "NVFP4_MOE_ERR_NOT_IMPLEMENTED",
    9: "NVFP4_MOE_ERR_DEVICE_CHECK",
}
STATUS_CODE = {v: k for k, v in STATUS.items()}
PATH_AUTO, PATH_DECODE, PATH_PREFILL = 0, 1, 2
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
HEADER = os.path.join(ROOT, "include", "nvfp4_moe.h")


class Nvfp4MoeError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


class Config(ctypes.Structure):
    _fields_ = [("num_experts", ctypes.c_int), ("hidden", ctypes.c_int), ("inter", ctypes.c_int),
                ("max_tokens", ctypes.c_int), ("max_top_k", ctypes.c_int),
                ("decode_max_tokens", ctypes.c_int), ("logits_dtype", ctypes.c_int),
                ("device", ctypes.c_int), ("out_dtype", ctypes.c_int),
                ("num_shared_experts", ctypes.c_int)]


class LinearConfig(ctypes.Structure):
    _fields_ = [("out_features", ctypes.c_int), ("in_features", ctypes.c_int), ("max_tokens", ctypes.c_int),
                ("decode_max_tokens", ctypes.c_int), ("out_dtype", ctypes.c_int), ("device", ctypes.c_int)]


class GroupedConfig(ctypes.Structure):
    _fields_ = [("num_experts", ctypes.c_int), ("out_features", ctypes.c_int), ("in_features", ctypes.c_int),
                ("max_rows", ctypes.c_int), ("out_dtype", ctypes.c_int), ("device", ctypes.c_int)]


class Int4Config(ctypes.Structure):
    _fields_ = [("out_features", ctypes.c_int), ("in_features", ctypes.c_int), ("group_size", ctypes.c_int),
                ("max_tokens", ctypes.c_int), ("act_dtype", ctypes.c_int), ("out_f32", ctypes.c_int),
                ("device", ctypes.c_int)]


class Int8Config(ctypes.Structure):
    _fields_ = [("out_features", ctypes.c_int), ("in_features", ctypes.c_int), ("max_tokens", ctypes.c_int),
                ("out_dtype", ctypes.c_int), ("device", ctypes.c_int)]


class RouteConfig(ctypes.Structure):
    _fields_ = [("num_experts", ctypes.c_int), ("top_k", ctypes.c_int), ("groups", ctypes.c_int),
                ("top_groups", ctypes.c_int), ("group_top", ctypes.c_int), ("score", ctypes.c_int),
                ("renormalize", ctypes.c_int), ("scale", ctypes.c_float), ("logits_dtype", ctypes.c_int),
                ("device", ctypes.c_int)]


class NormConfig(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int), ("eps", ctypes.c_float), ("act_dtype", ctypes.c_int),
                ("device", ctypes.c_int)]


class SwiGLUConfig(ctypes.Structure):
    _fields_ = [("inter", ctypes.c_int), ("act_dtype", ctypes.c_int), ("device", ctypes.c_int)]


_lib = None


def header_functions():
    """Names of the functions include/nvfp4_moe.h declares."""
    with open(HEADER) as f:
        text = f.read()
    return sorted(set(re.findall(r"\b(nvfp4_(?:moe|linear|grouped|int4|int8|route|norm|swiglu)_[a-z_0-9]+)\s*\(", text)))


def load_library(path: str | None = None):
    """Load libnvfp4moe.so (raises if it is missing or incomplete)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB
    if not os.path.exists(p):
        raise FileNotFoundError(f"{p} is missing: run __graft_entry__.build() (nvcc, sm_103a) first")
    lib = ctypes.CDLL(p)
    vp, i, f, ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_int64
    sigs = {
        "nvfp4_moe_create": (i, [ctypes.POINTER(Config), ctypes.POINTER(vp)]),
        "nvfp4_moe_pack": (i, [vp, vp, vp, vp, vp, vp, vp]),
        "nvfp4_moe_forward": (i, [vp, vp, i, i, vp, vp, vp]),
        "nvfp4_moe_forward_host": (i, [vp, vp, i, i, vp, vp, vp]),
        "nvfp4_moe_get_status": (i, [vp, ctypes.POINTER(ctypes.c_uint32)]),
        "nvfp4_moe_set_path": (i, [vp, i]),
        "nvfp4_moe_status_string": (ctypes.c_char_p, [i]),
        "nvfp4_moe_last_error": (ctypes.c_char_p, [vp]),
        "nvfp4_moe_destroy": (None, [vp]),
        "nvfp4_moe_debug_route": (i, [vp, vp, i, i, vp, vp, vp, vp, vp]),
        "nvfp4_moe_debug_dequant": (i, [vp, i, i, vp, vp]),
        "nvfp4_moe_debug_intermediates": (i, [vp, vp, vp, vp]),
        "nvfp4_moe_debug_set_fault": (i, [vp, i]),
        "nvfp4_moe_set_profiling": (i, [vp, i]),
        "nvfp4_moe_debug_packed_blob": (i, [vp, vp, ctypes.c_size_t, vp]),
        "nvfp4_moe_forward_decode_static": (i, [vp, vp, i, i, i, vp, i, i, i, vp, vp, vp]),
        "nvfp4_moe_static_get_status": (i, [ctypes.POINTER(ctypes.c_uint32)]),
        "nvfp4_moe_static_debug_set_fault": (i, [i]),
        "nvfp4_moe_debug_poison_workspace": (i, [vp, i, vp]),
        "nvfp4_moe_decode_status_word": (i, [ctypes.c_uint32]),
        "nvfp4_moe_debug_trace": (i, [vp, ctypes.POINTER(ctypes.c_uint64), ctypes.c_size_t,
                                      ctypes.POINTER(ctypes.c_size_t)]),
        "nvfp4_moe_get_stage_times": (i, [vp, ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_int)]),
        "nvfp4_moe_set_scoring": (i, [vp, i, i, f, vp, vp]),
        "nvfp4_moe_set_router": (i, [vp, vp, vp]),
        "nvfp4_moe_set_act_quant": (i, [vp, vp, vp]),
        "nvfp4_moe_forward_routed": (i, [vp, i, i, vp, vp, vp]),
        "nvfp4_moe_debug_logits": (i, [vp, vp, vp]),
        "nvfp4_linear_create": (i, [ctypes.POINTER(LinearConfig), ctypes.POINTER(vp)]),
        "nvfp4_linear_pack": (i, [vp, vp, vp, vp, vp]),
        "nvfp4_linear_forward": (i, [vp, i, vp, vp, vp]),
        "nvfp4_grouped_create": (i, [ctypes.POINTER(GroupedConfig), ctypes.POINTER(vp)]),
        "nvfp4_grouped_pack": (i, [vp, vp, vp, vp, vp]),
        "nvfp4_grouped_forward": (i, [vp, i, vp, vp, ll, vp, ll, vp]),
        "nvfp4_grouped_backward": (i, [vp, i, vp, vp, ll, vp, ll, vp]),
        "nvfp4_int4_create": (i, [ctypes.POINTER(Int4Config), ctypes.POINTER(vp)]),
        "nvfp4_int4_pack": (i, [vp, vp, vp, vp, vp]),
        "nvfp4_int4_forward": (i, [vp, i, vp, ll, vp, ll, vp]),
        "nvfp4_int8_create": (i, [ctypes.POINTER(Int8Config), ctypes.POINTER(vp)]),
        "nvfp4_int8_pack": (i, [vp, vp, vp, vp, vp]),
        "nvfp4_int8_quantize": (i, [vp, i, vp, i, ll, vp, ll, vp, vp]),
        "nvfp4_int8_forward": (i, [vp, i, vp, ll, vp, vp, ll, vp]),
        "nvfp4_route_create": (i, [ctypes.POINTER(RouteConfig), ctypes.POINTER(vp)]),
        "nvfp4_route_forward": (i, [vp, i, vp, ll, vp, vp, vp, vp, vp, vp, vp]),
        "nvfp4_route_backward": (i, [vp, i, vp, ll, vp, vp, vp, ll, vp]),
        "nvfp4_norm_create": (i, [ctypes.POINTER(NormConfig), ctypes.POINTER(vp)]),
        "nvfp4_norm_forward": (i, [vp, i, vp, ll, vp, ll, vp, vp, ll, vp, ll, vp, ll, vp, vp, vp]),
        "nvfp4_norm_backward": (i, [vp, i, vp, ll, vp, ll, vp, vp, vp, ll, vp, ll, vp, vp]),
        "nvfp4_swiglu_create": (i, [ctypes.POINTER(SwiGLUConfig), ctypes.POINTER(vp)]),
        "nvfp4_swiglu_forward": (i, [vp, i, vp, ll, vp, ll, vp, ll, vp, vp, vp]),
        "nvfp4_swiglu_backward": (i, [vp, i, vp, vp, vp, ll, vp, ll, vp, ll, vp]),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path is None:
        _lib = lib
    return lib


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return ctypes.c_void_p(t.data_ptr())


def _whole(t, shape, dtype, device, what):
    """Address of a contiguous tensor of this shape and type on cuda:`device`."""
    if t.shape != shape or t.dtype is not dtype:
        raise ValueError(f"{what}: expected {shape} {dtype}, got {tuple(t.shape)} {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{what}: expected a CUDA tensor on the handle's device, cuda:{device}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous tensor")
    return t.data_ptr()


def _whole_or_none(t, shape, dtype, device, what):
    return None if t is None else _whole(t, shape, dtype, device, what)


def _rows_like(t, shape, dtype, device, what):
    """(address, row stride) of a matrix of this shape on cuda:`device` whose rows are contiguous; (None, 0) of None."""
    if t is None:
        return None, 0
    if t.shape != shape or t.dtype is not dtype:
        raise ValueError(f"{what}: expected {shape} {dtype}, got {tuple(t.shape)} {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{what}: expected a CUDA tensor on the handle's device, cuda:{device}")
    ld, one = t.stride()
    if one != 1:
        raise ValueError(f"{what}: expected contiguous rows")
    # a single row has no stride to speak of
    return t.data_ptr(), ld if shape[0] > 1 else -(-shape[1] // 8) * 8


def _rows(t, cols, dtype, device, what):
    """(address, row stride, rows) of a matrix [rows][cols] on cuda:`device` whose rows are contiguous.

    Each of a tensor's attributes costs some 0.1 us, and these calls' smallest take 4 us, so none is asked for twice."""
    shape = t.shape
    if len(shape) != 2 or shape[1] != cols or t.dtype != dtype:
        raise ValueError(f"{what}: expected [rows][{cols}] {dtype}, got {tuple(shape)} {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{what}: expected a CUDA tensor on the handle's device, cuda:{device}")
    ld, one = t.stride()
    if one != 1:
        raise ValueError(f"{what}: expected contiguous rows")
    rows = shape[0]
    # a single row has no stride to speak of
    return t.data_ptr(), ld if rows > 1 else -(-cols // 8) * 8, rows


def _host_ptr(t):
    """A page-locked CPU tensor's address (the library checks that CUDA maps it)."""
    if t.is_cuda or not t.is_pinned():
        raise ValueError("expected a page-locked (pinned) CPU tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None, device=None):
    """`stream`, or the current one of `device` (default: the current device)."""
    import torch
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


class MoELayer:
    """One handle of the library (nvfp4_moe_create ... nvfp4_moe_destroy)."""

    def __init__(self, num_experts, hidden, inter, max_tokens, max_top_k, decode_max_tokens=16,
                 logits_bf16=False, device=0, out_f32=False, num_shared_experts=0):
        self.lib = load_library()
        self.cfg = Config(num_experts, hidden, inter, max_tokens, max_top_k, decode_max_tokens,
                          1 if logits_bf16 else 0, device, 1 if out_f32 else 0, num_shared_experts)
        self.out_f32 = out_f32
        self.E, self.H, self.I = num_experts, hidden, inter
        self.S = num_shared_experts  # the shared expert is expert E of the blob
        self.device = device
        h = ctypes.c_void_p()
        st = self.lib.nvfp4_moe_create(ctypes.byref(self.cfg), ctypes.byref(h))
        if st != 0:
            raise Nvfp4MoeError(st, "nvfp4_moe_create: " + self.lib.nvfp4_moe_status_string(st).decode())
        self.h = h

    def _check(self, st, what):
        if st != 0:
            msg = self.lib.nvfp4_moe_last_error(self.h).decode()
            raise Nvfp4MoeError(st, f"{what}: {msg}")

    def close(self):
        if getattr(self, "h", None):
            self.lib.nvfp4_moe_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def nvfp4_moe_pack(self, w13_q, w13_s, w2_q, w2_s, gscale, stream=None):
        st = self.lib.nvfp4_moe_pack(self.h, _ptr(w13_q), _ptr(w13_s), _ptr(w2_q), _ptr(w2_s),
                                     _ptr(gscale), _stream(stream))
        self._check(st, "nvfp4_moe_pack")

    def nvfp4_moe_forward(self, logits, x, top_k, out, stream=None):
        T = x.shape[0]
        st = self.lib.nvfp4_moe_forward(self.h, _ptr(logits), T, top_k, _ptr(x), _ptr(out), _stream(stream))
        self._check(st, "nvfp4_moe_forward")
        return out

    def nvfp4_moe_forward_host(self, logits, x, top_k, out, stream=None):
        """nvfp4_moe_forward on pinned CPU tensors, read and written in place by the decode kernel."""
        T = x.shape[0]
        st = self.lib.nvfp4_moe_forward_host(self.h, _host_ptr(logits), T, top_k, _host_ptr(x), _host_ptr(out),
                                             _stream(stream))
        self._check(st, "nvfp4_moe_forward_host")
        return out

    def nvfp4_moe_forward_raw(self, logits_ptr, T, top_k, x_ptr, out_ptr, stream_handle):
        """Pointer-level call (for benchmarks that time the bare ABI)."""
        return self.lib.nvfp4_moe_forward(self.h, ctypes.c_void_p(logits_ptr), T, top_k, ctypes.c_void_p(x_ptr),
                                          ctypes.c_void_p(out_ptr), ctypes.c_void_p(stream_handle))

    def nvfp4_moe_get_status(self):
        n = ctypes.c_uint32(0)
        st = self.lib.nvfp4_moe_get_status(self.h, ctypes.byref(n))
        return st, int(n.value)

    def nvfp4_moe_set_path(self, path):
        self._check(self.lib.nvfp4_moe_set_path(self.h, path), "nvfp4_moe_set_path")

    def nvfp4_moe_debug_route(self, logits, T, top_k, stream=None):
        import torch
        dev = logits.device
        K = top_k + self.S  # slots per token; the shared expert's is last
        ids = torch.empty((T, K), dtype=torch.int32, device=dev)
        w = torch.empty((T, K), dtype=torch.float32, device=dev)
        off = torch.empty((self.E + self.S + 1,), dtype=torch.int32, device=dev)
        perm = torch.empty((T * K,), dtype=torch.int32, device=dev)
        st = self.lib.nvfp4_moe_debug_route(self.h, _ptr(logits), T, top_k, _ptr(ids), _ptr(w), _ptr(off),
                                            _ptr(perm), _stream(stream))
        self._check(st, "nvfp4_moe_debug_route")
        return ids, w, off, perm

    def nvfp4_moe_debug_trace(self):
        import numpy as np
        n = 152 * 16 * 16 * 4
        buf = (ctypes.c_uint64 * n)()
        got = ctypes.c_size_t(0)
        self._check(self.lib.nvfp4_moe_debug_trace(self.h, buf, n, ctypes.byref(got)), "nvfp4_moe_debug_trace")
        return np.frombuffer(buf, dtype=np.uint64)[:got.value].copy()

    def nvfp4_moe_debug_packed_blob(self, stream=None):
        import torch
        n = (self.E + self.S) * 3 * self.H * self.I * 9 // 16
        out = torch.empty((n,), dtype=torch.uint8, device=f"cuda:{self.device}")
        st = self.lib.nvfp4_moe_debug_packed_blob(self.h, _ptr(out), n, _stream(stream))
        self._check(st, "nvfp4_moe_debug_packed_blob")
        return out

    def nvfp4_moe_debug_dequant(self, expert, which, via_bf16=False, stream=None):
        import torch
        n, k = (self.H, self.I) if which == 2 else (self.I, self.H)
        out = torch.empty((n, k), dtype=torch.float32, device=f"cuda:{self.device}")
        st = self.lib.nvfp4_moe_debug_dequant(self.h, expert, which | (4 if via_bf16 else 0), _ptr(out),
                                              _stream(stream))
        self._check(st, "nvfp4_moe_debug_dequant")
        return out

    def nvfp4_moe_debug_intermediates(self, rows, stream=None):
        import torch
        hid = torch.empty((rows, self.I), dtype=torch.float32, device=f"cuda:{self.device}")
        y = torch.empty((rows, self.H), dtype=torch.float32, device=f"cuda:{self.device}")
        st = self.lib.nvfp4_moe_debug_intermediates(self.h, _ptr(hid), _ptr(y), _stream(stream))
        self._check(st, "nvfp4_moe_debug_intermediates")
        return hid, y

    def nvfp4_moe_set_profiling(self, on):
        self._check(self.lib.nvfp4_moe_set_profiling(self.h, 1 if on else 0), "nvfp4_moe_set_profiling")

    def nvfp4_moe_get_stage_times(self):
        ms = (ctypes.c_float * 4)()
        n = ctypes.c_int(0)
        self._check(self.lib.nvfp4_moe_get_stage_times(self.h, ms, ctypes.byref(n)), "nvfp4_moe_get_stage_times")
        return [float(v) for v in ms], int(n.value)

    def nvfp4_moe_set_scoring(self, score="softmax", renormalize=True, scale=1.0, bias=None, stream=None):
        """score: "softmax" | "sigmoid"; bias: a CUDA float32 tensor [num_experts] or None."""
        code = {"softmax": SCORE_SOFTMAX, "sigmoid": SCORE_SIGMOID}[score]
        st = self.lib.nvfp4_moe_set_scoring(self.h, code, 1 if renormalize else 0, float(scale), _ptr(bias),
                                            _stream(stream))
        self._check(st, "nvfp4_moe_set_scoring")

    def nvfp4_moe_set_act_quant(self, input_scale, stream=None):
        """input_scale: a CUDA float32 tensor [num_experts][2] (W4A4), or None (W4A16)."""
        st = self.lib.nvfp4_moe_set_act_quant(self.h, _ptr(input_scale), _stream(stream))
        self._check(st, "nvfp4_moe_set_act_quant")

    def nvfp4_moe_set_router(self, w_router, stream=None):
        """w_router: a CUDA BF16 tensor [num_experts][hidden]."""
        self._check(self.lib.nvfp4_moe_set_router(self.h, _ptr(w_router), _stream(stream)), "nvfp4_moe_set_router")

    def nvfp4_moe_forward_routed(self, x, top_k, out, stream=None):
        st = self.lib.nvfp4_moe_forward_routed(self.h, x.shape[0], top_k, _ptr(x), _ptr(out), _stream(stream))
        self._check(st, "nvfp4_moe_forward_routed")
        return out

    def nvfp4_moe_forward_routed_raw(self, T, top_k, x_ptr, out_ptr, stream_handle):
        """Pointer-level call (for benchmarks that time the bare ABI)."""
        return self.lib.nvfp4_moe_forward_routed(self.h, T, top_k, ctypes.c_void_p(x_ptr), ctypes.c_void_p(out_ptr),
                                                 ctypes.c_void_p(stream_handle))

    def nvfp4_moe_debug_logits(self, T, stream=None):
        import torch
        out = torch.empty((T, self.E), dtype=torch.float32, device=f"cuda:{self.device}")
        self._check(self.lib.nvfp4_moe_debug_logits(self.h, _ptr(out), _stream(stream)), "nvfp4_moe_debug_logits")
        return out

    def nvfp4_moe_debug_poison_workspace(self, byte=0xFF, stream=None):
        self._check(self.lib.nvfp4_moe_debug_poison_workspace(self.h, int(byte), _stream(stream)),
                    "nvfp4_moe_debug_poison_workspace")

    def nvfp4_moe_debug_set_fault(self, fault):
        self._check(self.lib.nvfp4_moe_debug_set_fault(self.h, fault), "nvfp4_moe_debug_set_fault")


class Linear(MoELayer):
    """A dense W4A16 NVFP4 linear handle (nvfp4_linear_create ... nvfp4_moe_destroy)."""

    def __init__(self, out_features, in_features, max_tokens, decode_max_tokens=16, device=0, out_f32=False):
        self.lib = load_library()
        self.cfg = LinearConfig(out_features, in_features, max_tokens, decode_max_tokens, 1 if out_f32 else 0, device)
        self.out_f32 = out_f32
        self.N, self.K = out_features, in_features
        self.device = device
        h = ctypes.c_void_p()
        st = self.lib.nvfp4_linear_create(ctypes.byref(self.cfg), ctypes.byref(h))
        if st != 0:
            raise Nvfp4MoeError(st, "nvfp4_linear_create: " + self.lib.nvfp4_moe_status_string(st).decode())
        self.h = h

    def nvfp4_linear_pack(self, w_q, w_s, gscale, stream=None):
        st = self.lib.nvfp4_linear_pack(self.h, _ptr(w_q), _ptr(w_s), _ptr(gscale), _stream(stream))
        self._check(st, "nvfp4_linear_pack")

    def nvfp4_linear_forward(self, x, out, stream=None):
        st = self.lib.nvfp4_linear_forward(self.h, x.shape[0], _ptr(x), _ptr(out), _stream(stream))
        self._check(st, "nvfp4_linear_forward")
        return out

    def nvfp4_linear_forward_raw(self, T, x_ptr, out_ptr, stream_handle):
        """Pointer-level call (for benchmarks that time the bare ABI)."""
        return self.lib.nvfp4_linear_forward(self.h, T, ctypes.c_void_p(x_ptr), ctypes.c_void_p(out_ptr),
                                             ctypes.c_void_p(stream_handle))

    def nvfp4_moe_debug_packed_blob(self, stream=None):
        import torch
        n = (self.N + 127) // 128 * 128 * self.K * 9 // 16  # rows padded to whole 128-row blocks
        out = torch.empty((n,), dtype=torch.uint8, device=f"cuda:{self.device}")
        st = self.lib.nvfp4_moe_debug_packed_blob(self.h, _ptr(out), n, _stream(stream))
        self._check(st, "nvfp4_moe_debug_packed_blob")
        return out


class Grouped(MoELayer):
    """NVFP4 experts over ragged row groups (nvfp4_grouped_create ... nvfp4_moe_destroy)."""

    def __init__(self, num_experts, out_features, in_features, max_rows, device=0, out_f32=False):
        self.lib = load_library()
        self.cfg = GroupedConfig(num_experts, out_features, in_features, max_rows, 1 if out_f32 else 0, device)
        self.out_f32 = out_f32
        self.E, self.N, self.K = num_experts, out_features, in_features
        self.device = device
        import torch
        self._int32, self._act, self._out = torch.int32, torch.bfloat16, torch.float32 if out_f32 else torch.bfloat16
        self._current_stream = torch._C._cuda_getCurrentRawStream
        h = ctypes.c_void_p()
        st = self.lib.nvfp4_grouped_create(ctypes.byref(self.cfg), ctypes.byref(h))
        if st != 0:
            raise Nvfp4MoeError(st, "nvfp4_grouped_create: " + self.lib.nvfp4_moe_status_string(st).decode())
        self.h = h

    def nvfp4_grouped_pack(self, w_q, w_s, gscale, stream=None):
        """w_q [E][N][K/2] and w_s [E][N][K/16] uint8, gscale [E] float32."""
        import torch
        for t, shape, dt in ((w_q, (self.E, self.N, self.K // 2), torch.uint8),
                             (w_s, (self.E, self.N, self.K // 16), torch.uint8), (gscale, (self.E,), torch.float32)):
            if tuple(t.shape) != shape or t.dtype != dt or t.get_device() != self.device:
                raise ValueError(f"nvfp4_grouped_pack: expected {shape} {dt} on cuda:{self.device}, "
                                 f"got {tuple(t.shape)} {t.dtype} on {t.device}")
        st = self.lib.nvfp4_grouped_pack(self.h, _ptr(w_q), _ptr(w_s), _ptr(gscale), _stream(stream, self.device))
        self._check(st, "nvfp4_grouped_pack")

    def _product(self, fn, what, x, offsets, out, wi, wo, stream):
        if offsets.dtype != self._int32 or offsets.numel() != self.E + 1 or not offsets.is_contiguous() \
                or offsets.get_device() != self.device:
            raise ValueError(f"{what}: expected contiguous int32 offsets [{self.E + 1}] on cuda:{self.device}")
        xp, ldx, R = _rows(x, wi, self._act, self.device, what)
        op, ldo, Ro = _rows(out, wo, self._out, self.device, what)
        if R != Ro:
            raise ValueError(f"{what}: the input has {R} rows, the output {Ro}")
        st = fn(self.h, R, offsets.data_ptr(), xp, ldx, op, ldo,
                stream.cuda_stream if stream is not None else self._current_stream(self.device))
        if st:
            self._check(st, what)
        return out

    def nvfp4_grouped_forward(self, x, offsets, out, stream=None):
        """out[r] = gs_e W_e x[r] for the rows of every expert e; other rows of out stay as they are."""
        return self._product(self.lib.nvfp4_grouped_forward, "nvfp4_grouped_forward", x, offsets, out, self.K, self.N,
                             stream)

    def nvfp4_grouped_backward(self, dy, offsets, dx, stream=None):
        """dx[r] = gs_e W_e^T dy[r]: the gradient of nvfp4_grouped_forward's input."""
        return self._product(self.lib.nvfp4_grouped_backward, "nvfp4_grouped_backward", dy, offsets, dx, self.N, self.K,
                             stream)

    def nvfp4_moe_debug_packed_blob(self, stream=None):
        import torch
        n = self.E * ((self.N + 127) // 128 * 128) * self.K * 9 // 16
        out = torch.empty((n,), dtype=torch.uint8, device=f"cuda:{self.device}")
        st = self.lib.nvfp4_moe_debug_packed_blob(self.h, _ptr(out), n, _stream(stream, self.device))
        self._check(st, "nvfp4_moe_debug_packed_blob")
        return out


class Int4Linear(MoELayer):
    """A dense linear with INT4 weights and group scales (nvfp4_int4_create ... nvfp4_moe_destroy)."""

    def __init__(self, out_features, in_features, group_size, max_tokens=16, act_f16=False, device=0, out_f32=False):
        self.lib = load_library()
        self.cfg = Int4Config(out_features, in_features, group_size, max_tokens, 1 if act_f16 else 0,
                              1 if out_f32 else 0, device)
        self.out_f32, self.act_f16 = out_f32, act_f16
        self.N, self.K, self.group = out_features, in_features, group_size
        self.device = device
        import torch
        self._act = torch.float16 if act_f16 else torch.bfloat16
        self._out = torch.float32 if out_f32 else self._act
        self._current_stream = torch._C._cuda_getCurrentRawStream
        h = ctypes.c_void_p()
        st = self.lib.nvfp4_int4_create(ctypes.byref(self.cfg), ctypes.byref(h))
        if st != 0:
            raise Nvfp4MoeError(st, "nvfp4_int4_create: " + self.lib.nvfp4_moe_status_string(st).decode())
        self.h = h

    def nvfp4_int4_pack(self, w_q, scale, zero=None, stream=None):
        """w_q [N][K/2] uint8, scale [N][K/group] in x's type, zero [N][K/group] uint8 or None (8 everywhere)."""
        import torch
        groups = (self.N, self.K // self.group)
        for t, shape, dt in ((w_q, (self.N, self.K // 2), torch.uint8), (scale, groups, self._act),
                             (zero, groups, torch.uint8)):
            if t is not None and (tuple(t.shape) != shape or t.dtype != dt or t.get_device() != self.device):
                raise ValueError(f"nvfp4_int4_pack: expected {shape} {dt} on cuda:{self.device}, "
                                 f"got {tuple(t.shape)} {t.dtype} on {t.device}")
        st = self.lib.nvfp4_int4_pack(self.h, _ptr(w_q), _ptr(scale), _ptr(zero), _stream(stream, self.device))
        self._check(st, "nvfp4_int4_pack")

    def nvfp4_int4_forward(self, x, out, stream=None):
        """out [T][N] = x [T][K] times the matrix, T <= max_tokens."""
        xp, ldx, T = _rows(x, self.K, self._act, self.device, "nvfp4_int4_forward")
        op, ldo, To = _rows(out, self.N, self._out, self.device, "nvfp4_int4_forward")
        if T != To:
            raise ValueError(f"nvfp4_int4_forward: x has {T} rows, out {To}")
        st = self.lib.nvfp4_int4_forward(self.h, T, xp, ldx, op, ldo,
                                         stream.cuda_stream if stream is not None else self._current_stream(self.device))
        if st:
            self._check(st, "nvfp4_int4_forward")
        return out

    def nvfp4_moe_debug_packed_blob(self, stream=None):
        import torch
        n = (self.N + 31) // 32 * 32 * (self.K // 2 + 3 * (self.K // self.group))
        out = torch.empty((n,), dtype=torch.uint8, device=f"cuda:{self.device}")
        st = self.lib.nvfp4_moe_debug_packed_blob(self.h, _ptr(out), n, _stream(stream, self.device))
        self._check(st, "nvfp4_moe_debug_packed_blob")
        return out


class _Operator(MoELayer):
    """What the handles of the operators around the products share."""

    def _open(self, name, cfg):
        import torch
        self.lib = load_library()
        self.cfg, self.device = cfg, cfg.device
        self._int8, self._int32, self._f32 = torch.int8, torch.int32, torch.float32
        self._current_stream = torch._C._cuda_getCurrentRawStream
        h = ctypes.c_void_p()
        st = getattr(self.lib, name)(ctypes.byref(cfg), ctypes.byref(h))
        if st != 0:
            raise Nvfp4MoeError(st, f"{name}: " + self.lib.nvfp4_moe_status_string(st).decode())
        self.h = h

    def _st(self, stream):
        return stream.cuda_stream if stream is not None else self._current_stream(self.device)


class Route(_Operator):
    """Routing on its own (nvfp4_route_create ... nvfp4_moe_destroy)."""

    def __init__(self, num_experts, top_k, score="softmax", renormalize=True, scale=1.0, groups=1, top_groups=None,
                 group_top=1, logits_bf16=False, device=0):
        import torch
        code = {"softmax": SCORE_SOFTMAX, "sigmoid": SCORE_SIGMOID}[score]
        self.E, self.k = num_experts, top_k
        self._logits = torch.bfloat16 if logits_bf16 else torch.float32
        self._open("nvfp4_route_create",
                   RouteConfig(num_experts, top_k, groups, groups if top_groups is None else top_groups, group_top, code,
                               1 if renormalize else 0, float(scale), 1 if logits_bf16 else 0, device))

    def _matrix(self, t, what):
        """(address, row stride, rows) of logits: rows of any stride, elements next to one another."""
        shape = t.shape
        if len(shape) != 2 or shape[1] != self.E or t.dtype != self._logits:
            raise ValueError(f"{what}: expected [tokens][{self.E}] {self._logits}, got {tuple(shape)} {t.dtype}")
        if t.get_device() != self.device:
            raise ValueError(f"{what}: expected a CUDA tensor on the handle's device, cuda:{self.device}")
        ld, one = t.stride()
        if one != 1 and self.E > 1:
            raise ValueError(f"{what}: expected contiguous rows")
        return t.data_ptr(), ld if shape[0] > 1 else self.E, shape[0]

    def nvfp4_route_forward(self, logits, ids, weights, offsets, perm, inv, bias=None, stream=None):
        """ids, weights [T][k], offsets [E + 1], perm and inv [T * k], all of the caller's; returns (ids, weights)."""
        what, dev, i32, f32 = "nvfp4_route_forward", self.device, self._int32, self._f32
        lp, ld, T = self._matrix(logits, what)
        n = (T * self.k,)
        st = self.lib.nvfp4_route_forward(
            self.h, T, lp, ld, _whole_or_none(bias, (self.E,), f32, dev, what),
            _whole(ids, (T, self.k), i32, dev, what), _whole(weights, (T, self.k), f32, dev, what),
            _whole(offsets, (self.E + 1,), i32, dev, what), _whole(perm, n, i32, dev, what), _whole(inv, n, i32, dev, what),
            self._st(stream))
        if st:
            self._check(st, what)
        return ids, weights

    def nvfp4_route_backward(self, logits, ids, dweights, dlogits, stream=None):
        """The weights' gradient to the logits, for the choice ids."""
        what, dev = "nvfp4_route_backward", self.device
        lp, ld, T = self._matrix(logits, what)
        dp, ld_dl, Td = self._matrix(dlogits, what)
        if T != Td:
            raise ValueError(f"{what}: logits of {T} tokens, their gradient of {Td}")
        st = self.lib.nvfp4_route_backward(self.h, T, lp, ld, _whole(ids, (T, self.k), self._int32, dev, what),
                                           _whole(dweights, (T, self.k), self._f32, dev, what), dp, ld_dl, self._st(stream))
        if st:
            self._check(st, what)
        return dlogits


class Norm(_Operator):
    """RMS norm with the residual's addition (nvfp4_norm_create ... nvfp4_moe_destroy)."""

    def __init__(self, hidden, eps=1e-6, act_f16=False, device=0):
        import torch
        self.H = hidden
        self._act = torch.float16 if act_f16 else torch.bfloat16
        self._open("nvfp4_norm_create", NormConfig(hidden, float(eps), 1 if act_f16 else 0, device))

    def nvfp4_norm_forward(self, x, weight, residual=None, sum=None, y=None, q=None, q_scale=None, rstd=None, stream=None):
        """sum (with a residual), y (16 bits), q with q_scale (int8 and a scale a row) and rstd are the caller's."""
        what, dev, H, act = "nvfp4_norm_forward", self.device, self.H, self._act
        xp, ldx, T = _rows(x, H, act, dev, what)
        shape, vec, f32 = (T, H), (T,), self._f32
        rp, ldr = _rows_like(residual, shape, act, dev, what)
        sp, lds = _rows_like(sum, shape, act, dev, what)
        yp, ldy = _rows_like(y, shape, act, dev, what)
        qp, ldq = _rows_like(q, shape, self._int8, dev, what)
        st = self.lib.nvfp4_norm_forward(self.h, T, xp, ldx, rp, ldr, _whole(weight, (H,), act, dev, what), sp, lds, yp, ldy,
                                         qp, ldq, _whole_or_none(q_scale, vec, f32, dev, what),
                                         _whole_or_none(rstd, vec, f32, dev, what), self._st(stream))
        if st:
            self._check(st, what)
        return y if y is not None else q

    def nvfp4_norm_backward(self, dy, sum, weight, rstd, dx, dweight=None, dsum=None, stream=None):
        """dx, the gradient of sum, x and residual alike, and dweight (float32), both the caller's."""
        what, dev, H, act = "nvfp4_norm_backward", self.device, self.H, self._act
        dp, ldd, T = _rows(dy, H, act, dev, what)
        shape = (T, H)
        sp, lds = _rows_like(sum, shape, act, dev, what)
        xp, ldx = _rows_like(dx, shape, act, dev, what)
        rp, ldr = _rows_like(dsum, shape, act, dev, what)
        st = self.lib.nvfp4_norm_backward(self.h, T, dp, ldd, sp, lds, _whole(weight, (H,), act, dev, what),
                                          _whole(rstd, (T,), self._f32, dev, what), rp, ldr, xp, ldx,
                                          _whole_or_none(dweight, (H,), self._f32, dev, what), self._st(stream))
        if st:
            self._check(st, what)
        return dx


class SwiGLU(_Operator):
    """SwiGLU with 8-bit checkpoints (nvfp4_swiglu_create ... nvfp4_moe_destroy)."""

    def __init__(self, inter, act_f16=False, device=0):
        import torch
        self.I = inter
        self.blocks = -(-inter // 128)
        self._act = torch.float16 if act_f16 else torch.bfloat16
        self._open("nvfp4_swiglu_create", SwiGLUConfig(inter, 1 if act_f16 else 0, device))

    def nvfp4_swiglu_forward(self, gate, up, out, codes=None, scales=None, stream=None):
        """out = silu(gate) up; codes [R][2][I] int8 and scales [R][2][blocks] float32 keep gate and up."""
        what, dev, I, act = "nvfp4_swiglu_forward", self.device, self.I, self._act
        gp, ldg, R = _rows(gate, I, act, dev, what)
        shape = (R, I)
        up_, ldu = _rows_like(up, shape, act, dev, what)
        op, ldo = _rows_like(out, shape, act, dev, what)
        st = self.lib.nvfp4_swiglu_forward(self.h, R, gp, ldg, up_, ldu, op, ldo,
                                           _whole_or_none(codes, (R, 2, I), self._int8, dev, what),
                                           _whole_or_none(scales, (R, 2, self.blocks), self._f32, dev, what),
                                           self._st(stream))
        if st:
            self._check(st, what)
        return out

    def nvfp4_swiglu_backward(self, codes, scales, dh, dgate, dup, stream=None):
        """dgate and dup from the forward's codes and scales."""
        what, dev, I, act = "nvfp4_swiglu_backward", self.device, self.I, self._act
        dp, ldd, R = _rows(dh, I, act, dev, what)
        shape = (R, I)
        gp, ldg = _rows_like(dgate, shape, act, dev, what)
        up_, ldu = _rows_like(dup, shape, act, dev, what)
        st = self.lib.nvfp4_swiglu_backward(self.h, R, _whole(codes, (R, 2, I), self._int8, dev, what),
                                            _whole(scales, (R, 2, self.blocks), self._f32, dev, what), dp, ldd, gp, ldg,
                                            up_, ldu, self._st(stream))
        if st:
            self._check(st, what)
        return dgate, dup


class Int8Linear(_Operator):
    """A dense linear with 8-bit integers on both sides (nvfp4_int8_create ... nvfp4_moe_destroy)."""

    def __init__(self, out_features, in_features, max_tokens, out="bf16", device=0):
        import torch
        code = {"bf16": 0, "f32": 1, "f16": 2}[out]
        self._out = (torch.bfloat16, torch.float32, torch.float16)[code]
        self._x_types = {torch.bfloat16: 0, torch.float16: 1}
        self.N, self.K = out_features, in_features
        self._open("nvfp4_int8_create", Int8Config(out_features, in_features, max_tokens, code, device))

    def nvfp4_int8_pack(self, w, w_scale, bias=None, stream=None):
        """w [N][K] int8, w_scale [N] float32, bias [N] float32 or None."""
        what, dev = "nvfp4_int8_pack", self.device
        st = self.lib.nvfp4_int8_pack(self.h, _whole(w, (self.N, self.K), self._int8, dev, what),
                                      _whole(w_scale, (self.N,), self._f32, dev, what),
                                      _whole_or_none(bias, (self.N,), self._f32, dev, what), self._st(stream))
        self._check(st, what)

    def nvfp4_int8_quantize(self, x, q, q_scale, stream=None):
        """q [T][K] int8 and q_scale [T] float32 of x [T][K], BF16 or FP16."""
        what, dev = "nvfp4_int8_quantize", self.device
        code = self._x_types.get(x.dtype)
        if code is None:
            raise ValueError(f"{what}: expected a bfloat16 or float16 x, got {x.dtype}")
        xp, ldx, T = _rows(x, self.K, x.dtype, dev, what)
        qp, ldq = _rows_like(q, (T, self.K), self._int8, dev, what)
        st = self.lib.nvfp4_int8_quantize(self.h, T, xp, code, ldx, qp, ldq, _whole(q_scale, (T,), self._f32, dev, what),
                                          self._st(stream))
        if st:
            self._check(st, what)
        return q, q_scale

    def nvfp4_int8_forward(self, x, x_scale, out, stream=None):
        """out [T][N] = x_scale w_scale (x [T][K] times the matrix) + bias, T <= max_tokens."""
        what, dev = "nvfp4_int8_forward", self.device
        xp, ldx, T = _rows(x, self.K, self._int8, dev, what)
        if T <= 1:
            ldx = -(-self.K // 16) * 16
        op, ldo = _rows_like(out, (T, self.N), self._out, dev, what)
        st = self.lib.nvfp4_int8_forward(self.h, T, xp, ldx, _whole(x_scale, (T,), self._f32, dev, what), op, ldo,
                                         self._st(stream))
        if st:
            self._check(st, what)
        return out

    def nvfp4_moe_debug_packed_blob(self, stream=None):
        import torch
        n = -(-self.N // 128) * 128 * -(-self.K // 128) * 128
        out = torch.empty((n,), dtype=torch.uint8, device=f"cuda:{self.device}")
        st = self.lib.nvfp4_moe_debug_packed_blob(self.h, _ptr(out), n, _stream(stream, self.device))
        self._check(st, "nvfp4_moe_debug_packed_blob")
        return out


def nvfp4_moe_forward_decode_static(packed_experts, gscale, num_experts, hidden, inter, logits, top_k, x, out,
                                    logits_bf16=False, stream=None):
    """The allocation-free decode forward: every argument is caller memory."""
    lib = load_library()
    return lib.nvfp4_moe_forward_decode_static(_ptr(packed_experts), _ptr(gscale), num_experts, hidden, inter,
                                               _ptr(logits), 1 if logits_bf16 else 0, x.shape[0], top_k,
                                               _ptr(x), _ptr(out), _stream(stream))


def nvfp4_moe_static_get_status():
    """(status, nan_logits) of the allocation-free path on the current device
    (synchronous; reads and clears the status word)."""
    lib = load_library()
    n = ctypes.c_uint32(0)
    st = lib.nvfp4_moe_static_get_status(ctypes.byref(n))
    return st, int(n.value)


def nvfp4_moe_static_debug_set_fault(fault):
    return load_library().nvfp4_moe_static_debug_set_fault(int(fault))


def upload_layer(layer: MoELayer, weights, device="cuda:0"):
    """Copy an ExpertWeights-like set of numpy arrays to the device and pack it."""
    import torch
    t = lambda a: torch.from_numpy(a).to(device)
    layer.nvfp4_moe_pack(t(weights.w13_q), t(weights.w13_s), t(weights.w2_q), t(weights.w2_s), t(weights.gscale))
    torch.cuda.synchronize()
