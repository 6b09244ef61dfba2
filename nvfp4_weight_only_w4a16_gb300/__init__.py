"""Routed-expert MoE layer with weight-only NVFP4 (W4A16) experts on GB300,
the dense W4A16 NVFP4 linear that shares its kernels, and 4-bit weight-only
products on their own: NVFP4 experts over ragged row groups (with the gradient
of their input) and a dense INT4 linear with group scales; and what a block has
around them: routing with its gradient, SwiGLU with 8-bit checkpoints, the RMS
norm with the residual's addition, an INT8 linear.

The computation lives in the CUDA library libnvfp4moe.so (C ABI declared in
include/nvfp4_moe.h); this package holds its sources (csrc/), the in-tree
build step (build.py) and a ctypes binding (binding.py).
"""
from .build import build, LIB  # noqa: F401
from . import binding  # noqa: F401
from .binding import (  # noqa: F401
    MoELayer, Linear, Grouped, Int4Linear, Int8Linear, Route, Norm, SwiGLU, Nvfp4MoeError, load_library, header_functions, upload_layer,
    PATH_AUTO, PATH_DECODE, PATH_PREFILL, STATUS, STATUS_CODE,
)
