"""Microscaled rows: the 8- and 4-bit form in which a projection after the
mixture takes its input.

    q = mx.add_rms_norm(prefix, delta, weight)   # residual + RMSNorm -> codes and scales
    q = mx.quantize(rows, "mxfp4")               # bf16 rows -> codes and scales
    y = mx.matmul(q, w)                          # [rows, n] = q @ w^T, bf16
    x = mx.dequantize(q)                         # the bf16 values that q stands for

``MxTensor`` holds a matrix in one of the formats "mxfp8", "mxfp4" and
"nvfp4"; ``include/attn_res.h`` defines them, their roundings and the layout of
codes and scales.  Every step runs in the kernels of ``libattn_res.so`` (the
``attn_res_mx_*`` entry points); there is no CPU or PyTorch fallback.  The
calls are compiled (``csrc/mx_binding.cpp``, marshalling only) and loaded at
their first use; if the library or the binding is not built, that raises.

Each call takes ``stream``: the stream that it runs on, as torch.cuda.stream
would set it (outputs are allocated there too); the current one by default.
Tensors on another device than the current one run there.  ``pdl`` is
programmatic dependent launch (see ATTN_RES_FLAG_PDL and the notes on the
microscaled calls).  Arguments that cannot be marshalled raise ValueError (or
TypeError where another type was given for a tensor, a matrix or a number),
those that the library refuses AttnResError.
"""
from __future__ import annotations

import importlib.machinery
import importlib.util
import os
import threading

from . import _build, lib

GROUP = {"mxfp8": 32, "mxfp4": 32, "nvfp4": 16}
# Forms of the product (matmul's kernel=; 0: automatic), see attn_res_mx_matmul.
KERNEL_NARROW, KERNEL_WIDE, KERNEL_WIDER = 1, 2, 3
_CALLS = ("MxTensor", "quantize", "dequantize", "add_rms_norm", "matmul")
_loading = threading.Lock()


def scales_shape(format: str, rows: int, cols: int) -> tuple:
    """Shape of the scale tensor: entry [i, j, r, p, g] is the scale of row
    128 i + 32 p + r and group 4 j + g; zero codes past the last of either."""
    return ((rows + 127) // 128, (cols // GROUP[format] + 3) // 4, 32, 4, 4)


def _load():
    import torch  # noqa: F401  (the binding's libraries)

    lib()
    if not os.path.exists(_build.BINDING):
        raise RuntimeError(
            f"{_build.BINDING} is missing: build it with "
            "attention_residual_fusion_gb300._build.build() (or __graft_entry__.build())")
    loader = importlib.machinery.ExtensionFileLoader("_mx", _build.BINDING)
    spec = importlib.util.spec_from_file_location("_mx", _build.BINDING, loader=loader)
    module = importlib.util.module_from_spec(spec)
    loader.exec_module(module)
    globals().update({name: getattr(module, name) for name in _CALLS})


def __getattr__(name: str):
    if name not in _CALLS:
        raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
    with _loading:  # a second thread's load would find the module half made
        if name not in globals():
            _load()
    return globals()[name]
