"""The feed-forward block in 8 bits: e4m3 codes with fp32 scales for blocks of
128, products, the gated block and its backward pass.

    x, xt = f8.quantize(rows, transposed=True)   # bf16 rows -> codes and scales, and x^T's
    w = f8.quantize(weights, 128)                # a scale for each 128 x 128
    h, g, u = f8.gated(x, gate, up, save=True)   # act(x gate^T) * (x up^T); g, u kept in 8 bits
    y = f8.matmul(h, down)                       # [T, n] = h @ down^T, bf16

and backwards, with the transposed weights from ``quantize(..., transposed=True)``:

    dyq, dyt = f8.quantize(dy, transposed=True)
    dh = f8.matmul(dyq, down_t)
    dg, du, dgt, dut, ht = f8.gated_backward(dh, g, u)
    dx = f8.matmul(dg, gate_t, plus=(du, up_t))
    d_gate = f8.matmul(dgt, xt, dtype=torch.float32)     # also add=True, into out
    d_up = f8.matmul(dut, xt, dtype=torch.float32)
    d_down = f8.matmul(dyt, ht, dtype=torch.float32)

``F8Tensor`` holds a matrix; ``include/attn_res.h`` defines the format, its
roundings and layouts.  Every step runs in the kernels of ``libattn_res.so`` (the
``attn_res_f8_*`` entry points); there is no CPU or PyTorch fallback.  The calls
are compiled (``csrc/f8_binding.cpp``, marshalling only) and loaded at their first
use; if the library or the binding is not built, that raises.

``stream``, ``pdl``, devices and errors are as in ``mx``.
"""
from __future__ import annotations

import threading

from . import _build, load_binding

BLOCK = 128
# Forms of the products (kernel=; 0: automatic), see attn_res_f8_matmul.
KERNEL_NARROW, KERNEL_WIDE = 1, 2
_CALLS = ("F8Tensor", "quantize", "dequantize", "matmul", "gated", "gated_backward")
_loading = threading.Lock()


def scales_shape(rows: int, cols: int, block: int = 1) -> tuple:
    """Shape of the scale tensor: entry [b, r] is the scale of row r and columns
    128 b .. (block 1), entry [i, b] that of rows 128 i .. and columns 128 b ..
    (block 128)."""
    b = (cols + BLOCK - 1) // BLOCK
    return (b, rows) if block == 1 else ((rows + BLOCK - 1) // BLOCK, b)


def __getattr__(name: str):
    if name not in _CALLS:
        raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
    with _loading:  # a second thread's load would find the module half made
        if name not in globals():
            globals().update(load_binding("_f8", _build.F8_BINDING, _CALLS))
    return globals()[name]
