"""Microscaled rows: the 8- and 4-bit form in which a projection after the
mixture takes its input.

    q = mx.add_rms_norm(prefix, delta, weight)   # residual + RMSNorm -> codes and scales
    q = mx.quantize(rows, "mxfp4")               # bf16 rows -> codes and scales
    y = mx.matmul(q, w)                          # [rows, n] = q @ w^T, bf16
    x = mx.dequantize(q)                         # the bf16 values that q stands for

Thin binding of the ``attn_res_mx_*`` entry points of ``include/attn_res.h``,
which defines the formats ("mxfp8", "mxfp4", "nvfp4"), their roundings and the
layout of codes and scales.  Every step runs in the kernels of
``libattn_res.so``; there is no CPU or PyTorch fallback.

``stream``: the stream that the call runs on, as torch.cuda.stream would set
it (outputs are allocated there too); the current one by default.  Tensors on
another device than the current one run there.  ``pdl``: programmatic
dependent launch (see ATTN_RES_FLAG_PDL and the microscaled calls' notes).
"""
from __future__ import annotations

import ctypes
import struct

import torch
from torch._C import _cuda_getCurrentRawStream, _cuda_getDevice

from . import FLAG_PDL, AttnResError, lib, status_string

FORMATS = {"mxfp8": 1, "mxfp4": 2, "nvfp4": 3}
GROUP = {"mxfp8": 32, "mxfp4": 32, "nvfp4": 16}
_DATA = {"mxfp8": torch.float8_e4m3fn, "mxfp4": torch.uint8, "nvfp4": torch.uint8}
_SCALES = {"mxfp8": torch.float8_e8m0fnu, "mxfp4": torch.float8_e8m0fnu,
           "nvfp4": torch.float8_e4m3fn}
_BF16 = torch.bfloat16

# attn_res_mx_t as the bytes of its members: a call then passes one pointer
# (building a ctypes.Structure takes longer than the rest of a small call).
_pack = struct.Struct("ixxxxqqqqqq").pack
_calls: dict = {}


def _call(name: str):
    """The entry point `attn_res_mx_<name>`, its matrices passed as bytes."""
    f = _calls.get(name)
    if f is None:
        vp, i64, u32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint32
        f = lib()["attn_res_mx_" + name]  # a function object of its own
        f.restype = ctypes.c_int
        f.argtypes = {"quantize": [vp, i64, vp, u32, vp], "dequantize": [vp, vp, i64, u32, vp],
                      "norm": [vp, i64, vp, i64, vp, ctypes.c_float, vp, i64, vp, u32, vp],
                      "matmul": [vp, vp, vp, i64, u32, vp]}[name]
        _calls[name] = f
    return f


def _raise(st: int):
    raise AttnResError(st, status_string(st))


def _elsewhere(call, device, stream, *args, **kw):
    """`call` with another device or stream made current."""
    if stream is None:
        with torch.cuda.device(device):
            return call(*args, **kw)
    if stream.device != device:
        raise ValueError("stream must belong to the tensors' device")
    with torch.cuda.stream(stream):
        return call(*args, **kw)


def scales_shape(format: str, rows: int, cols: int) -> tuple:
    """Shape of the scale tensor: entry [i, j, r, p, g] is the scale of row
    128 i + 32 p + r and group 4 j + g; zero codes past the last of either."""
    return ((rows + 127) // 128, (cols // GROUP[format] + 3) // 4, 32, 4, 4)


class MxTensor:
    """A matrix [rows, cols] in a microscaled format.

    data: [rows, cols] float8_e4m3fn ("mxfp8") or [rows, cols // 2] uint8 (two
    e2m1 codes a byte, the even column low), unit inner stride; scales:
    ``scales_shape``, contiguous, float8_e8m0fnu or (nvfp4) float8_e4m3fn;
    global_scale: one fp32 on the device, nvfp4 only, or None.
    """
    __slots__ = ("data", "scales", "format", "global_scale", "shape", "device", "_c")

    def __init__(self, data, scales, format: str, global_scale=None):
        if format not in FORMATS:
            raise ValueError(f"format must be one of {', '.join(FORMATS)}")
        if data.dtype is not _DATA[format] or data.dim() != 2 or not data.is_cuda or \
                (data.stride(1) != 1 and data.shape[1] > 1):
            raise ValueError(f"data must be a CUDA {_DATA[format]} matrix with unit inner stride")
        rows, cols = data.shape
        if format != "mxfp8":
            cols *= 2
        device = data.device
        if scales.dtype is not _SCALES[format] or scales.device != device or \
                scales.shape != scales_shape(format, rows, cols) or not scales.is_contiguous():
            raise ValueError(f"scales must be a contiguous {_SCALES[format]} tensor of shape "
                             f"{scales_shape(format, rows, cols)} beside data")
        g = global_scale
        if g is not None and (format != "nvfp4" or g.dtype is not torch.float32 or
                              g.numel() != 1 or g.device != device):
            raise ValueError("global_scale must be one float32 beside data (nvfp4 only)")
        self._set(data, scales, format, g, rows, cols, device)

    def _set(self, data, scales, format, g, rows, cols, device):
        self.data, self.scales, self.format, self.global_scale = data, scales, format, g
        self.shape, self.device = (rows, cols), device
        # the stride of a single row says nothing: it may be anything
        row = data.stride(0) if rows > 1 else (data.shape[1] + 15) // 16 * 16
        self._c = _pack(FORMATS[format], rows, cols, data.data_ptr(), row, scales.data_ptr(),
                        0 if g is None else g.data_ptr())

    @classmethod
    def empty(cls, rows: int, cols: int, format: str, global_scale=None, device="cuda"):
        """Uninitialised codes and scales for [rows, cols] (cols a multiple of 32)."""
        if format not in FORMATS:
            raise ValueError(f"format must be one of {', '.join(FORMATS)}")
        if rows < 0 or cols <= 0 or cols % 32:
            raise ValueError("rows must be >= 0 and cols a positive multiple of 32")
        data = torch.empty((rows, cols if format == "mxfp8" else cols // 2), dtype=_DATA[format],
                           device=device)
        scales = torch.empty(scales_shape(format, rows, cols), dtype=_SCALES[format], device=device)
        return cls(data, scales, format, global_scale)


def _out(rows: int, cols: int, format: str, g, device) -> MxTensor:
    """MxTensor.empty for a call's own result: what the tensors are is known."""
    if format not in FORMATS:
        raise ValueError(f"format must be one of {', '.join(FORMATS)}")
    if cols <= 0 or cols % 32:
        raise ValueError("the rows' width must be a positive multiple of 32")
    if g is not None and (format != "nvfp4" or g.dtype is not torch.float32 or g.numel() != 1 or
                          g.device != device):
        raise ValueError("global_scale must be one float32 beside the rows (nvfp4 only)")
    q = MxTensor.__new__(MxTensor)
    q._set(torch.empty((rows, cols if format == "mxfp8" else cols // 2), dtype=_DATA[format],
                       device=device),
           torch.empty(scales_shape(format, rows, cols), dtype=_SCALES[format], device=device),
           format, g, rows, cols, device)
    return q


def _check_out(out: MxTensor, format: str, g, shape, device) -> None:
    if out.format != format or (g is not None and g is not out.global_scale):
        raise ValueError("out has another format or global_scale")
    if out.shape != tuple(shape) or out.device != device:
        raise ValueError(f"out must be a {tuple(shape)} MxTensor on {device}")


def _check_rows(name: str, t, shape, device) -> None:
    """bf16 rows with unit inner stride (and the given shape and device, if any)."""
    if t.dtype is not _BF16 or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA bfloat16 tensor")
    if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1) or (shape is not None and t.shape != shape):
        raise ValueError(f"{name} must be a {tuple(shape) if shape else '2-D'} matrix with unit inner stride")
    if device is not None and t.device != device:
        raise ValueError("all tensors of a call must be on one device")


def _row(t) -> int:
    # as for the codes: a single row's stride says nothing
    return t.stride(0) if t.shape[0] > 1 else (t.shape[1] + 7) // 8 * 8


def quantize(x, format: str = "mxfp4", global_scale=None, out: MxTensor | None = None, *,
             pdl: bool = False, stream=None) -> MxTensor:
    """bf16 rows [rows, cols] to ``format`` (attn_res_mx_quantize).  cols is a
    multiple of 32; ``global_scale`` (nvfp4) is the tensor's scale, 1 if None.
    Returns ``out`` (allocated if not given; its own global_scale then holds)."""
    _check_rows("x", x, None, None)
    device = x.device
    if stream is not None or device.index != _cuda_getDevice():
        return _elsewhere(quantize, device, stream, x, format, global_scale, out, pdl=pdl)
    if out is None:
        rows, cols = x.shape
        out = _out(rows, cols, format, global_scale, device)
    else:
        _check_out(out, format, global_scale, x.shape, device)
    st = _call("quantize")(x.data_ptr(), _row(x), out._c, FLAG_PDL if pdl else 0,
                           _cuda_getCurrentRawStream(device.index))
    if st:
        _raise(st)
    return out


def dequantize(q: MxTensor, out=None, *, pdl: bool = False, stream=None):
    """The bf16 values [rows, cols] that ``q`` stands for (attn_res_mx_dequantize)."""
    device = q.device
    if stream is not None or device.index != _cuda_getDevice():
        return _elsewhere(dequantize, device, stream, q, out, pdl=pdl)
    if out is None:
        out = torch.empty(q.shape, dtype=_BF16, device=device)
    else:
        _check_rows("out", out, q.shape, device)
    st = _call("dequantize")(q._c, out.data_ptr(), _row(out), FLAG_PDL if pdl else 0,
                             _cuda_getCurrentRawStream(device.index))
    if st:
        _raise(st)
    return out


def add_rms_norm(prefix, delta, weight, eps: float = 1e-6, format: str = "mxfp8",
                 global_scale=None, out: MxTensor | None = None, norm_out=None, *,
                 pdl: bool = False, stream=None) -> MxTensor:
    """Residual addition and RMSNorm of token rows, quantised (attn_res_mx_norm).

    c = bf16(prefix + delta) (prefix if ``delta`` is None; prefix [T, H] is
    updated in place otherwise), y = c * weight / sqrt(mean(c^2) + eps); the
    result is y in ``format``, from fp32.  ``norm_out`` [T, H] receives y in
    bf16 as well, if given.  H is a multiple of 32, at most 65536.
    """
    _check_rows("prefix", prefix, None, None)
    device, shape = prefix.device, prefix.shape
    if stream is not None or device.index != _cuda_getDevice():
        return _elsewhere(add_rms_norm, device, stream, prefix, delta, weight, eps, format,
                          global_scale, out, norm_out, pdl=pdl)
    rows, cols = shape
    d_ptr = d_row = n_ptr = n_row = 0
    if delta is not None:
        _check_rows("delta", delta, shape, device)
        d_ptr, d_row = delta.data_ptr(), _row(delta)
    if norm_out is not None:
        _check_rows("norm_out", norm_out, shape, device)
        n_ptr, n_row = norm_out.data_ptr(), _row(norm_out)
    if weight.dtype is not _BF16 or weight.device != device or weight.shape != (cols,) or \
            not weight.is_contiguous():
        raise ValueError("weight must be a contiguous bfloat16 [H] tensor beside prefix")
    if out is None:
        out = _out(rows, cols, format, global_scale, device)
    else:
        _check_out(out, format, global_scale, shape, device)
    st = _call("norm")(prefix.data_ptr(), _row(prefix), d_ptr, d_row, weight.data_ptr(), eps,
                       n_ptr, n_row, out._c, FLAG_PDL if pdl else 0,
                       _cuda_getCurrentRawStream(device.index))
    if st:
        _raise(st)
    return out


def matmul(a: MxTensor, w: MxTensor, out=None, *, pdl: bool = False, stream=None):
    """``a`` [m, k] times the transpose of ``w`` [n, k], of one format: bf16
    [m, n], fp32 sums (attn_res_mx_matmul)."""
    device = a.device
    m, k = a.shape
    n, wk = w.shape
    if a.format != w.format or k != wk:
        raise ValueError("a and w must have one format and one width")
    if w.device != device:
        raise ValueError("all tensors of a call must be on one device")
    if stream is not None or device.index != _cuda_getDevice():
        return _elsewhere(matmul, device, stream, a, w, out, pdl=pdl)
    if out is None:
        # rows start on 16-byte boundaries, whatever n
        row = (n + 7) // 8 * 8
        out = torch.empty((m, row), dtype=_BF16, device=device)
        if row != n:
            out = out[:, :n]
    else:
        _check_rows("out", out, (m, n), device)
        row = _row(out)
    st = _call("matmul")(a._c, w._c, out.data_ptr(), row, FLAG_PDL if pdl else 0,
                         _cuda_getCurrentRawStream(device.index))
    if st:
        _raise(st)
    return out
