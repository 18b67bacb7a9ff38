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
"""
from __future__ import annotations

import ctypes

import torch

from . import FLAG_PDL, AttnResError, Mx, check_bf16_cuda, lib, status_string

FORMATS = {"mxfp8": 1, "mxfp4": 2, "nvfp4": 3}
GROUP = {"mxfp8": 32, "mxfp4": 32, "nvfp4": 16}
_DATA = {"mxfp8": torch.float8_e4m3fn, "mxfp4": torch.uint8, "nvfp4": torch.uint8}
_SCALES = {"mxfp8": torch.float8_e8m0fnu, "mxfp4": torch.float8_e8m0fnu,
           "nvfp4": torch.float8_e4m3fn}


def scales_shape(format: str, rows: int, cols: int) -> tuple:
    """Shape of the scale tensor: entry [i, j, r, p, g] is the scale of row
    128 i + 32 p + r and group 4 j + g; zero codes past the last of either."""
    return (-(-rows // 128), -(-(cols // GROUP[format]) // 4), 32, 4, 4)


class MxTensor:
    """A matrix [rows, cols] in a microscaled format.

    data: [rows, cols] float8_e4m3fn ("mxfp8") or [rows, cols // 2] uint8 (two
    e2m1 codes a byte, the even column low), unit inner stride; scales:
    ``scales_shape``, contiguous, float8_e8m0fnu or (nvfp4) float8_e4m3fn;
    global_scale: one fp32 on the device, nvfp4 only, or None.
    """
    __slots__ = ("data", "scales", "format", "global_scale", "_c")

    def __init__(self, data, scales, format: str, global_scale=None):
        if format not in FORMATS:
            raise ValueError(f"format must be one of {', '.join(FORMATS)}")
        if data.dim() != 2 or data.dtype != _DATA[format] or not data.is_cuda or \
                (data.shape[1] > 1 and data.stride(1) != 1):
            raise ValueError(f"data must be a CUDA {_DATA[format]} matrix with unit inner stride")
        rows, cols = data.shape
        if format != "mxfp8":
            cols *= 2
        if scales.dtype != _SCALES[format] or scales.device != data.device or \
                not scales.is_contiguous() or tuple(scales.shape) != scales_shape(format, rows, cols):
            raise ValueError(f"scales must be a contiguous {_SCALES[format]} tensor of shape "
                             f"{scales_shape(format, rows, cols)} beside data")
        g = global_scale
        if g is not None and (format != "nvfp4" or g.dtype != torch.float32 or g.numel() != 1 or
                              g.device != data.device):
            raise ValueError("global_scale must be one float32 beside data (nvfp4 only)")
        self.data, self.scales, self.format, self.global_scale = data, scales, format, g
        self._c = Mx(FORMATS[format], rows, cols, data.data_ptr(), _row(data), scales.data_ptr(),
                     None if g is None else g.data_ptr())

    @property
    def shape(self) -> tuple:
        return (self._c.rows, self._c.cols)

    @property
    def device(self):
        return self.data.device

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


def _row(t) -> int:
    # the stride of a single row says nothing: a tensor of one row may have any
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), -(-t.shape[1] // 16) * 16)


def _rows(name: str, t, shape=None):
    if t.dim() != 2 or t.stride(1) != 1 or (shape is not None and tuple(t.shape) != tuple(shape)):
        raise ValueError(f"{name} must be a {'x'.join(map(str, shape)) if shape else '2-D'} matrix "
                         "with unit inner stride")
    return t


class _On:
    """The device and the stream of a call: makes both current while outputs
    are allocated and the kernel is launched."""
    __slots__ = ("device", "stream", "guard", "handle")

    def __init__(self, device, stream, *tensors):
        for t in tensors:
            if t is not None and t.device != device:
                raise ValueError("all tensors of a call must be on one device")
        self.device, self.stream = device, stream

    def __enter__(self):
        self.guard = None
        if self.stream is not None:
            if self.stream.device != self.device:
                raise ValueError("stream must belong to the tensors' device")
            self.guard = torch.cuda.stream(self.stream)
            self.guard.__enter__()
            self.handle = self.stream.cuda_stream
        else:
            if self.device.index != torch.cuda.current_device():
                self.guard = torch.cuda.device(self.device)
                self.guard.__enter__()
            self.handle = torch.cuda.current_stream(self.device).cuda_stream
        return self

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _check(st: int) -> None:
    if st != 0:
        raise AttnResError(st, status_string(st))


def quantize(x, format: str = "mxfp4", global_scale=None, out: MxTensor | None = None, *,
             pdl: bool = False, stream=None) -> MxTensor:
    """bf16 rows [rows, cols] to ``format`` (attn_res_mx_quantize).  cols is a
    multiple of 32; ``global_scale`` (nvfp4) is the tensor's scale, 1 if None.
    Returns ``out`` (allocated if not given; its own global_scale then holds)."""
    check_bf16_cuda(x=x)
    _rows("x", x, None if out is None else out.shape)
    if out is not None and (out.format != format or
                            (global_scale is not None and global_scale is not out.global_scale)):
        raise ValueError("out has another format or global_scale")
    with _On(x.device, stream, global_scale, None if out is None else out.data) as on:
        if out is None:
            out = MxTensor.empty(x.shape[0], x.shape[1], format, global_scale, x.device)
        _check(lib().attn_res_mx_quantize(x.data_ptr(), x.stride(0), out._c, FLAG_PDL if pdl else 0,
                                          on.handle))
    return out


def dequantize(q: MxTensor, out=None, *, pdl: bool = False, stream=None):
    """The bf16 values [rows, cols] that ``q`` stands for (attn_res_mx_dequantize)."""
    if out is not None:
        check_bf16_cuda(out=out)
        _rows("out", out, q.shape)
    with _On(q.device, stream, out) as on:
        if out is None:
            out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
        _check(lib().attn_res_mx_dequantize(q._c, out.data_ptr(), out.stride(0),
                                            FLAG_PDL if pdl else 0, on.handle))
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
    check_bf16_cuda(prefix=prefix, delta=delta, weight=weight, norm_out=norm_out)
    shape = prefix.shape if out is None else out.shape
    _rows("prefix", prefix, shape)
    if delta is not None:
        _rows("delta", delta, shape)
    if norm_out is not None:
        _rows("norm_out", norm_out, shape)
    if weight.dim() != 1 or weight.shape[0] != shape[1] or weight.stride(0) != 1:
        raise ValueError("weight must be a contiguous [H] tensor")
    if out is not None and (out.format != format or
                            (global_scale is not None and global_scale is not out.global_scale)):
        raise ValueError("out has another format or global_scale")
    with _On(prefix.device, stream, delta, weight, norm_out, global_scale,
             None if out is None else out.data) as on:
        if out is None:
            out = MxTensor.empty(shape[0], shape[1], format, global_scale, prefix.device)
        _check(lib().attn_res_mx_norm(
            prefix.data_ptr(), prefix.stride(0), None if delta is None else delta.data_ptr(),
            0 if delta is None else delta.stride(0), weight.data_ptr(), eps,
            None if norm_out is None else norm_out.data_ptr(),
            0 if norm_out is None else norm_out.stride(0), out._c, FLAG_PDL if pdl else 0, on.handle))
    return out


def matmul(a: MxTensor, w: MxTensor, out=None, *, pdl: bool = False, stream=None):
    """``a`` [m, k] times the transpose of ``w`` [n, k], of one format: bf16
    [m, n], fp32 sums (attn_res_mx_matmul)."""
    if a.format != w.format or a.shape[1] != w.shape[1]:
        raise ValueError("a and w must have one format and one width")
    m, n = a.shape[0], w.shape[0]
    if out is not None:
        check_bf16_cuda(out=out)
        _rows("out", out, (m, n))
    with _On(a.device, stream, w.data, out) as on:
        if out is None:
            # rows start on 16-byte boundaries, whatever n
            out = torch.empty((m, -(-n // 8) * 8), dtype=torch.bfloat16, device=a.device)[:, :n]
        _check(lib().attn_res_mx_matmul(a._c, w._c, out.data_ptr(), out.stride(0),
                                        FLAG_PDL if pdl else 0, on.handle))
    return out
