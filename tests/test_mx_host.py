"""The microscaled entry points on the host: the restated formats against
hand-worked values, the scale layout, and every refusal (validation precedes
the first CUDA call, so no GPU is needed)."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import attention_residual_fusion_gb300 as ar
from attention_residual_fusion_gb300 import _build, mx
from tests import mx_restatement as R

BASE, GAP = 1 << 40, 1 << 34


def addr(i, off=0):
    return BASE + i * GAP + off


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return ar.lib()


# ---- the formats --------------------------------------------------------------


def test_e4m3_table_is_the_type():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(R.e4m3(np.arange(256)), t)


def test_e8m0_table_is_the_type():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e8m0fnu).double().numpy()
    np.testing.assert_array_equal(R.e8m0(np.arange(256)), t)


@pytest.mark.parametrize("v,code", [(0, 0), (0.25, 0), (0.26, 1), (0.75, 2), (1.25, 2), (1.75, 4),
                                    (2.5, 4), (2.51, 5), (3.5, 6), (5, 6), (5.01, 7), (6, 7), (9, 7)])
def test_e2m1_rounding(v, code):
    assert R.nearest_code(np.array([float(v)]), R.E2M1)[0] == code


@pytest.mark.parametrize("fmt,amax,code", [
    ("mxfp8", 448.0, 127), ("mxfp8", 449.0, 128), ("mxfp8", 896.0, 128), ("mxfp8", 1.0, 119),
    ("mxfp8", 0.0, 0), ("mxfp8", 2.0 ** -133, 0), ("mxfp8", 2.0 ** 127 * 1.99, 247),
    ("mxfp4", 6.0, 127), ("mxfp4", 6.03125, 128), ("mxfp4", 4.0, 127), ("mxfp4", 3.0, 126),
    ("mxfp4", 2.0 ** 127 * 1.99, 253), ("mxfp4", np.inf, 255), ("mxfp8", np.nan, 255),
    ("nvfp4", 6.0, 0x38), ("nvfp4", 6 * 448.0, 126), ("nvfp4", 1e6, 126), ("nvfp4", 0.0, 0),
    ("nvfp4", 6 * 2.0 ** -9, 1), ("nvfp4", 6 * 2.0 ** -10, 0), ("nvfp4", np.inf, 127)])
def test_scale_codes(fmt, amax, code):
    assert R.scale_codes(np.array([[amax]]), fmt)[0, 0] == code


def test_tile_order_is_the_tensor_shape():
    """The byte formula and the five-dimensional view of the binding agree."""
    rng = np.random.default_rng(0)
    codes = rng.integers(1, 250, (300, 9)).astype(np.uint8)
    flat = R.tile(codes)
    t = flat.reshape(mx.scales_shape("mxfp8", 300, 9 * 32))
    for r, j in [(0, 0), (31, 3), (32, 4), (127, 8), (128, 1), (299, 8), (200, 5)]:
        assert t[r // 128, j // 4, r % 32, r // 32 % 4, j % 4] == codes[r, j]
    np.testing.assert_array_equal(R.untile(flat, 300, 9), codes)
    assert (flat != 0).sum() == codes.size


def test_scale_bytes(lib):
    f = lib.attn_res_mx_scale_bytes
    assert f(1, 1, 32) == 512 and f(1, 128, 128) == 512 and f(1, 129, 160) == 2 * 2 * 512
    assert f(2, 8192, 7168) == 8192 * 7168 // 32 and f(3, 8192, 7168) == 8192 * 7168 // 16
    assert f(3, 0, 64) == 0
    for bad in [(0, 1, 32), (4, 1, 32), (1, -1, 32), (1, 1, 0), (1, 1, 48), (2, 1, -32),
                (1, 1 << 31, 32), (1, 1, 1 << 31)]:
        assert f(*bad) == -1


# ---- refusals -------------------------------------------------------------------


def matrix(i, fmt=2, rows=40, cols=256, **change):
    kw = dict(format=fmt, rows=rows, cols=cols, data=addr(i), row_bytes=cols if fmt == 1 else cols // 2,
              scales=addr(i, 1 << 32), tensor_scale=0)
    kw.update(change)
    return ar.Mx(*(kw[n] for n, _ in ar.Mx._fields_))


def quantize(q=None, x=addr(0), x_row=256, flags=0):
    return ar.lib().attn_res_mx_quantize(x, x_row, matrix(1) if q is None else q, flags, None)


def dequantize(q=None, x=addr(0), x_row=256, flags=0):
    return ar.lib().attn_res_mx_dequantize(matrix(1) if q is None else q, x, x_row, flags, None)


def norm(q=None, prefix=addr(0), prefix_row=256, delta=addr(2), delta_row=256, weight=addr(3), eps=1e-6,
         norm_out=addr(4), norm_row=256, flags=0):
    return ar.lib().attn_res_mx_norm(prefix, prefix_row, delta, delta_row, weight, eps, norm_out, norm_row,
                                     matrix(1) if q is None else q, flags, None)


def matmul(a=None, w=None, out=addr(0), out_row=72, flags=0):
    return ar.lib().attn_res_mx_matmul(matrix(1) if a is None else a, matrix(2, rows=70) if w is None else w,
                                       out, out_row, flags, None)


@pytest.mark.parametrize("call", [quantize, dequantize, norm, matmul])
def test_valid_arguments_reach_the_device_check(lib, call):
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    assert call() in (4, 5)
    assert call(flags=ar.FLAG_PDL) in (4, 5)


BAD_MATRIX = [
    (dict(fmt=0), 1), (dict(fmt=4), 1), (dict(rows=-1), 1), (dict(rows=1 << 31), 1),
    (dict(cols=0), 1), (dict(cols=48), 1), (dict(cols=1 << 31), 1),
    (dict(data=0), 1), (dict(scales=0), 1), (dict(row_bytes=112), 1), (dict(row_bytes=1 << 41), 1),
    (dict(rows=1 << 30, row_bytes=1 << 40), 1),
    (dict(tensor_scale=addr(9)), 1),              # only nvfp4 has one
    (dict(data=addr(1, 8)), 2), (dict(scales=addr(5, 4)), 2), (dict(row_bytes=136), 2),
    (dict(fmt=3, tensor_scale=addr(9, 2)), 2),
]


@pytest.mark.parametrize("change,status", BAD_MATRIX)
@pytest.mark.parametrize("call", [quantize, dequantize, norm])
def test_matrix_refusals(lib, call, change, status):
    assert call(q=matrix(1, **change)) == status


@pytest.mark.parametrize("change,status", BAD_MATRIX)
def test_matmul_matrix_refusals(lib, change, status):
    other = {k: change[k] for k in ("fmt", "cols") if k in change}
    assert matmul(a=matrix(1, **change), w=matrix(2, **other)) == status
    assert matmul(a=matrix(2, **other), w=matrix(1, **change)) == status


@pytest.mark.parametrize("call,change,status", [
    (quantize, dict(x=0), 1), (quantize, dict(x_row=248), 1), (quantize, dict(x=addr(0, 8)), 2),
    (quantize, dict(x_row=260), 2), (quantize, dict(flags=2), 1), (quantize, dict(x=addr(1)), 3),
    (quantize, dict(x=addr(1, 1 << 32)), 3), (quantize, dict(x_row=1 << 41), 1),
    (dequantize, dict(x=0), 1), (dequantize, dict(x=addr(1, -512)), 3),
    (dequantize, dict(x=addr(1, (1 << 32) - 1024)), 3), (dequantize, dict(x_row=1 << 41), 1),
    (dequantize, dict(flags=ar.FLAG_KERNEL(1)), 1),
    (norm, dict(prefix=0), 1), (norm, dict(weight=0), 1), (norm, dict(eps=-1.0), 1),
    (norm, dict(eps=float("nan")), 1), (norm, dict(eps=float("inf")), 1),
    (norm, dict(prefix_row=248), 1), (norm, dict(delta_row=0), 1), (norm, dict(norm_row=8), 1),
    (norm, dict(prefix=addr(0, 2)), 2), (norm, dict(delta=addr(2, 8)), 2),
    (norm, dict(weight=addr(3, 8)), 2), (norm, dict(norm_out=addr(4, 4)), 2),
    (norm, dict(prefix_row=257), 2), (norm, dict(delta_row=260), 2), (norm, dict(norm_row=260), 2),
    (norm, dict(delta=addr(0)), 3), (norm, dict(norm_out=addr(0, 64)), 3),
    (norm, dict(weight=addr(4, 1024)), 3), (norm, dict(norm_out=addr(1, 512)), 3),
    (norm, dict(norm_out=addr(2)), 3), (norm, dict(flags=4), 1),
    (matmul, dict(out=0), 1), (matmul, dict(out_row=64), 1), (matmul, dict(out=addr(0, 4)), 2),
    (matmul, dict(out_row=76), 2), (matmul, dict(out=addr(1)), 3), (matmul, dict(out=addr(2, 1024)), 3),
    (matmul, dict(out=addr(2, 1 << 32)), 3), (matmul, dict(flags=2), 1),
    (matmul, dict(flags=ar.FLAG_KERNEL(4)), 1), (matmul, dict(flags=ar.FLAG_STAGES(2)), 1),
    (matmul, dict(flags=ar.FLAG_SPLIT(1)), 1), (matmul, dict(flags=ar.FLAG_KERNEL(2) | ar.FLAG_SPLIT(1)), 1),
    (matmul, dict(flags=ar.FLAG_KERNEL(1) | ar.FLAG_SPLIT(2)), 1),  # one block of K
    (matmul, dict(flags=ar.FLAG_KERNEL(1) | ar.FLAG_SPLIT(7), a=matrix(1, cols=8192),
                  w=matrix(2, rows=70, cols=8192)), 1),
])
def test_refusals(lib, call, change, status):
    assert call(**change) == status


def test_matmul_wants_one_format_and_width(lib):
    assert matmul(w=matrix(2, fmt=3)) == 1
    assert matmul(w=matrix(2, cols=288)) == 1


def test_norm_width_limit(lib):
    kw = dict(prefix_row=65568, delta_row=65568, norm_row=65568)
    assert norm(q=matrix(1, cols=65568), **kw) == 1


def test_norm_without_delta_or_second_output(lib):
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    # neither is looked at when absent; prefix may then share nothing but itself
    assert norm(delta=None, delta_row=0, norm_out=None, norm_row=0) in (4, 5)


def test_no_rows_is_a_no_op(lib):
    assert quantize(q=matrix(1, rows=0), x=0) == 0
    assert dequantize(q=matrix(1, rows=0, data=0), x=0) == 0
    assert norm(q=matrix(1, rows=0), prefix=0) == 0
    assert matmul(a=matrix(1, rows=0), out=0) == 0
    assert matmul(w=matrix(2, rows=0), out=0) == 0
    # the scalars are looked at all the same
    assert quantize(q=matrix(1, rows=0, cols=40), x=0) == 1
    assert norm(q=matrix(1, rows=0), eps=-1.0) == 1


def test_null_matrices(lib):
    null = ctypes.POINTER(ar.Mx)()
    assert ar.lib().attn_res_mx_quantize(addr(0), 256, null, 0, None) == 1
    assert ar.lib().attn_res_mx_matmul(null, matrix(1), addr(0), 72, 0, None) == 1
    assert ar.lib().attn_res_mx_matmul(matrix(1), null, addr(0), 72, 0, None) == 1


def test_binding_refuses_what_is_not_on_the_gpu(lib):
    with pytest.raises(ValueError):
        mx.quantize(torch.zeros(4, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        mx.MxTensor(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(1), "mxfp4")
    with pytest.raises(ValueError):
        mx.MxTensor.empty(4, 64, "mxfp6")
    with pytest.raises(ValueError):
        mx.MxTensor.empty(4, 48, "mxfp4")


def test_wide_forms_take_columns_up_to_their_32_bit_places(lib):
    """A tile that reaches past the last column stays below 2^31."""
    def status(n, kernel):
        w = matrix(2, fmt=2, rows=n, cols=32, row_bytes=16, scales=addr(9))
        return matmul(a=matrix(1, rows=1, cols=32, row_bytes=16), w=w, out_row=(n + 7) // 8 * 8,
                      flags=ar.FLAG_KERNEL(kernel))
    largest = (1 << 31) - 256
    for kernel in (2, 3):
        assert status(largest, kernel) == 1
        assert status((1 << 31) - 767, kernel) == 1
    if not torch.cuda.is_available():
        assert all(status(largest, k) in (4, 5) for k in (0, 1))
        assert all(status((1 << 31) - 768, k) in (4, 5) for k in (2, 3))


THREADS = r"""
import sys
import threading
import torch
from attention_residual_fusion_gb300 import mx
sys.setswitchinterval(1e-6)
start, got, errors = threading.Barrier(16), [], []
def first():
    start.wait()
    try:
        got.append((mx.MxTensor, mx.matmul))
    except BaseException as e:
        errors.append(repr(e))
threads = [threading.Thread(target=first) for _ in range(16)]
for t in threads:
    t.start()
for t in threads:
    t.join()
assert not errors, errors
assert len(got) == 16 and len(set(got)) == 1
"""


def test_first_use_from_many_threads(lib):
    """The binding is loaded once, whichever of the threads come first."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", THREADS], cwd=root, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
