"""The 8-bit entry points on the host: the restated format against hand-worked
values, and every refusal (validation precedes the first CUDA call, so no GPU is
needed)."""
import ctypes

import pytest
import torch

import attention_residual_fusion_gb300 as ar
from attention_residual_fusion_gb300 import _build, f8
from tests import f8_restatement as R

BASE, GAP = 1 << 40, 1 << 34


def addr(i, off=0):
    return BASE + i * GAP + off


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return ar.lib()


# ---- the format ---------------------------------------------------------------


def test_e4m3_table_is_the_type():
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    assert torch.equal(torch.tensor(R.E4M3, dtype=torch.float64), t)


@pytest.mark.parametrize("v,code", [(0.0, 0), (-0.0, 128), (448.0, 126), (500.0, 126), (-448.0, 254), (17.0, 0x58), (19.0, 0x5A),
                                    (2.0 ** -10, 0), (2.0 ** -9, 1), (1.5 * 2.0 ** -9, 2), (1.0, 0x38), (1.0625, 0x38)])
def test_e4m3_rounding(v, code):
    assert R.nearest_code(torch.tensor([v], dtype=torch.float64)).item() == code


def test_quantisation_by_hand():
    x = torch.zeros(3, 130, dtype=torch.bfloat16)
    x[0, 0], x[0, 1], x[0, 129] = 448.0, -17.0, 2.0
    x[1, 3] = 2.0 ** -130
    x[2, 5] = float("inf")
    codes, s = R.quantize(x, 1)
    assert s.shape == (2, 3) and s[0, 0] == 1.0 and s[1, 0] == torch.tensor(2.0).div(448.0)
    assert codes[0, 0] == 126 and codes[0, 1] == 0x58 | 128 and codes[0, 129] == 126
    assert s[0, 1] == 2.0 ** -126 and codes[1, 3] == R.nearest_code(torch.tensor([2.0 ** -4], dtype=torch.float64)).item()
    assert s[1, 1] == 1.0 and torch.isnan(s[0, 2]) and not codes[2].any()
    codes, s = R.quantize(x[:2], 128)
    assert s.shape == (1, 2) and s[0, 0] == 1.0


def test_scales_shape():
    assert f8.scales_shape(300, 1000) == (8, 300) and f8.scales_shape(300, 1000, 128) == (3, 8)
    assert f8.scales_shape(0, 128) == (1, 0) and f8.scales_shape(5, 0) == (0, 5)


# ---- refusals -------------------------------------------------------------------

ROWS, SQUARE = 1, 128


def matrix(i, block=ROWS, rows=40, cols=256, **change):
    b = R.scales_shape(rows, cols, block)[1] if rows > 0 and cols > 0 else 0
    kw = dict(block=block, rows=rows, cols=cols, data=addr(i), row_bytes=(cols + 15) // 16 * 16, scales=addr(i, 1 << 32),
              scales_row=(b + 3) // 4 * 4)
    kw.update(change)
    return ar.F8(*(kw[n] for n, _ in ar.F8._fields_))


NULL = ctypes.POINTER(ar.F8)()


def quantize(q=None, qt=None, x=addr(0), x_row=256, flags=0):
    return ar.lib().attn_res_f8_quantize(x, x_row, q or matrix(1), NULL if qt is None else qt, flags, None)


def quantize_both(q=None, qt=None, **kw):
    return quantize(q, matrix(2, rows=256, cols=40) if qt is None else qt, **kw)


def dequantize(q=None, x=addr(0), x_row=256, flags=0):
    return ar.lib().attn_res_f8_dequantize(q or matrix(1), x, x_row, flags, None)


def matmul(a=None, w=None, a2=None, w2=None, out=addr(0), out_row=72, out_type=0, flags=0):
    return ar.lib().attn_res_f8_matmul(a or matrix(1), w or matrix(2, SQUARE, rows=70), a2 or NULL, w2 or NULL, out, out_row,
                                       out_type, flags, None)


def matmul_pair(a2=None, w2=None, **kw):
    return matmul(a2=a2 or matrix(3, cols=100), w2=w2 or matrix(4, SQUARE, rows=70, cols=100), **kw)


def gated(x=None, gate=None, up=None, act=1, h=None, rows=0, row=0, g=None, u=None, flags=0):
    if h is None and not rows:
        h = matrix(4, cols=72)
    return ar.lib().attn_res_f8_gated(x or matrix(1), gate or matrix(2, SQUARE, rows=72), up or matrix(3, SQUARE, rows=72), act,
                                      h or NULL, rows, row, g or NULL, u or NULL, flags, None)


def gated_saving(g=None, u=None, **kw):
    return gated(g=g or matrix(5, cols=72), u=u or matrix(6, cols=72), **kw)


def backward(dh=addr(0), dh_row=256, g=None, u=None, act=1, dg=None, du=None, t=(), flags=0):
    t = list(t) + [NULL] * (3 - len(t))
    return ar.lib().attn_res_f8_gated_backward(dh, dh_row, g or matrix(1), u or matrix(2), act, dg or matrix(3), du or matrix(4),
                                               *t, flags, None)


def transposes(**change):
    return [matrix(5 + i, rows=256, cols=40, **change) for i in range(3)]


def backward_all(t=None, **kw):
    return backward(t=transposes() if t is None else t, **kw)


@pytest.mark.parametrize("call", [quantize, quantize_both, dequantize, matmul, matmul_pair, gated, gated_saving, backward,
                                  backward_all])
def test_valid_arguments_reach_the_device_check(lib, call):
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    assert call() in (4, 5)
    assert call(flags=ar.FLAG_PDL) in (4, 5)
    assert call(flags=2) == 1


BAD = [
    (dict(block=0), 1), (dict(block=2), 1), (dict(rows=-1), 1), (dict(rows=(1 << 31) - 1023), 1), (dict(cols=-1), 1),
    (dict(cols=1 << 31), 1), (dict(data=0), 1), (dict(scales=0), 1), (dict(row_bytes=240), 1), (dict(row_bytes=1 << 41), 1),
    (dict(scales_row=36), 1), (dict(scales_row=1 << 41), 1), (dict(data=addr(1, 8)), 2), (dict(row_bytes=264), 2),
    (dict(scales=addr(1, (1 << 32) + 8)), 2), (dict(scales_row=42), 2),
]


@pytest.mark.parametrize("change,status", BAD)
def test_matrix_refusals(lib, change, status):
    kw = dict(change)
    block = kw.pop("block", ROWS)
    assert quantize(matrix(1, block, **kw)) == status
    assert dequantize(matrix(1, block, **kw)) == status
    cols = kw.get("cols", 256)
    assert matmul(a=matrix(1, block, **kw), w=matrix(2, SQUARE, rows=70, cols=cols)) == status
    if block == ROWS:
        assert gated(x=matrix(1, **kw), gate=matrix(2, SQUARE, rows=72, cols=cols),
                     up=matrix(3, SQUARE, rows=72, cols=cols)) == status
        assert backward(g=matrix(1, **kw)) == status
        assert backward(dg=matrix(1, **kw)) == status
        t = transposes()
        t[1] = matrix(6, rows=256, cols=40, **kw) if "rows" not in kw and "cols" not in kw and "row_bytes" not in kw and \
            "scales_row" not in kw else t[1]
        if t[1].rows == 256 and change.keys() & {"data", "scales"}:
            assert backward(t=t) == status


@pytest.mark.parametrize("change,status", [
    (dict(scales_row=1), 1), (dict(scales=addr(1, (1 << 32) + 2)), 2), (dict(data=0), 1), (dict(row_bytes=264), 2)])
def test_block_scaled_refusals(lib, change, status):
    assert quantize(matrix(1, SQUARE, **change)) == status
    assert matmul(w=matrix(1, SQUARE, rows=70, **change), a=matrix(2)) == status
    assert gated(up=matrix(3, SQUARE, rows=72, **{k: v for k, v in change.items()})) == status


def test_block_scales_need_no_alignment(lib):
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    assert quantize(matrix(1, SQUARE, scales=addr(1, (1 << 32) + 4), scales_row=3)) in (4, 5)


@pytest.mark.parametrize("call,change,status", [
    (quantize, dict(x=0), 1), (quantize, dict(x_row=248), 1), (quantize, dict(x=addr(0, 8)), 2), (quantize, dict(x_row=260), 2),
    (quantize, dict(x=addr(1)), 3), (quantize, dict(x=addr(1, 1 << 32)), 3),
    (quantize_both, dict(qt=matrix(2, rows=256, cols=41)), 1), (quantize_both, dict(qt=matrix(2, rows=255, cols=40)), 1),
    (quantize_both, dict(qt=matrix(2, SQUARE, rows=256, cols=40)), 1), (quantize_both, dict(qt=matrix(1, rows=256, cols=40)), 3),
    (quantize_both, dict(qt=matrix(2, rows=256, cols=40, scales=addr(1, (1 << 32) + 160))), 3),
    (quantize_both, dict(qt=matrix(2, rows=256, cols=40, data=addr(2, 4))), 2),
    (quantize_both, dict(qt=matrix(0, rows=256, cols=40)), 3),
    (dequantize, dict(x=0), 1), (dequantize, dict(x=addr(1, -512)), 3), (dequantize, dict(x_row=1 << 41), 1),
    (dequantize, dict(x=addr(1, (1 << 32) - 1024)), 3), (dequantize, dict(flags=ar.FLAG_KERNEL(1)), 1),
    (matmul, dict(out=0), 1), (matmul, dict(out_row=64), 1), (matmul, dict(out=addr(0, 4)), 2), (matmul, dict(out_row=76), 2),
    (matmul, dict(out_type=3), 1), (matmul, dict(out_type=-1), 1), (matmul, dict(out_type=1, out_row=74), 2),
    (matmul, dict(out_type=1, out=addr(0, 8)), 2), (matmul, dict(out=addr(1)), 3), (matmul, dict(out=addr(2, 1024)), 3),
    (matmul, dict(out=addr(2, 1 << 32)), 3), (matmul, dict(a=matrix(1, SQUARE)), 1), (matmul, dict(w=matrix(2, cols=257)), 1),
    (matmul, dict(a2=matrix(3)), 1), (matmul, dict(w2=matrix(3)), 1),
    (matmul_pair, dict(a2=matrix(3, rows=41, cols=100)), 1), (matmul_pair, dict(w2=matrix(4, rows=70, cols=100)), 1),
    (matmul_pair, dict(w2=matrix(4, SQUARE, rows=70, cols=101)), 1), (matmul_pair, dict(a2=matrix(3, SQUARE, cols=100)), 1),
    (matmul_pair, dict(w2=matrix(4, SQUARE, rows=71, cols=100)), 1), (matmul_pair, dict(out=addr(3)), 3),
    (matmul_pair, dict(out=addr(4, 1 << 32)), 3), (matmul_pair, dict(a2=matrix(3, cols=100, data=addr(3, 1))), 2),
    (gated, dict(act=0), 1), (gated, dict(act=3), 1), (gated, dict(x=matrix(1, SQUARE)), 1), (gated, dict(x=matrix(1, cols=255)), 1),
    (gated, dict(gate=matrix(2, rows=72)), 1), (gated, dict(up=matrix(3, SQUARE, rows=73)), 1),
    (gated, dict(h=matrix(4, cols=73)), 1), (gated, dict(h=matrix(4, SQUARE, cols=72)), 1), (gated, dict(h=matrix(1, cols=72)), 3),
    (gated, dict(h=matrix(4, cols=72), rows=addr(7), row=72), 1), (gated, dict(rows=addr(7), row=64), 1),
    (gated, dict(rows=addr(7, 2), row=72), 2), (gated, dict(rows=addr(2), row=72), 3),
    (gated, dict(g=matrix(5, cols=72)), 1), (gated, dict(u=matrix(5, cols=72)), 1),
    (gated_saving, dict(g=matrix(5, cols=71)), 1), (gated_saving, dict(u=matrix(5, cols=72)), 3),
    (gated_saving, dict(u=matrix(4, cols=72)), 3), (gated_saving, dict(g=matrix(5, cols=72, data=addr(5, 8))), 2),
    (backward, dict(dh=0), 1), (backward, dict(dh_row=248), 1), (backward, dict(dh=addr(0, 8)), 2), (backward, dict(dh_row=260), 2),
    (backward, dict(act=0), 1), (backward, dict(u=matrix(2, cols=255)), 1), (backward, dict(g=matrix(1, SQUARE)), 1),
    (backward, dict(du=matrix(4, rows=41)), 1), (backward, dict(dg=matrix(1)), 3), (backward, dict(du=matrix(3)), 3),
    (backward, dict(dg=matrix(0)), 3), (backward, dict(t=transposes()[:2]), 1), (backward, dict(t=[NULL, NULL, transposes()[0]]), 1),
    (backward_all, dict(t=[transposes()[0]] * 2 + [transposes()[2]]), 3),
    (backward_all, dict(t=transposes()[:2] + [matrix(7, rows=256, cols=41)]), 1),
    (backward_all, dict(t=transposes()[:2] + [matrix(7, rows=40, cols=256)]), 1),
])
def test_refusals(lib, call, change, status):
    assert call(**change) == status


@pytest.mark.parametrize("call", [matmul, gated])
def test_forms(lib, call):
    big = dict(a=matrix(1, cols=4096), w=matrix(2, SQUARE, rows=70, cols=4096)) if call is matmul else dict(
        x=matrix(1, cols=4096), gate=matrix(2, SQUARE, rows=72, cols=4096), up=matrix(3, SQUARE, rows=72, cols=4096))
    K, S = ar.FLAG_KERNEL, ar.FLAG_SPLIT
    for flags in (K(3), S(1), K(2) | S(1), K(1) | S(3), ar.FLAG_STAGES(2), ar.FLAG_TP_GRAM):
        assert call(flags=flags) == 1  # (two blocks of K)
    assert call(flags=K(1) | S(9), **big) == 1
    if not torch.cuda.is_available():
        for flags in (K(1), K(2), K(1) | S(2), K(1) | ar.FLAG_PDL):
            assert call(flags=flags) in (4, 5)
        assert call(flags=K(1) | S(8), **big) in (4, 5)


def test_nothing_to_write_is_a_no_op(lib):
    assert quantize(matrix(1, rows=0, data=0), x=0) == 0
    assert quantize(matrix(1, cols=0, data=0), x=0) == 0
    assert quantize_both(matrix(1, rows=0), qt=matrix(2, rows=256, cols=0), x=0) == 0
    assert dequantize(matrix(1, rows=0), x=0) == 0
    assert matmul(a=matrix(1, rows=0), out=0) == 0
    assert matmul(w=matrix(2, SQUARE, rows=0), out=0) == 0
    assert gated(x=matrix(1, rows=0), h=matrix(4, rows=0, cols=72)) == 0
    assert backward(dh=0, g=matrix(1, rows=0), u=matrix(2, rows=0), dg=matrix(3, rows=0), du=matrix(4, rows=0)) == 0
    # the scalars are looked at all the same
    assert quantize(matrix(1, 3, rows=0), x=0) == 1
    assert matmul(a=matrix(1, rows=0), out_type=7) == 1
    assert backward(act=5, g=matrix(1, rows=0), u=matrix(2, rows=0), dg=matrix(3, rows=0), du=matrix(4, rows=0)) == 1


def test_a_width_of_zero_still_has_a_result(lib):
    """The sum over no columns is written: its out is checked."""
    a, w = matrix(1, cols=0, data=0, scales=0), matrix(2, SQUARE, rows=70, cols=0, data=0, scales=0)
    assert matmul(a=a, w=w, out=0) == 1
    if not torch.cuda.is_available():
        assert matmul(a=a, w=w) in (4, 5)


def test_null_matrices(lib):
    L = lib
    assert L.attn_res_f8_quantize(addr(0), 256, NULL, NULL, 0, None) == 1
    assert L.attn_res_f8_dequantize(NULL, addr(0), 256, 0, None) == 1
    for a, w in ((NULL, matrix(2, SQUARE, rows=70)), (matrix(1), NULL)):
        assert L.attn_res_f8_matmul(a, w, NULL, NULL, addr(0), 72, 0, 0, None) == 1
    m, s, h = matrix(1), [matrix(2 + i, SQUARE, rows=72) for i in range(2)], matrix(4, cols=72)
    for args in ((NULL, s[0], s[1]), (m, NULL, s[1]), (m, s[0], NULL)):
        assert L.attn_res_f8_gated(*args, 1, h, None, 0, NULL, NULL, 0, None) == 1
    assert L.attn_res_f8_gated(m, *s, 1, NULL, None, 0, NULL, NULL, 0, None) == 1  # no result
    assert L.attn_res_f8_gated_backward(addr(0), 256, NULL, m, 1, h, h, NULL, NULL, NULL, 0, None) == 1


def test_binding_refuses_what_is_not_on_the_gpu(lib):
    with pytest.raises(ValueError):
        f8.quantize(torch.zeros(4, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        f8.F8Tensor(torch.zeros(4, 32, dtype=torch.float8_e4m3fn), torch.zeros(1, 4))
    with pytest.raises(ValueError):
        f8.F8Tensor.empty(4, 64, 64)
    with pytest.raises(ValueError):
        f8.F8Tensor.empty(4, -1)
    with pytest.raises(ValueError):
        f8.F8Tensor.empty(4, 64, device="cpu")
    with pytest.raises(AttributeError):
        f8.nothing
