"""Sizes and strides that the 8-bit kernels cannot take are refused before the
first CUDA call (so no GPU is needed)."""
import pytest
import torch

import attention_residual_fusion_gb300 as ar
from tests.test_f8_host import SQUARE, addr, backward, gated, lib, matmul, matrix  # noqa: F401  (lib: a fixture)


def one_token(i, **kw):
    return matrix(i, rows=1, **kw)


def backward_of_one_token(g=None, u=None, **kw):
    return backward(g=g or one_token(1), u=u or one_token(2), dg=one_token(3), du=one_token(4), **kw)


@pytest.mark.parametrize("change", [
    dict(dh_row=1 << 39), dict(dh_row=1 << 40), dict(g=one_token(1, scales_row=1 << 38)), dict(u=one_token(2, scales_row=1 << 38)),
    dict(u=one_token(2, scales_row=(1 << 40) - 4))])
def test_backward_strides_beyond_tensor_maps(lib, change):  # noqa: F811
    """The stride of a single row too; 2^40 bytes are the first that a tensor map does not hold."""
    assert backward_of_one_token(**change) == 1


@pytest.mark.skipif(torch.cuda.is_available(), reason="a device is present")
@pytest.mark.parametrize("change", [
    dict(), dict(dh_row=(1 << 39) - 8), dict(g=one_token(1, scales=addr(200), scales_row=(1 << 38) - 4))])
def test_backward_strides_below(lib, change):  # noqa: F811
    """What tensor maps hold passes the checks."""
    assert backward_of_one_token(**change) in (4, 5)


FAR = 1 << 60  # results of that size, beyond every other argument


def large_product(rows, n, flags=0):
    # (rows of 16 bytes; the scales of a's rows far behind its codes)
    a = matrix(1, rows=rows, cols=8, scales=1 << 58)
    return matmul(a=a, w=matrix(2, SQUARE, rows=n, cols=8, scales=1 << 57), out=FAR, out_row=n, flags=flags)


def large_block(T, F, flags=0):
    x = matrix(1, rows=T, cols=8, scales=1 << 58)
    gate, up = (matrix(2 + i, SQUARE, rows=F, cols=8, data=(1 << 56) + (i << 50), scales=(1 << 57) + (i << 50)) for i in range(2))
    return gated(x=x, gate=gate, up=up, rows=FAR, row=F, flags=flags)


@pytest.mark.parametrize("call,rows,n", [(large_product, 1 << 23, 1 << 23), (large_product, (1 << 23) + 1, 1 << 23),
                                         (large_block, 1 << 23, 1 << 22)])
def test_tiles_that_the_wide_form_counts(lib, call, rows, n):  # noqa: F811
    """2^30 - 1 tiles are the most; the narrow form takes 65535 tiles of tokens and any columns."""
    assert call(rows, n + 256) == 1
    assert call(rows, n + 256, ar.FLAG_KERNEL(2)) == 1
    if not torch.cuda.is_available():
        assert call(rows, n - 256 * 128) in (4, 5)
        assert call(rows, n - 256 * 128, ar.FLAG_KERNEL(2)) in (4, 5)
        assert call(1 << 20, 1 << 28, ar.FLAG_KERNEL(1)) in (4, 5)
