"""Sizes and strides that the 8-bit kernels cannot take are refused before the
first CUDA call (so no GPU is needed)."""
import pytest
import torch

from tests.test_f8_host import addr, backward, lib, matrix  # noqa: F401  (lib: a fixture)


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
