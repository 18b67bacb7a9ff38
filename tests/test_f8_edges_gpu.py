"""The 8-bit calls at the ends of what their documentation allows."""
import pytest
import torch

import attention_residual_fusion_gb300 as ar
from attention_residual_fusion_gb300 import _build, f8
from tests.test_f8_gpu import Matrix, Rows

pytestmark = pytest.mark.gpu

KERNELS = [f8.KERNEL_NARROW, f8.KERNEL_WIDE, 0]
ONE = 0x38  # the code of 1


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    ar.device_status(clear=True)
    yield
    assert ar.device_status() == 0


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T,F", [(1, 1), (20, 300), (300, 260)])
def test_gated_without_columns(T, F, act, kernel):
    """Projections of nothing are zeros: codes 0 with the scale 1, and nothing beside them."""
    x, w = f8.F8Tensor.empty(T, 0), f8.F8Tensor.empty(F, 0, 128)
    out = [Matrix(T, F, 1, 1) for _ in range(3)]
    f8.gated(x, w, w, act, out[0].t, save=(out[1].t, out[2].t), kernel=kernel)
    for o in out:
        assert bool((o.codes & 0x7F == 0).all()) and bool((o.scales == 1).all()) and o.intact()
    rows = Rows(T, F, 8)
    f8.gated(x, w, w, act, rows.t, kernel=kernel)
    assert bool((rows.t == 0).all()) and rows.intact()


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("m,n", [(3, 200), (300, 257)])
def test_products_of_scales_beyond_fp32(m, n, block, kernel):
    """Above 2^128 infinite, NaN where the block's sum is 0; below 2^-149 zero.  (Columns 0 and 1 hold codes of 1 and -1
    in a; in w a 1 in column 0, and in the odd rows in column 1 too.)"""
    a, w = Matrix(m, 130), Matrix(n, 130, block)
    a.codes.zero_()
    w.codes.zero_()
    a.codes[:, 0], a.codes[:, 1] = ONE, ONE | 128
    w.codes[:, 0], w.codes[1::2, 1] = ONE, ONE
    for e, of_ones in ((65.0, float("inf")), (-75.0, 0.0)):
        a.scales.fill_(2.0 ** e)
        w.scales.fill_(2.0 ** e)
        a.scales[1], w.scales[(slice(None), 1) if block == 128 else 1] = 1.0, 1.0  # (the second block of K: nothing)
        f = f8.matmul(a.t, w.t, dtype=torch.float32, kernel=kernel)
        assert bool((f[:, ::2] == of_ones).all())
        assert bool(torch.isnan(f[:, 1::2]).all() if e > 0 else (f[:, 1::2] == 0).all())
