"""Products of the longest rows that the entry points take (2^30 columns)."""
import pytest
import torch

import attention_residual_fusion_gb300 as ar
from attention_residual_fusion_gb300 import _build, mx

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    ar.device_status(clear=True)
    yield
    assert ar.device_status() == 0


@pytest.mark.slow
@pytest.mark.parametrize("kernel,split", [(0, 0), (1, 1), (2, 0), (3, 0)])
def test_products_of_the_longest_rows(kernel, split):
    """All of K in one CTA or pair takes seconds: longer than a wait that has
    lost its completion is given.  The ends of the rows count."""
    rows, cols = 2, 1 << 30
    shape = mx.scales_shape("mxfp8", rows, cols)
    scales = torch.zeros(shape, dtype=torch.uint8, device="cuda")
    scales[0, :, :rows, 0] = 127  # 1, for the rows that exist
    data = torch.zeros(rows, cols, dtype=torch.uint8, device="cuda")
    at = torch.tensor([0, 31, 1 << 20, (1 << 29) + 5, cols - 33, cols - 1], device="cuda")
    codes = torch.tensor([[0x38, 0x40, 0x38, 0x40, 0x48, 0x38], [0x40, 0xB8, 0x38, 0xC0, 0x38, 0x40]],
                         dtype=torch.uint8, device="cuda")  # 1, 2, 1, 2, 4, 1 and 2, -1, 1, -2, 1, 2
    data[:, at] = codes
    q = mx.MxTensor(data.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu), "mxfp8")
    v = codes.view(torch.float8_e4m3fn).double()
    out = mx.matmul(q, q, kernel=kernel, split=split)
    torch.cuda.synchronize()
    assert ar.device_status() == 0
    assert torch.equal(out.double(), v @ v.t())
