"""The 8-bit row kernels, the gated block and the backward pass beyond 2^32 bytes and
2^32 elements of their buffers' starts."""
import pytest
import torch

import attention_residual_fusion_gb300 as ar
from attention_residual_fusion_gb300 import _build, f8
from tests import f8_restatement as R
from tests.test_f8_gpu import Rows, activations, backward_want, equal_with_nan, within

pytestmark = pytest.mark.gpu

FAR = 1 << 32  # bytes from a matrix's first row to its last, at least


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    ar.device_status(clear=True)
    yield
    assert ar.device_status() == 0
    torch.cuda.empty_cache()


def far_rows(rows, cols, dtype):
    """Rows so far apart that the last lies FAR bytes behind the first."""
    size = torch.empty(0, dtype=dtype).element_size()
    apart = -(-FAR // (max(1, rows - 1) * size) // 16) * 16 + 16
    return torch.empty((rows - 1) * apart + cols, dtype=dtype, device="cuda").as_strided((rows, cols), (apart, 1))


def far_matrix(rows, cols, block=1):
    scales = far_rows(*R.scales_shape(rows, cols, block), torch.float32)
    return f8.F8Tensor(far_rows(rows, cols, torch.uint8).view(torch.float8_e4m3fn), scales, block)


def far_copy(q):
    t = far_matrix(*q.shape, q.block)
    t.data.view(torch.uint8).copy_(q.data.view(torch.uint8))
    t.scales.copy_(q.scales)
    return t


def same(got, want):
    for a, b in zip(got, want):
        assert torch.equal(a.data.view(torch.uint8), b.data.view(torch.uint8)) and torch.equal(a.scales, b.scales)


# the near calls are those that the other tests hold against 64 bits
T, F, H = 130, 260, 300


def near_rows(rows, cols, seed, scale=1.0):
    return Rows(rows, cols, 0, activations(rows, cols, seed, scale)).t


@pytest.mark.parametrize("block", [1, 128])
def test_quantize_and_back(block):
    near = near_rows(T, F, 1)
    x = far_rows(T, F, torch.bfloat16).copy_(near)
    q, t = far_matrix(T, F, block), far_matrix(F, T, block)
    f8.quantize(x, block, q, transposed=t)
    want = f8.quantize(near, block, transposed=True)
    same((q, t), want)
    q.data.view(torch.uint8).zero_()
    f8.quantize(x, block, q)
    same((q,), want)
    back = far_rows(T, F, torch.bfloat16)
    f8.dequantize(q, back)
    assert torch.equal(back, f8.dequantize(want[0]))


@pytest.mark.parametrize("kernel", [f8.KERNEL_NARROW, f8.KERNEL_WIDE])
def test_gated(kernel):
    x = f8.quantize(near_rows(T, H, 1))
    gate, up = (f8.quantize(near_rows(F, H, i, 0.05), 128) for i in (2, 3))
    want = f8.gated(x, gate, up, save=True, kernel=kernel)
    far = [far_copy(t) for t in (x, gate, up)]
    out = [far_matrix(T, F) for _ in range(3)]
    f8.gated(*far, out=out[0], save=out[1:], kernel=kernel)
    same(out, want)
    rows = far_rows(T, F, torch.bfloat16)
    f8.gated(*far, out=rows, kernel=kernel)
    assert torch.equal(rows, f8.gated(x, gate, up, dtype=torch.bfloat16, kernel=kernel))


def test_backward():
    dh, g, u = near_rows(T, F, 1), f8.quantize(near_rows(T, F, 2)), f8.quantize(near_rows(T, F, 3))
    want = f8.gated_backward(dh, g, u)
    out = [far_matrix(T, F) for _ in range(2)] + [far_matrix(F, T) for _ in range(3)]
    f8.gated_backward(far_rows(T, F, torch.bfloat16).copy_(dh), far_copy(g), far_copy(u), out=out)
    same(out, want)


# ---- dense: tiles beyond 2^32 elements ----------------------------------------------------

ROWS, COLS = 70000, 65536
SOME_ROWS, SOME_COLS = [0, 32767, 32768, 65535, 69999], [0, 127, 128, 40000, 65535]


def check_rows(q, want, rows):
    """The codes and scales of some rows."""
    assert torch.equal(q.data[rows].view(torch.uint8), want[0]) and equal_with_nan(q.scales[:, rows], want[1])


def test_dense_quantize():
    x = torch.empty(ROWS, COLS, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    q, t = f8.quantize(x, transposed=True)
    check_rows(q, R.quantize(x[SOME_ROWS], 1), SOME_ROWS)
    check_rows(t, R.quantize(x[:, SOME_COLS].t().contiguous(), 1), SOME_COLS)
    q, t = f8.quantize(x, 128, transposed=True)
    for r0 in (0, 32768, ROWS - ROWS % 128):  # whole rows of blocks
        codes, scales = R.quantize(x[r0:r0 + 128, -896:], 128)
        assert torch.equal(q.data[r0:r0 + 128, -896:].view(torch.uint8), codes)
        assert torch.equal(q.scales[r0 // 128, -7:], scales[0])
        assert torch.equal(t.data[-896:, r0:r0 + 128].view(torch.uint8), codes.t())
        assert torch.equal(t.scales[-7:, r0 // 128], scales[0])


def test_dense_gated():
    """Results of 70000 x 65536: those of some tokens alone."""
    x = f8.quantize(activations(ROWS, 128, 1))
    gate, up = (f8.quantize(activations(COLS, 128, i, 0.1), 128) for i in (2, 3))
    got = f8.gated(x, gate, up, save=True)
    part = f8.F8Tensor(x.data[SOME_ROWS], x.scales[:, SOME_ROWS + [0] * 3][:, :len(SOME_ROWS)])
    want = f8.gated(part, gate, up, save=True, kernel=f8.KERNEL_WIDE)
    for a, b in zip(got, want):
        check_rows(a, (b.data.view(torch.uint8), b.scales), SOME_ROWS)


def test_dense_backward():
    gen = torch.Generator(device="cuda").manual_seed(2)
    dh = torch.empty(ROWS, COLS, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    g, u = (f8.F8Tensor(torch.randint(0, 0x7F, (ROWS, COLS), dtype=torch.uint8, device="cuda", generator=gen).view(torch.float8_e4m3fn),
                        torch.rand(COLS // 128, ROWS, device="cuda", generator=gen) * 0.01 + 0.001) for _ in range(2))
    got = f8.gated_backward(dh, g, u)

    def check(q, rows, want, error):
        part = f8.F8Tensor(q.data[rows], q.scales[:, rows])
        s = part.scales.t().repeat_interleave(128, 1)[:, :want.shape[1]].double()
        v = part.data.double() * s
        within(v, want, R.code_bound(want, error, s))

    def values(m, rows, cols):
        s = m.scales.t()[rows][:, [c // 128 for c in cols]] if cols else m.scales.t()[rows].repeat_interleave(128, 1)
        codes = m.data[rows] if not cols else m.data[:, cols]
        return codes.double() * s.double()

    (dg, e1), (du, e2), _ = backward_want(dh[SOME_ROWS], values(g, SOME_ROWS, None), values(u, SOME_ROWS, None), "silu")
    check(got[0], SOME_ROWS, dg, e1)
    check(got[1], SOME_ROWS, du, e2)
    every = slice(None)
    (dg, e1), (du, e2), (h, e3) = backward_want(dh[:, SOME_COLS], values(g, every, SOME_COLS), values(u, every, SOME_COLS), "silu")
    for q, want, e in zip(got[2:], (dg, du, h), (e1, e2, e3)):
        check(q, SOME_COLS, want.t().contiguous(), e.t().contiguous())
