"""The persistent forms of the 8-bit kernels where every CTA goes through several
tiles: phases of the barriers and rings of scales that carry over from tile to tile
(with blocks of K that are no multiple of four), the next tile's work beside the
last one's end, stages and maxima used again."""
import pytest
import torch

import attention_residual_fusion_gb300 as ar
from attention_residual_fusion_gb300 import _build, f8
from tests.test_f8_gpu import BF16_HALF, Matrix, Rows, activations, backward_want, check_codes, gated_want, product_want, quantized, within

pytestmark = pytest.mark.gpu

WIDE = dict(kernel=f8.KERNEL_WIDE)


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    ar.device_status(clear=True)
    yield
    assert ar.device_status() == 0


# 18 x 16 tiles of 256 x 256 for 76 pairs of CTAs: three or four each, the last of the bands of token tiles two high
M, N = 4355, 3852


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("k", [(650,), (128,), (1020,), (650, 300)], ids=str)
def test_products(k, block):
    """Six blocks of K, one, eight; two pairs of six and three."""
    pairs = [(quantized(M, kk, i, pad=i), quantized(N, kk, i + 5, block, scale=0.05)) for i, kk in enumerate(k)]
    (a, w), plus = pairs[0], None if len(k) == 1 else (pairs[1][0].t, pairs[1][1].t)
    want, bound = product_want(pairs, sum(k) + 128 * (len(k) - 1))
    f = f8.matmul(a.t, w.t, dtype=torch.float32, plus=plus, **WIDE)  # (rows of 3852 floats: no multiple of 32 bytes)
    within(f, want, bound, "fp32")
    assert torch.equal(f, f8.matmul(a.t, w.t, dtype=torch.float32, plus=plus, **WIDE))
    out = Rows(M, N, 8)
    f8.matmul(a.t, w.t, out.t, plus=plus, **WIDE)
    assert torch.equal(out.t, f.to(torch.bfloat16)) and out.intact()
    within(out.t, want, bound + BF16_HALF * (want.abs() + bound), "bf16")
    del out
    for row in (N, N + 4):  # fp32 rows from 16-byte and from 32-byte boundaries, added to
        buf = torch.full((M, row), 3.25, device="cuda")
        buf[:, :N] = torch.randn(M, N, generator=torch.Generator(device="cuda").manual_seed(5), device="cuda")
        before = buf[:, :N].clone()
        f8.matmul(a.t, w.t, buf[:, :N], add=True, plus=plus, **WIDE)
        assert torch.equal(buf[:, :N], before + f) and bool((buf[:, N:] == 3.25).all())


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("H", [650, 128, 1020])
def test_gated(H, act):
    """18 x 16 tiles of 256 x 128; codes and scales of the result and of the checkpoint."""
    T, F = M, 1930
    x = quantized(T, H, 1)
    wg, wu = quantized(F, H, 2, 128, scale=H ** -0.5), quantized(F, H, 3, 128, pad=1, scale=H ** -0.5)
    g, u, h, eg, eu, eh = gated_want(x, wg, wu, act)
    out = [Matrix(T, F, 1, i) for i in range(3)]
    f8.gated(x.t, wg.t, wu.t, act, out[0].t, save=(out[1].t, out[2].t), **WIDE)
    for got, want, e, what in zip(out, (h, g, u), (eh, eg, eu), ("h", "g", "u")):
        check_codes(got, want, e, what)
    again = f8.gated(x.t, wg.t, wu.t, act, **WIDE)
    assert torch.equal(again.data.view(torch.uint8), out[0].codes) and torch.equal(again.scales, out[0].scales)
    rows = Rows(T, F, 8)
    f8.gated(x.t, wg.t, wu.t, act, rows.t, **WIDE)
    within(rows.t, h, eh + BF16_HALF * (h.abs() + eh), "bf16")
    assert rows.intact()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_backward(act):
    """24 x 21 tiles of 128 x 128 for 152 CTAs."""
    T, F = 3003, 2600
    dh = Rows(T, F, 8, activations(T, F, 1, 1e-3))
    g, u = quantized(T, F, 2, pad=1, scale=2.0), quantized(T, F, 3)
    out = [Matrix(T, F, 1, 1), Matrix(T, F)] + [Matrix(F, T, 1, i) for i in range(3)]
    f8.gated_backward(dh.t, g.t, u.t, act, [o.t for o in out])
    (dg, eg), (du, eu), (h, eh) = backward_want(dh.t, g.values(), u.values(), act)
    check_codes(out[0], dg, eg, "dg")
    check_codes(out[1], du, eu, "du")
    for got, want, e, what in zip(out[2:], (dg, du, h), (eg, eu, eh), ("dg^T", "du^T", "h^T")):
        check_codes(got, want.t().contiguous(), e.t().contiguous(), what)
    assert dh.intact() and g.intact() and u.intact()
    for o, t in zip(out, f8.gated_backward(dh.t, g.t, u.t, act, transposed=False)):
        assert torch.equal(t.data.view(torch.uint8), o.codes) and torch.equal(t.scales, o.scales)
