"""The 8-bit feed-forward operators on the GPU against the format restated in 64
bits (tests/f8_restatement.py)."""
import numpy as np
import pytest
import torch

import attention_residual_fusion_gb300 as ar
from attention_residual_fusion_gb300 import _build, f8
from tests import f8_restatement as R
from tests.test_mx_gpu import Guarded, Rows, activations

pytestmark = pytest.mark.gpu

BF16_HALF = 2.0 ** -8  # half a step relative to the value, at most
F32_HALF = 2.0 ** -24
# The fast exponential's documented error is 2 + floor(1.173 |x|) units of 2^-23:
# 105 at |x| = 88, with the reciprocal's and the sum's one each below 2^-16; a
# quotient of less than 2^-126 is off by 2^-149 more, or 0 from 2^-128 on
# (times |g| up to 100 below 2^-119).
ACT = 2.0 ** -16
ACT_LEAST = 2.0 ** -119


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    ar.lib()
    ar.device_status(clear=True)
    yield
    assert ar.device_status() == 0


class Matrix:
    """An F8Tensor in guarded buffers, rows of codes and of scales padded."""

    def __init__(self, rows, cols, block=1, pad=0):
        self.rows, self.cols, self.block = rows, cols, block
        self.row_bytes = -(-cols // 16) * 16 + 16 * pad
        sr, sc = R.scales_shape(rows, cols, block)
        self.scales_row = -(-sc // 4) * 4 + 4 * pad
        self.gd = Guarded(rows * self.row_bytes)
        self.gs = Guarded(sr * self.scales_row * 4)
        self.full = self.gd.view.view(rows, self.row_bytes)
        self.full_s = self.gs.view.view(torch.float32).view(sr, self.scales_row)
        self.codes = self.full[:, :cols]
        self.scales = self.full_s[:, :sc]
        self.t = f8.F8Tensor(self.codes.view(torch.float8_e4m3fn), self.scales, block)

    def set(self, codes, scales):
        self.codes.copy_(codes)
        self.scales.copy_(scales)
        return self

    def values(self):
        return R.values(self.codes.contiguous(), self.scales.contiguous(), self.block)

    def scale_of(self):
        """[rows, cols] fp64: each element's scale."""
        idx = R.group_index(self.rows, self.cols, self.block, "cuda")
        return self.scales.contiguous().double().view(-1)[idx]

    def intact(self):
        pad = self.full_s[:, self.scales.shape[1]:].contiguous().view(torch.uint8)
        return (self.gd.intact() and self.gs.intact() and bool((self.full[:, self.cols:] == 0x5A).all())
                and bool((pad == 0x5A).all()))


def quantized(rows, cols, seed, block=1, pad=0, scale=1.0):
    return Matrix(rows, cols, block, pad).set(*R.quantize(activations(rows, cols, seed, scale), block))


def equal_with_nan(a, b):
    return bool(torch.equal(torch.isnan(a), torch.isnan(b))) and bool(torch.equal(torch.nan_to_num(a, nan=7.0),
                                                                              torch.nan_to_num(b, nan=7.0)))


def within(got, want, bound, what=""):
    got, err = got.double(), (got.double() - want).abs()
    bad = ~(err <= bound)  # (a NaN is outside)
    if bool(bad.any()):
        i = int((err / bound.clamp(min=1e-300)).nan_to_num(nan=1e300).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; worst at {i}: got "
                             f"{got.view(-1)[i].item()!r} want {want.view(-1)[i].item()!r} bound {bound.view(-1)[i].item()!r}")


# ---- quantisation -------------------------------------------------------------------


def special(rows, cols, seed):
    """Values at which quantisation can go wrong, here and there."""
    x = activations(rows, cols, seed)
    flat = x.view(-1)
    for i, v in enumerate([0.0, -0.0, 2.0 ** -133, 2.0 ** -126, 3.3e38, -3.3e38, float("inf"), float("-inf"),
                           float("nan"), 448.0, 1e-30, 1e30, 2.0 ** -120, 7.0]):
        flat[(i * 397) % flat.numel()] = v
    if rows > 3:
        x[1] = 0.0
        x[2] = -0.0
        x[3] *= 2.0 ** -126
    if cols > 130:
        x[:, 5] = 0.0
        x[:, 129] *= 2.0 ** 90
    return x


SHAPES = [(1, 1, 0), (1, 8, 0), (1, 7168, 0), (2, 96, 8), (3, 127, 0), (16, 128, 0), (17, 129, 8), (33, 2048, 16),
          (127, 290, 0), (128, 256, 0), (129, 1030, 64), (300, 64, 0), (257, 1120, 8), (1003, 520, 0)]


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("rows,cols,pad", SHAPES)
def test_quantize(rows, cols, pad, transposed, block):
    """Codes and scales bit for bit, and nothing beside them."""
    for make in (activations, special):
        x = Rows(rows, cols, pad, make(rows, cols, rows + cols))
        q, t = Matrix(rows, cols, block, pad // 8), Matrix(cols, rows, block, pad // 8)
        f8.quantize(x.t, block, q.t, transposed=t.t if transposed else None)
        codes, scales = R.quantize(x.t, block)
        assert equal_with_nan(q.scales, scales)
        assert torch.equal(q.codes, codes)
        if transposed:
            codes, scales = R.quantize(x.t.t(), block)
            assert equal_with_nan(t.scales, scales)
            assert torch.equal(t.codes, codes)
        else:
            assert bool((t.codes == 0x5A).all())
        assert x.intact() and q.intact() and t.intact()


def test_quantize_every_bf16_pattern():
    """All numbers, in rows of one magnitude class each, and every quotient's rounding."""
    bits = torch.arange(1 << 16, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16)
    x = bits.view(512, 128).contiguous()  # neighbours share the exponent: 128 mantissas of one sign
    mixed = bits.view(128, 512).t().contiguous()
    for v in (x, mixed):
        q = f8.quantize(v)
        codes, scales = R.quantize(v, 1)
        assert equal_with_nan(q.scales, scales)
        assert torch.equal(q.data.view(torch.uint8), codes)


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("rows,cols,pad", SHAPES)
def test_dequantize(rows, cols, pad, block):
    codes, scales = R.quantize(special(rows, cols, 3), block)
    q = Matrix(rows, cols, block, pad // 8).set(codes, scales)
    x = Rows(rows, cols, pad)
    f8.dequantize(q.t, x.t)
    want = q.values().to(torch.float32).to(torch.bfloat16)  # (code * s is exact to fp32's rounding)
    assert equal_with_nan(x.t, want)
    assert x.intact() and q.intact()


# ---- products -------------------------------------------------------------------------

# (m, n, k): one token to many, ragged in each direction, several tiles each way
PRODUCTS = [(1, 1, 1), (1, 128, 128), (1, 300, 100), (3, 257, 640), (16, 130, 1000), (33, 512, 256), (64, 1000, 2050),
            (65, 128, 4096), (100, 700, 129), (128, 256, 127), (200, 640, 3000), (256, 256, 512), (257, 513, 384),
            (300, 1030, 777), (1000, 520, 1111), (600, 4000, 260)]


def product_want(pairs, cols):
    want = sum(a.values() @ w.values().t() for a, w in pairs)
    mag = sum(a.values().abs() @ w.values().abs().t() for a, w in pairs)
    return want, R.product_bound(mag, cols)


# the forms of a product, the narrow one with K split over clusters of several sizes
FORMS = [dict(kernel=f8.KERNEL_WIDE)] + [dict(kernel=f8.KERNEL_NARROW, split=s) for s in (1, 2, 3, 5, 8)] + [dict()]


def form(kw, k):
    """The override as far as K's blocks allow."""
    return {**kw, "split": min(kw["split"], max(1, R.blocks(k)))} if "split" in kw else kw


@pytest.mark.parametrize("kw", FORMS, ids=lambda kw: "-".join(f"{a}{b}" for a, b in kw.items()) or "auto")
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_matmul(m, n, k, block, kw):
    kw = form(kw, k)
    a, w = quantized(m, k, 1), quantized(n, k, 2, block, scale=0.02)
    want, bound = product_want([(a, w)], k)
    out = Rows(m, n, 8)
    f8.matmul(a.t, w.t, out.t, **kw)
    within(out.t, want, bound + BF16_HALF * (want.abs() + bound), "bf16")
    assert out.intact() and a.intact() and w.intact()
    f = f8.matmul(a.t, w.t, dtype=torch.float32, **kw)
    assert f.shape == (m, n) and f.dtype == torch.float32
    within(f, want, bound, "fp32")
    # the same bits again, and bf16 is fp32 rounded
    assert torch.equal(f, f8.matmul(a.t, w.t, dtype=torch.float32, **kw))
    assert torch.equal(out.t, f.to(torch.bfloat16))
    # added to what is there: one more rounding
    g = torch.Generator(device="cuda").manual_seed(5)
    before = torch.randn(m, n, generator=g, device="cuda")
    buf = torch.full((m, -(-n // 4) * 4 + 4), 3.25, device="cuda")
    buf[:, :n] = before
    f8.matmul(a.t, w.t, buf[:, :n], add=True, **kw)
    assert torch.equal(buf[:, :n], before + f)
    assert bool((buf[:, n:] == 3.25).all())


@pytest.mark.parametrize("kw", FORMS, ids=str)
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("m,n,k,k2", [(1, 200, 256, 100), (40, 300, 129, 513), (300, 520, 1000, 128), (513, 256, 1, 2000)])
def test_matmul_of_two_pairs(m, n, k, k2, block, kw):
    kw = form(kw, 128 * (R.blocks(k) + R.blocks(k2)))
    pairs = [(quantized(m, kk, s), quantized(n, kk, s + 1, block, pad=1, scale=0.05)) for kk, s in ((k, 1), (k2, 3))]
    want, bound = product_want(pairs, k + k2 + 128)
    (a, w), (a2, w2) = pairs
    f = f8.matmul(a.t, w.t, dtype=torch.float32, plus=(a2.t, w2.t), **kw)
    within(f, want, bound)
    h = f8.matmul(a.t, w.t, plus=(a2.t, w2.t), **kw)
    assert torch.equal(h, f.to(torch.bfloat16))


@pytest.mark.parametrize("block", [1, 128])
def test_matmul_without_columns(block):
    """A sum over no tokens is zero; behind it a second pair counts alone."""
    for m, n in ((130, 300), (20, 300)):
        without_columns(m, n, block)


def without_columns(m, n, block):
    a, w = f8.F8Tensor.empty(m, 0), f8.F8Tensor.empty(n, 0, block)
    out = torch.full((m, n), 9.0, device="cuda")
    f8.matmul(a, w, out)
    assert bool((out == 0).all())
    out.fill_(9.0)
    f8.matmul(a, w, out, add=True)
    assert bool((out == 9).all())
    a2, w2 = quantized(m, 200, 1), quantized(n, 200, 2, block)
    alone = f8.matmul(a2.t, w2.t)
    assert torch.equal(f8.matmul(a, w, plus=(a2.t, w2.t)), alone)
    assert torch.equal(f8.matmul(a2.t, w2.t, plus=(a, w)), alone)


def test_without_rows():
    a, w = f8.F8Tensor.empty(0, 256), quantized(300, 256, 1, 128)
    assert f8.matmul(a, w.t).shape == (0, 300)
    q, t = f8.quantize(torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"), transposed=True)
    assert q.shape == (0, 256) and t.shape == (256, 0)
    assert f8.dequantize(q).shape == (0, 256)
    h, g, u = f8.gated(a, w.t, w.t, save=True)
    assert h.shape == g.shape == u.shape == (0, 300)
    dg, du, dgt, dut, ht = f8.gated_backward(torch.empty(0, 300, dtype=torch.bfloat16, device="cuda"), g, u)
    assert dg.shape == (0, 300) and ht.shape == (300, 0)
    # and the gradient of a weight matrix that no token reached
    x = f8.F8Tensor.empty(256, 0)
    assert bool((f8.matmul(dgt, x, dtype=torch.float32) == 0).all())


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("ea,ew", [(-126, 0), (-126, 20), (-126, 120), (-60, -60), (-63, -62), (100, -126), (119, -120),
                                   (50, 50), (60, 40), (119, -30)])
def test_matmul_far_scales(ea, ew, block):
    """Scales near the ends of fp32, whose products fp32 holds: a result is out of range only if its value is."""
    for m, n, k in ((3, 200, 300), (300, 257, 260)):
        a, w = quantized(m, k, 1), quantized(n, k, 2, block)
        a.scales.copy_(torch.exp2(torch.full(a.scales.shape, float(ea), dtype=torch.float64, device="cuda")))
        w.scales.copy_(torch.exp2(torch.full(w.scales.shape, float(ew), dtype=torch.float64, device="cuda")))
        a.scales[:, ::2] *= 1.3
        w.scales[0] *= 1.7
        want, bound = product_want([(a, w)], k)
        # (what a sum loses below the smallest normal number: a step of 2^-149 for each block)
        bound = bound + 2.0 ** -149 * (R.blocks(k) + 1)
        f = f8.matmul(a.t, w.t, dtype=torch.float32).double()
        within(f, want, bound)


@pytest.mark.parametrize("block", [1, 128])
def test_matmul_scales_out_of_range(block):
    """Results beyond fp32 are infinite, those far below it 0."""
    for m, n, k in ((3, 200, 300), (300, 257, 260)):
        a, w = quantized(m, k, 1), quantized(n, k, 2, block)
        a.codes &= 0x7F  # no signs: every sum is positive
        w.codes &= 0x7F
        a.codes[:, 0] = w.codes[:, 0] = 0x38  # and not zero
        for e, result in ((70.0, float("inf")), (-110.0, 0.0)):
            a.scales.copy_(torch.exp2(torch.full(a.scales.shape, e, dtype=torch.float64, device="cuda")))
            w.scales.copy_(torch.exp2(torch.full(w.scales.shape, e, dtype=torch.float64, device="cuda")))
            assert bool((f8.matmul(a.t, w.t, dtype=torch.float32) == result).all())


@pytest.mark.parametrize("block", [1, 128])
def test_matmul_nan_and_zero_scales(block):
    """A group that stands for NaN makes the results that it enters NaN and no others; a scale of 0 makes 0."""
    for m, n, k in ((5, 300, 400), (300, 300, 400)):
        a, w = quantized(m, k, 1), quantized(n, k, 2, block)
        a.scales[1, 2] = float("nan")
        w.scales[0, 0] = 0.0
        if block == 1:
            w.scales[2, 7] = float("nan")
            bad_cols = [7]
        else:
            w.scales[1, 3] = float("nan")
            bad_cols = range(128, 256)
        want, _ = product_want([(a, w)], k)
        f = f8.matmul(a.t, w.t, dtype=torch.float32)
        bad = torch.zeros(m, n, dtype=torch.bool, device="cuda")
        bad[2] = True
        bad[:, list(bad_cols)] = True
        assert torch.equal(torch.isnan(f), bad)
        a.scales[1, 2] = 1.0
        w.scales[torch.isnan(w.scales)] = 1.0
        want, bound = product_want([(a, w)], k)
        within(torch.where(bad, 0.0, f.double()), torch.where(bad, 0.0, want), bound.nan_to_num(nan=0.0) + 1e-30)


# ---- the gated block --------------------------------------------------------------------

# (T, F, H)
GATED = [(1, 1, 1), (1, 128, 256), (2, 300, 1000), (17, 130, 129), (64, 512, 2048), (65, 256, 300), (128, 1000, 520),
         (200, 128, 4096), (257, 700, 384), (520, 129, 1111), (1003, 400, 260)]


def gated_want(x, wg, wu, act):
    """h and the bounds of g, u and h."""
    g, u = x.values() @ wg.values().t(), x.values() @ wu.values().t()
    eg = R.product_bound(x.values().abs() @ wg.values().abs().t(), x.cols)
    eu = R.product_bound(x.values().abs() @ wu.values().abs().t(), x.cols)
    a, _ = R.act(g, act)
    ea = 1.13 * eg + a.abs() * ACT + ACT_LEAST  # (|act'| is below 1.13)
    eh = ea * (u.abs() + eu) + a.abs() * eu + (a * u).abs() * F32_HALF
    return g, u, a * u, eg, eu, eh


def check_codes(got, want, error, what):
    within(got.values(), want, R.code_bound(want, error, got.scale_of()), what)
    # the scale is that of the group's largest value
    idx = R.group_index(got.rows, got.cols, 1, "cuda").reshape(-1)
    top = torch.zeros(got.scales.numel(), dtype=torch.float64, device="cuda").scatter_reduce(
        0, idx, want.abs().reshape(-1), "amax")
    slack = torch.zeros_like(top).scatter_reduce(0, idx, error.reshape(-1), "amax")
    s = got.scales.contiguous().double().view(-1)
    within(torch.where(top <= slack, top / 448, s), top / 448, slack / 448 + top * 2.0 ** -24 + 2.0 ** -126, what + " scales")
    assert got.intact()


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("kw", FORMS, ids=str)
@pytest.mark.parametrize("T,F,H", GATED)
def test_gated(T, F, H, act, kw):
    kw = form(kw, H)
    x = quantized(T, H, 1)
    wg, wu = quantized(F, H, 2, 128, scale=H ** -0.5), quantized(F, H, 3, 128, pad=1, scale=H ** -0.5)
    g, u, h, eg, eu, eh = gated_want(x, wg, wu, act)
    out = [Matrix(T, F, 1, i) for i in range(3)]
    f8.gated(x.t, wg.t, wu.t, act, out[0].t, save=(out[1].t, out[2].t), **kw)
    for got, want, e, what in zip(out, (h, g, u), (eh, eg, eu), ("h", "g", "u")):
        check_codes(got, want, e, what)
    # without the checkpoint the same h; in bf16 from the same sums
    again = f8.gated(x.t, wg.t, wu.t, act, **kw)
    assert torch.equal(again.data.view(torch.uint8), out[0].codes) and torch.equal(again.scales, out[0].scales)
    rows = Rows(T, F, 8)
    f8.gated(x.t, wg.t, wu.t, act, rows.t, **kw)
    within(rows.t, h, eh + BF16_HALF * (h.abs() + eh), "bf16")
    assert rows.intact()
    b, sg, su = f8.gated(x.t, wg.t, wu.t, act, dtype=torch.bfloat16, save=True, **kw)
    assert torch.equal(b, rows.t)
    assert torch.equal(sg.data.view(torch.uint8), out[1].codes) and torch.equal(su.scales, out[2].scales)


@pytest.mark.parametrize("kw", FORMS[:3], ids=str)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_of_large_and_special_values(act, kw):
    """Projections far beyond the activation's bend, rows of NaN, rows of zeros."""
    T, F, H = 140, 260, 300
    x = quantized(T, H, 1, scale=30.0)
    x.scales[:, 3] = float("nan")
    x.scales[1, 7] = float("inf")
    x.codes[9] = 0
    x.scales[:, 11] *= 2.0 ** 40
    wg, wu = quantized(F, H, 2, 128), quantized(F, H, 3, 128)
    out = [Matrix(T, F) for _ in range(3)]
    f8.gated(x.t, wg.t, wu.t, act, out[0].t, save=(out[1].t, out[2].t), **kw)
    for o in out:
        assert bool(torch.isnan(o.scales[:, 3]).all()) and bool(torch.isnan(o.scales[:, 7]).all())
        assert bool((o.codes[3] == 0).all())
        assert bool((o.scales[:, 9] == 1).all()) and bool((o.codes[9] & 0x7F == 0).all())
        assert o.intact()
    x.scales[:, 3] = 1.0
    x.scales[1, 7] = 1.0
    g, u, h, eg, eu, eh = gated_want(x, wg, wu, act)
    for got, want, e in zip(out, (h, g, u), (eh, eg, eu)):
        v, s = got.values(), got.scale_of()
        bad = torch.zeros(T, F, dtype=torch.bool, device="cuda")
        bad[[3, 7]] = True
        bound = R.code_bound(want, e, s)
        within(torch.where(bad, 0.0, v), torch.where(bad, 0.0, want), torch.where(bad, 1.0, bound))


# ---- its backward pass --------------------------------------------------------------------


def backward_want(dh, g, u, act):
    a, da = R.act(g, act)
    dz = 1.0 if act == "silu" else 1.6 * (1 + 0.135 * g * g)
    # slope p + g p (1 - p) z': p is off by ACT of itself, 1 - p by as much of p, at most 2^-20 where p is not small
    # (then |z| is), and so is what |g| z' multiplies
    gc = g.abs().clamp(max=100.0)
    p = torch.sigmoid(g if act == "silu" else 1.6 * (g + 0.044715 * g ** 3))
    eda = 2 * ACT * p * (1 + gc * dz * (1 - p)) + 2.0 ** -20 * p * gc * dz + ACT_LEAST
    ea = ACT * a.abs() + ACT_LEAST
    d = dh.double()
    return ((d * u * da, (d * u).abs() * eda + (d * u * da).abs() * 2.0 ** -22),
            (d * a, d.abs() * ea + (d * a).abs() * 2.0 ** -22),
            (a * u, ea * u.abs() + (a * u).abs() * 2.0 ** -22))


BACKWARD = [(1, 1, 0), (1, 128, 0), (3, 300, 8), (16, 130, 0), (64, 512, 8), (127, 1000, 0), (129, 128, 16), (300, 260, 8),
            (520, 129, 0)]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T,F,pad", BACKWARD)
def test_gated_backward(T, F, pad, act):
    dh = Rows(T, F, pad, activations(T, F, 1, 1e-3))
    g, u = quantized(T, F, 2, pad=pad // 8, scale=2.0), quantized(T, F, 3)
    out = [Matrix(T, F, 1, 1), Matrix(T, F)] + [Matrix(F, T, 1, i) for i in range(3)]
    f8.gated_backward(dh.t, g.t, u.t, act, [o.t for o in out])
    (dg, eg), (du, eu), (h, eh) = backward_want(dh.t, g.values(), u.values(), act)
    check_codes(out[0], dg, eg, "dg")
    check_codes(out[1], du, eu, "du")
    for got, want, e, what in zip(out[2:], (dg, du, h), (eg, eu, eh), ("dg^T", "du^T", "h^T")):
        check_codes(got, want.t().contiguous(), e.t().contiguous(), what)
    assert dh.intact() and g.intact() and u.intact()
    # by rows alone, the same
    two = f8.gated_backward(dh.t, g.t, u.t, act, transposed=False)
    assert len(two) == 2
    for o, t in zip(out, two):
        assert torch.equal(t.data.view(torch.uint8), o.codes) and torch.equal(t.scales, o.scales)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_backward_against_differences(act):
    """dg and du are the differences of sum(dh * act(g) * u), in 64 bits, to their rounding."""
    T, F, step = 37, 150, 1e-5
    dh = Rows(T, F, 0, activations(T, F, 1, 0.1)).t
    g, u = quantized(T, F, 2, scale=0.5), quantized(T, F, 3)
    dg, du = f8.gated_backward(dh, g.t, u.t, act, transposed=False)
    gv, uv, d = g.values(), u.values(), dh.double()

    def loss(gv, uv):  # element by element: every sum is of one term
        return d * R.act(gv, act)[0] * uv

    for got, diff in ((dg, (loss(gv + step, uv) - loss(gv - step, uv)) / (2 * step)),
                      (du, (loss(gv, uv + step) - loss(gv, uv - step)) / (2 * step))):
        v = R.values(got.data, got.scales, 1)
        s = got.scales.double().contiguous().view(-1)[R.group_index(T, F, 1, "cuda")]
        # a central difference: step^2 / 6 times a third derivative below 4 |dh u|, and 2^-52 of the losses over the step
        e = (d * uv).abs() * (4 * step ** 2 / 6 + 40 * ACT) + d.abs() * ACT * gv.abs() + \
            2.0 ** -50 * loss(gv, uv).abs() / step
        within(v, diff, R.code_bound(diff, e, s))


def test_gated_backward_of_special_values():
    """Saturated gates have slopes of 1 and 0; a NaN stays in its groups."""
    T, F = 130, 256
    dh = activations(T, F, 1)
    g, u = quantized(T, F, 2), quantized(T, F, 3)
    g.codes[0] = 0x7E   # 448
    g.codes[1] = 0xFE   # -448
    g.scales[:, :2] = 1e30
    g.scales[1, 5] = float("nan")
    dh[20, 40] = float("inf")
    dh[21] = 0.0
    for act in ("silu", "gelu"):
        dg, du, dgt, dut, ht = f8.gated_backward(dh, g.t, u.t, act)
        val = lambda t: R.values(t.data, t.scales, 1)  # noqa: E731
        want = dh[0].double() * u.values()[0]
        s = dg.scales.double()[:, 0].repeat_interleave(128)
        within(val(dg)[0], want, R.code_bound(want, want.abs() * 2.0 ** -22, s))
        assert bool((val(dg)[1] == 0).all()) and bool((val(du)[1] == 0).all())
        assert bool(torch.isnan(dg.scales[1, 5])) and bool(torch.isnan(dg.scales[0, 20]))
        assert not bool(torch.isnan(dg.scales[0, 5])) and not bool(torch.isnan(dg.scales[1, 20]))
        assert bool((dg.scales[:, 21] == 1).all())
        # transposed: the first block of tokens of the columns 128.. and of column 40
        bad = torch.zeros(F, dtype=torch.bool, device="cuda")
        bad[128:] = True
        bad[40] = True
        assert torch.equal(torch.isnan(dgt.scales[0]), bad) and not bool(torch.isnan(dgt.scales[1]).any())


# ---- together ---------------------------------------------------------------------------


@pytest.mark.parametrize("T,H,F,N", [(1, 256, 128, 256), (130, 264, 200, 264), (300, 520, 384, 300)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_a_training_step(T, H, F, N, act):
    """Forward and backward through the block, against the same steps in 64 bits from the quantised values."""
    x = Rows(T, H, 0, activations(T, H, 1)).t
    wg, wu, wd = (Rows(r, c, 0, activations(r, c, 2 + i, c ** -0.5)).t for i, (r, c) in enumerate(((F, H), (F, H), (N, F))))
    dy = Rows(T, N, 0, activations(T, N, 9, 1e-2)).t
    xq, xt = f8.quantize(x, transposed=True)
    (gate, gate_t), (up, up_t), (down, down_t) = (f8.quantize(w, 128, transposed=True) for w in (wg, wu, wd))
    val = lambda t: R.values(t.data, t.scales.contiguous(), t.block)  # noqa: E731
    # block scales: the transposed matrix has the same values
    assert torch.equal(val(gate), val(gate_t).t()) and torch.equal(val(down), val(down_t).t())
    h, g, u = f8.gated(xq, gate, up, act, save=True)
    y = f8.matmul(h, down)
    dyq, dyt = f8.quantize(dy, transposed=True)
    dh = f8.matmul(dyq, down_t)
    dg, du, dgt, dut, ht = f8.gated_backward(dh, g, u, act)
    dx = f8.matmul(dg, gate_t, plus=(du, up_t))
    grads = [f8.matmul(p, q, dtype=torch.float32) for p, q in ((dgt, xt), (dut, xt), (dyt, ht))]

    def close(got, parts, cols, half):
        want = sum(val(p) @ val(q).t() for p, q in parts)
        e = R.product_bound(sum(val(p).abs() @ val(q).abs().t() for p, q in parts), cols)
        # a product of scales below 2^-126 (a single token's gradient through a closed gate) is a multiple of 2^-149:
        # off by half of that, times the codes' products, and so is the sum
        e = e + 2.0 ** -150 * (1 + sum(p.data.double().abs() @ q.data.double().abs().t() for p, q in parts))
        within(got, want, e + half * (want.abs() + e))

    close(y, [(h, down)], F, BF16_HALF)
    close(dh, [(dyq, down_t)], N, BF16_HALF)
    close(dx, [(dg, gate_t), (du, up_t)], 2 * F + 256, BF16_HALF)
    for got, (p, q) in zip(grads, ((dgt, xt), (dut, xt), (dyt, ht))):
        close(got, [(p, q)], T, F32_HALF)
    # and the whole step is the step of the unquantised block to what 8 bits hold: in the 2-norm each rounding to
    # codes takes at most 2^-4 (in every value), and a path has at most six of them on the way
    xd, gd, ud, dd, dyd = (t.double() for t in (x, wg, wu, wd, dy))
    a, da = R.act(xd @ gd.t(), act)
    hh, dhh = a * (xd @ ud.t()), dyd @ dd
    want_y = hh @ dd.t()
    want_dd = dyd.t() @ hh
    for got, want in ((y, want_y), (grads[2], want_dd)):
        assert (got.double() - want).norm() <= 6 * 2.0 ** -4 * want.norm()
