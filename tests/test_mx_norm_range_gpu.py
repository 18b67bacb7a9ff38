"""The norm's statistics: their accuracy, and rows whose squares fp32 does not hold."""
import numpy as np
import pytest
import torch

import attention_residual_fusion_gb300 as ar
from attention_residual_fusion_gb300 import _build, mx
from tests import mx_restatement as R
from tests.test_mx_gpu import F32_HALF, FORMATS, Matrix, Rows, activations, f64

pytestmark = pytest.mark.gpu

# Roundings between a row and y, all of fp32 (half a step is 2^-24): a thread
# adds up at most 8 vectors of 4 pairs (32 roundings, or 34 where a square is
# rounded before it is added), the pair, five steps of a warp and five of its
# CTA (11), then the quotient and eps (2): 47 of terms that are all positive,
# half of that under the root; the root and the last product: 2 more, one for
# the second-order terms.
SLACK = (47 / 2 + 2 + 1) * F32_HALF


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    ar.device_status(clear=True)
    yield
    assert ar.device_status() == 0


def bf16_round(v: np.ndarray) -> np.ndarray:
    """64-bit values to the nearest bf16 values (ties to even, infinity past the largest)."""
    _, e = np.frexp(v)
    step = np.exp2(np.maximum(e, -125).astype(np.float64) - 8)  # of [2^(e-1), 2^e); below 2^-126 2^-133
    r = np.rint(v / step) * step
    return np.where(np.abs(r) >= 2.0 ** 128, np.copysign(np.inf, v), r)


def check(p0, d0, w, eps, fmt, pad=0, g=None):
    """Every output is one that some y within SLACK of the 64-bit one gives."""
    T, H = p0.shape
    eps = float(np.float32(eps))
    p, d, out = Rows(T, H, pad, p0), None if d0 is None else Rows(T, H, pad, d0), Rows(T, H, pad)
    gt = None if g is None else torch.tensor([g], device="cuda")
    q = Matrix(T, H, fmt, 16 if pad else 0, gt)
    mx.add_rms_norm(p.t, None if d is None else d.t, w, eps, fmt, out=q.t, norm_out=out.t)
    torch.cuda.synchronize()
    c = p0 if d0 is None else (p0.float() + d0.float()).bfloat16()
    assert torch.equal(p.t.view(torch.int16), c.contiguous().view(torch.int16))
    assert p.intact() and q.intact() and out.intact() and (d is None or d.intact())
    c64 = f64(c)
    assert np.isfinite(c64).all()
    y = c64 * f64(w) / np.sqrt((c64 ** 2).mean(-1, keepdims=True) + eps)
    o = f64(out.t)
    lo, hi = y - SLACK * np.abs(y), y + SLACK * np.abs(y)
    tiny = 2.0 ** -149  # a y that is no normal number of fp32 is rounded to its steps as well
    lo, hi = np.where(np.abs(y) < 2.0 ** -125, lo - tiny, lo), np.where(np.abs(y) < 2.0 ** -125, hi + tiny, hi)
    assert ((o >= bf16_round(lo)) & (o <= bf16_round(hi))).all()
    data, flat, _ = q.host()
    groups = H // R.GROUP[fmt]
    sc = R.untile(flat, T, groups)
    np.testing.assert_array_equal(R.tile(sc), flat)
    yg = y.reshape(T, groups, -1)
    amax = np.abs(yg).max(-1)
    # a scale of nvfp4 is rounded from a quotient of three more roundings
    more = SLACK + (3 * F32_HALF if fmt == "nvfp4" else 0)
    assert (sc >= R.scale_codes(amax * (1 - more), fmt, g)).all()
    assert (sc <= R.scale_codes(amax * (1 + more), fmt, g)).all()
    s = (R.scales(flat, T, groups, fmt) * (1 if g is None else float(np.float32(g))))[..., None]
    e = R.elements(data, fmt).reshape(yg.shape)
    table = R.E4M3 if fmt == "mxfp8" else R.E2M1
    with np.errstate(all="ignore"):
        v = np.where(s == 0, 0, np.abs(yg) / s)
    edge = np.where(np.abs(yg) < 2.0 ** -125, tiny / np.where(s == 0, 1, s), 0)
    a = table[R.nearest_code(np.maximum(v * (1 - more) - edge, 0), table)]
    b = table[R.nearest_code(v * (1 + more) + edge, table)]
    assert ((np.abs(e) >= a) & (np.abs(e) <= b)).all()
    assert ((e == 0) | (np.sign(e) == np.sign(yg))).all()


def weight(H, seed):
    return (1 + 0.1 * torch.randn(H, generator=torch.Generator().manual_seed(seed))).bfloat16().cuda()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,H", [(3, 96), (65, 2048), (40, 7168), (17, 16384), (4, 65536), (1024, 256), (1025, 512),
                                 (1030, 1024), (1027, 2048), (1024, 4096), (1024, 7168)])
def test_statistics_are_accurate(fmt, T, H):
    """Every launch shape, a bound that a mean or root of fewer bits does not keep."""
    check(activations(T, H, 100), activations(T, H, 101), weight(H, 1), 1e-6, fmt, 8 if T % 2 else 0,
          0.004 if fmt == "nvfp4" else None)


ENDS = [(1e17, 1e-6), (3e18, 1e-6), (1e25, 0.0), (1e30, 3e38), (1e36, 1e-6), (1e-12, 0.0), (1e-16, 0.0),
        (1e-20, 0.0), (1e-23, 1e-45), (1e-30, 1e-38), (1e-30, 1e-33), (1e-37, 0.0), (1e-39, 1e-42), (1.0, 3e38),
        (5e18, 3.4e38), (1e-5, 3.4e38)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("scale,eps", ENDS)
def test_rows_at_both_ends_of_the_range(fmt, scale, eps):
    """Large rows, whose squares overflow, and small ones, whose squares are none or have lost bits."""
    for T, H in ((5, 7168), (1026, 512)):
        p, d = activations(T, H, 110, scale), activations(T, H, 111, scale / 3)
        w = weight(H, 2)
        if eps == 0.0:  # no row of zeros, of which the formula makes NaN
            p[:, 0] = torch.tensor(scale, device="cuda").bfloat16()
            p[:, 0] = torch.maximum(p[:, 0], torch.tensor(2.0 ** -133, device="cuda").bfloat16())
            d[:, 0] = 0
        check(p, d, w, eps, fmt)
        check((p.float() + d.float()).bfloat16(), None, w, eps, fmt, 8)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,H", [(6, 32), (9, 1120), (40, 4128), (8, 20000 // 32 * 32), (3, 65536), (1040, 288),
                                 (1030, 992), (1025, 2080), (1024, 8224)])
def test_every_shape_with_rows_of_all_sizes(fmt, T, H):
    """Rows of all magnitudes beside each other: each on its own."""
    e = torch.linspace(-125, 115, T, device="cuda")[torch.randperm(T, generator=torch.Generator().manual_seed(3))]
    p = (activations(T, H, 120).double() * torch.exp2(e.double().round())[:, None]).clamp(-1e38, 1e38).bfloat16()
    d = (p.double() * 0.25).bfloat16()
    p[:, 1] = torch.where(p[:, 1] == 0, torch.tensor(2.0 ** -133, device="cuda").bfloat16(), p[:, 1])
    check(p, d, weight(H, 4), 0.0, fmt)


def test_a_single_value_is_the_whole_row():
    """One value among zeros, of every exponent: y = +-sqrt(H), whatever it is."""
    H = 64
    v = torch.cat([2.0 ** torch.arange(-133, 128, dtype=torch.float64),
                   -1.5 * 2.0 ** torch.arange(-132, 127, dtype=torch.float64)]).bfloat16().cuda()
    p = torch.zeros(v.numel(), H, dtype=torch.bfloat16, device="cuda")
    p[:, 37] = v
    out = torch.empty_like(p)
    q = mx.add_rms_norm(p, None, torch.ones(H, dtype=torch.bfloat16, device="cuda"), 0.0, norm_out=out)
    want = torch.zeros_like(p)
    want[:, 37] = torch.sign(v.float()).bfloat16() * 8
    assert torch.equal(out, want) and torch.equal(mx.dequantize(q), want)


@pytest.mark.parametrize("T", [4, 1100])
def test_zeros_infinities_and_nan_stay(T):
    """With eps = 0 a row of zeros is NaN, by the formula; a NaN or an infinity takes its row."""
    p = activations(T, 352, 5)
    p[0] = 0
    p[1, 3], p[1, 200] = float("inf"), 3.3e38
    p[2, 300] = float("nan")
    w = torch.full((352,), 1.5, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(p)
    q = mx.add_rms_norm(p, None, w, 0.0, norm_out=out)
    o, v = f64(out), f64(mx.dequantize(q))
    assert np.isnan(o[0]).all() and np.isnan(v[0]).all()
    assert np.isnan(o[1, 3]) and (o[1][np.arange(352) != 3] == 0).all()
    assert np.isnan(v[1, :32]).all() and (v[1, 32:] == 0).all()
    assert np.isnan(o[2]).all() and np.isnan(v[2]).all()
    assert np.isfinite(o[3:]).all() and np.isfinite(v[3:]).all()
    out0 = torch.empty_like(p)
    q0 = mx.add_rms_norm(p[:1].contiguous(), None, w, 1e-40, norm_out=out0[:1])
    assert not out0[:1].any() and not q0.data.view(torch.uint8).any()
