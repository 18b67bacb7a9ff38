"""The microscaled operators on the GPU against the formats restated in numpy
(tests/mx_restatement.py) and 64-bit products."""
import numpy as np
import pytest
import torch

import attention_residual_fusion_gb300 as ar
from attention_residual_fusion_gb300 import _build, mx
from tests import mx_restatement as R

pytestmark = pytest.mark.gpu

FORMATS = R.FORMATS
BF16_HALF = 2.0 ** -8  # half a bf16 step, relative to the value, at most
F32_HALF = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    ar.lib()
    ar.device_status(clear=True)
    yield
    assert ar.device_status() == 0


class Guarded:
    """A device byte buffer inside a larger one of canaries that come back untouched."""
    PAD = 4096
    CANARY = 0xA5

    def __init__(self, nbytes: int, fill: int = 0x5A):
        self.buf = torch.full((nbytes + 2 * self.PAD,), self.CANARY, dtype=torch.uint8, device="cuda")
        self.view = self.buf[self.PAD:self.PAD + nbytes]
        self.view.fill_(fill)

    def intact(self) -> bool:
        b = self.buf.cpu().numpy()
        return bool((b[:self.PAD] == self.CANARY).all() and (b[-self.PAD:] == self.CANARY).all())


class Matrix:
    """An MxTensor in guarded buffers, rows row_bytes apart."""

    def __init__(self, rows, cols, fmt, pad=0, g=None):
        used = cols if fmt == "mxfp8" else cols // 2
        self.rows, self.cols, self.fmt, self.used = rows, cols, fmt, used
        self.row_bytes = -(-used // 16) * 16 + pad
        self.gd = Guarded(rows * self.row_bytes)
        shape = mx.scales_shape(fmt, rows, cols)
        self.gs = Guarded(int(np.prod(shape)))
        data = self.gd.view.view(rows, self.row_bytes)[:, :used]
        sdt = torch.float8_e4m3fn if fmt == "nvfp4" else torch.float8_e8m0fnu
        self.t = mx.MxTensor(data.view(torch.float8_e4m3fn) if fmt == "mxfp8" else data,
                             self.gs.view.view(sdt).view(shape), fmt, g)

    def set(self, data: np.ndarray, flat: np.ndarray):
        self.gd.view.view(self.rows, self.row_bytes)[:, :self.used] = torch.from_numpy(data).cuda()
        self.gs.view.copy_(torch.from_numpy(flat))
        return self

    def host(self):
        full = self.gd.view.cpu().numpy().reshape(self.rows, self.row_bytes)
        return full[:, :self.used], self.gs.view.cpu().numpy(), full[:, self.used:]

    def intact(self):
        return self.gd.intact() and self.gs.intact() and (self.host()[2] == 0x5A).all()


class Rows:
    """bf16 rows in a guarded buffer."""

    def __init__(self, rows, cols, pad=0, x=None):
        self.row = -(-cols // 8) * 8 + pad
        self.g = Guarded(rows * self.row * 2)
        self.full = self.g.view.view(torch.bfloat16).view(rows, self.row)
        self.t = self.full[:, :cols]
        if x is not None:
            self.t.copy_(x)

    def intact(self):
        pad = self.full[:, self.t.shape[1]:].contiguous().view(torch.uint8)
        return self.g.intact() and bool((pad == 0x5A).all())


def f64(t) -> np.ndarray:
    return t.double().cpu().numpy()


def activations(rows, cols, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, cols, generator=g, device="cuda") * scale
    x *= 1 + 49 * (torch.rand(rows, cols, generator=g, device="cuda") < 0.01)
    return x.bfloat16()


def special(rows, cols, seed):
    """Rows with the values at which quantisation can go wrong, group by group."""
    x = activations(rows, cols, seed)
    flat = x.view(-1)
    n = flat.numel() // 32
    bits = torch.arange(1 << 16, device="cuda", dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    for i, v in enumerate([0.0, -0.0, 2.0 ** -133, 2.0 ** -126, 3.3e38, -3.3e38, float("inf"),
                           float("-inf"), float("nan"), 448.0, 450.0, 6.0, 6.03125, 0.25, 1e-30]):
        if i < n:
            flat[32 * i:32 * i + 32] *= 0 if i < 3 or i > 10 else 1
            flat[32 * i + (7 * i) % 32] = v
    k = min(flat.numel() - 32 * 16, 1 << 16)
    if k > 0:  # every bf16 pattern that is a number below 8, as far as there is room
        some = bits[torch.isfinite(bits) & (bits.abs() < 8)][:k]
        flat[32 * 16:32 * 16 + some.numel()] = some
    return x


SHAPES = [(1, 32, 0), (1, 7168, 0), (2, 96, 8), (31, 160, 0), (33, 2048, 16), (127, 288, 0), (128, 256, 0),
          (129, 4128, 64), (300, 64, 0), (257, 1120, 8)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,cols,pad", SHAPES)
def test_quantize(fmt, rows, cols, pad):
    """Codes and scales bit for bit, the zero entries behind included."""
    for seed, make in ((1, activations), (2, special)):
        x = Rows(rows, cols, pad, make(rows, cols, seed))
        g = None if fmt != "nvfp4" or seed == 2 else torch.tensor([0.0123], device="cuda")
        q = Matrix(rows, cols, fmt, 16 if pad else 0, g)
        mx.quantize(x.t, fmt, out=q.t)
        want = R.quantize(f64(x.t), fmt, None if g is None else g.item())
        data, flat, _ = q.host()
        np.testing.assert_array_equal(flat, want[1])
        np.testing.assert_array_equal(data, want[0])
        assert x.intact() and q.intact()


@pytest.mark.parametrize("g,top", [(1.0, 2688), (0.0123, 30), (3.7e-5, 0.1), (911.0, 2e6), (1e-31, 2.6e-28),
                                   (1e-37, 1e-34), (1e-41, 1e-38), (1e33, 1e37), (1.0, 1e37), (1e-31, 1e37),
                                   (1e-40, 3e38), (0.5, 1e-30), (1e30, 1.0)])
def test_quantize_nvfp4_quotients(g, top):
    """Elements and scales are the correctly rounded fp32 quotients' codes, for
    tensor scales from the smallest to the largest, fitting the values or not
    (torch divides in IEEE)."""
    x = (activations(256, 4096, 6).double() * top / 150).clamp(-3e38, 3e38).bfloat16()
    gt = torch.tensor([g], device="cuda")
    q = mx.quantize(x, "nvfp4", gt)
    xg = x.float().view(256, 256, 16)
    s = (xg.abs().amax(-1) / (6.0 * gt)).clamp(max=448.0).to(torch.float8_e4m3fn)
    got = q.scales.view(torch.uint8).permute(0, 3, 2, 1, 4).reshape(256, 256)
    assert torch.equal(got, s.view(torch.uint8))
    d = s.float()[..., None] * gt
    v = torch.where(d > 0, xg / d, torch.zeros_like(xg)).view(256, 4096)
    a = v.abs().clamp(max=6.0).double()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    n = torch.round(a / step) * step
    code = torch.where(n <= 2, 2 * n, torch.where(n <= 4, n + 2, 7.0)).to(torch.uint8)
    code |= torch.signbit(v).to(torch.uint8) << 3
    assert torch.equal(q.data, code[:, ::2] | (code[:, 1::2] << 4))


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantize_allocates(fmt):
    x = activations(70, 416, 3)
    q = mx.quantize(x, fmt)
    want = R.quantize(f64(x), fmt)
    np.testing.assert_array_equal(q.data.view(torch.uint8).cpu().numpy(), want[0])
    np.testing.assert_array_equal(q.scales.view(torch.uint8).cpu().numpy().reshape(-1), want[1])
    assert q.shape == (70, 416)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("g", [None, 0.37])
def test_dequantize_every_code(fmt, g):
    """All element codes under all scale codes, bit for bit."""
    if g is not None and fmt != "nvfp4":
        pytest.skip("only nvfp4 has a tensor scale")
    group, codes = R.GROUP[fmt], 256 if fmt == "mxfp8" else 16
    per = -(-codes // group)  # groups that hold every element code once
    rows, cols = 256, max(32, per * group)
    elem = np.tile(np.arange(cols) % codes, (rows, 1)).astype(np.uint8)
    sc = np.repeat(np.arange(256)[:, None], cols // group, axis=1).astype(np.uint8)
    gt = None if g is None else torch.tensor([g], device="cuda")
    q = Matrix(rows, cols, fmt, 16, gt).set(R.pack(elem, fmt), R.tile(sc))
    out = Rows(rows, cols, 8)
    mx.dequantize(q.t, out.t)
    e = R.elements(R.pack(elem, fmt), fmt).astype(np.float32)
    s = np.repeat(R.scales(R.tile(sc), rows, cols // group, fmt), group, axis=1).astype(np.float32)
    with np.errstate(all="ignore"):
        v = e * s
        if g is not None:
            v = v * np.float32(g)
    want = torch.from_numpy(v).to(torch.bfloat16)
    got = out.t.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    fine = ~torch.isnan(want)
    assert torch.equal(got[fine], want[fine])
    assert out.intact() and q.intact()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,cols,pad", [(1, 32, 0), (3, 7168, 0), (129, 2080, 8), (300, 96, 0)])
def test_round_trip(fmt, rows, cols, pad):
    """Quantised and back, within half an element step and the bf16 rounding."""
    x = Rows(rows, cols, pad, activations(rows, cols, 5))
    q = mx.quantize(x.t, fmt)
    y = f64(mx.dequantize(q))
    v = f64(x.t)
    s = np.repeat(R.scales(q.scales.view(torch.uint8).cpu().numpy().reshape(-1), rows, cols // R.GROUP[fmt], fmt),
                  R.GROUP[fmt], axis=1)
    rel, least = (2.0 ** -4, 2.0 ** -10) if fmt == "mxfp8" else (0.25, 0.25)
    # e4m3: half a step is 2^-4 of the value, 2^-10 below its normal numbers;
    # e2m1: half the largest step is 1 of 4..6, at most a quarter of the value
    tol = np.maximum(rel * np.abs(v), least * s) + BF16_HALF * np.abs(v)
    if fmt == "nvfp4":
        # the group scale is rounded, by at most 2^-4 of it: the largest may be clipped by that
        tol += 2.0 ** -4 * np.abs(v) + 2.0 ** -9 * 6
    assert (np.abs(y - v) <= tol * (1 + 1e-12)).all()


# ---- residual + RMSNorm -------------------------------------------------------------


def check_norm(T, H, fmt, delta, pad, norm_out, seed, scale=1.0, eps=1e-6, g=None, edit=None, **kw):
    p0 = activations(T, H, seed, scale)
    d0 = activations(T, H, seed + 1, scale) if delta else None
    if edit is not None:
        edit(p0, d0)
    w = (1 + 0.1 * torch.randn(H, generator=torch.Generator().manual_seed(seed))).bfloat16().cuda()
    p, d = Rows(T, H, pad, p0), Rows(T, H, pad + 8 if pad else 0, d0) if delta else None
    out = Rows(T, H, pad) if norm_out else None
    gt = None if g is None else torch.tensor([g], device="cuda")
    q = Matrix(T, H, fmt, 16 if pad else 0, gt)
    mx.add_rms_norm(p.t, d.t if delta else None, w, eps, fmt, out=q.t, norm_out=out.t if norm_out else None, **kw)
    torch.cuda.synchronize()
    c = p0 if d0 is None else (p0.float() + d0.float()).bfloat16()
    assert torch.equal(p.t.view(torch.int16), c.contiguous().view(torch.int16))
    assert p.intact() and q.intact() and (d is None or d.intact()) and (out is None or out.intact())
    if delta:
        assert torch.equal(d.t.view(torch.int16), d0.view(torch.int16))
    c64 = f64(c)
    with np.errstate(all="ignore"):
        y = c64 / np.sqrt((c64 ** 2).mean(-1, keepdims=True) + eps) * f64(w)
    # fp32: the products c w are exact; the sum of H squares (every partial
    # sum of positive terms at most H roundings, half of that under the root),
    # mean, root and the final product add a few half steps
    slack = (H / 2 + 8) * F32_HALF
    fine = np.isfinite(y)
    if out is not None:
        o = f64(out.t)
        assert (np.isfinite(o) == fine).all()
        assert (np.abs(o - y)[fine] <= ((BF16_HALF + 2 * slack) * np.abs(y))[fine] + 2.0 ** -134).all()
    data, flat, _ = q.host()
    groups = H // R.GROUP[fmt]
    sc = R.untile(flat, T, groups)
    np.testing.assert_array_equal(R.tile(sc), flat)  # zero entries behind
    yg = y.reshape(T, groups, -1)
    amax = np.abs(yg).max(-1)
    bad = ~np.isfinite(yg).all(-1)
    nan_code = 127 if fmt == "nvfp4" else 255
    assert ((sc == nan_code) == bad).all()
    lo = R.scale_codes(np.where(bad, 1.0, amax * (1 - slack)), fmt, g)
    hi = R.scale_codes(np.where(bad, 1.0, amax * (1 + slack)), fmt, g)
    assert ((sc >= lo) & (sc <= hi) | bad).all()
    # every element is one of the nearest to a value within the slack of y
    s = (R.scales(flat, T, groups, fmt) * (1 if g is None else float(np.float32(g))))[..., None]
    e = R.elements(data, fmt).reshape(yg.shape)
    table = R.E4M3 if fmt == "mxfp8" else R.E2M1
    with np.errstate(all="ignore"):
        v = np.abs(yg) / s
        a = table[R.nearest_code(np.where(bad[..., None] | (s == 0), 0, v * (1 - 2 * slack)), table)]
        b = table[R.nearest_code(np.where(bad[..., None] | (s == 0), 0, v * (1 + 2 * slack)), table)]
    assert ((np.abs(e) >= a) & (np.abs(e) <= b)).all()
    assert (e[bad] == 0).all()
    assert ((e == 0) | (np.sign(e) == np.sign(yg)))[~bad].all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,H,pad", [(1, 32, 0), (1, 7168, 0), (5, 2080, 8), (128, 256, 0), (130, 96, 16),
                                     (33, 4128, 0), (7, 16384, 8), (2, 65536, 0), (257, 1120, 0)])
def test_norm(fmt, T, H, pad):
    g = 0.004 if fmt == "nvfp4" else None
    check_norm(T, H, fmt, True, pad, True, 11, g=g)
    check_norm(T, H, fmt, False, pad, False, 12)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,H", [(1024, 32), (1025, 288), (1100, 512), (1033, 992), (1151, 1056), (1030, 2048),
                                 (1027, 2080), (1024, 4096), (1026, 4128), (1025, 7168), (1024, 8224)])
def test_norm_of_many_rows(fmt, T, H):
    """The shapes for many rows, a warp a row among them."""
    check_norm(T, H, fmt, True, 8 if T % 2 else 0, bool(T % 3), 15, g=0.004 if fmt == "nvfp4" else None)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("scale,eps", [(1e-3, 1e-6), (1e-3, 0.0), (100.0, 1e-5), (1e-15, 1e-6)])
def test_norm_scales(fmt, scale, eps):
    check_norm(9, 512, fmt, True, 0, True, 13, scale, eps)


@pytest.mark.parametrize("fmt", FORMATS)
def test_norm_of_zero_and_nonfinite_rows(fmt):
    """A zero row stays zero with eps > 0; a NaN or an infinity takes its row
    (all of it: the statistics) and no other."""
    p = activations(4, 352, 3)
    p[1, 5] = float("nan")
    p[2] = 0
    w = torch.ones(352, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(p)
    q = mx.add_rms_norm(p, None, w, format=fmt, norm_out=out)
    o = f64(out)
    assert np.isnan(o[1]).all() and (o[2] == 0).all() and np.isfinite(o[[0, 3]]).all()
    v = f64(mx.dequantize(q))
    assert np.isnan(v[1]).all() and (v[2] == 0).all() and np.isfinite(v[[0, 3]]).all()


def test_norm_matches_the_mixture_without_bank_rows():
    """The same current row and output norm as attn_res with no bank rows."""
    T, H = 64, 7168
    p1, d = activations(T, H, 1), activations(T, H, 2)
    p2 = p1.clone()
    w = (1 + 0.1 * torch.randn(H, device="cuda")).bfloat16()
    one = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    out = ar.attn_res(p1, d, None, 0, -1, one, one, w)
    norm = torch.empty_like(out)
    mx.add_rms_norm(p2, d, w, norm_out=norm)
    assert torch.equal(p1, p2)
    # two fp32 evaluations of one formula, each rounded to bf16: they may fall
    # on different sides of a rounding border, a whole step apart
    a, b = f64(out), f64(norm)
    assert (np.abs(a - b) <= 2 * BF16_HALF * np.abs(a) + 1e-30).all()


# ---- products -------------------------------------------------------------------------


def random_matrix(rows, cols, fmt, seed, pad=0, scale=1.0, g=None):
    x = f64(activations(rows, cols, seed, scale))
    gt = None if g is None else torch.tensor([g], device="cuda")
    return Matrix(rows, cols, fmt, pad, gt).set(*R.quantize(x, fmt, g))


def matrix_values(m: Matrix, g=None) -> torch.Tensor:
    data, flat, _ = m.host()
    return torch.from_numpy(R.values(data, flat, m.fmt, g)).cuda()


def check_product(out, a, w, K):
    """bf16 rounding of fp32 sums: each of the ceil(K / 32) accumulations of a
    tensor-core step may lose two units of 2^-23 of the running magnitude,
    which is at most sum |a w|; a flush of results below 2^-126 at most that."""
    ref, mag = a @ w.t(), a.abs() @ w.abs().t()
    acc = (K / 32 + 4) * 2.0 ** -22 * mag
    err = (out.double() - ref).abs()
    tol = BF16_HALF * ref.abs() + (1 + BF16_HALF) * acc + 2.0 ** -126
    worst = (err / tol).max().item()
    assert worst <= 1, f"worst error {worst} of the tolerance"


PRODUCTS = [(1, 1, 32), (1, 128, 64), (2, 7, 96), (3, 129, 160), (15, 200, 224), (16, 64, 256), (17, 300, 512),
            (1, 2050, 7168), (32, 136, 1120), (33, 256, 416), (64, 1000, 736), (65, 72, 2048), (100, 96, 32),
            (127, 129, 480), (128, 128, 128), (129, 640, 800), (200, 257, 7200), (255, 255, 96), (256, 512, 1024),
            (300, 2050, 352), (513, 300, 640), (700, 1030, 288), (1025, 513, 4128)]


def k_blocks(fmt, K):
    return -(-(K if fmt == "mxfp8" else K // 2) // 128)


# Every form of the product: automatic; narrow with K whole, split in two and
# as often as it can be; both wide ones.
FORMS = {"auto": {}, "narrow1": dict(kernel=1, split=1), "narrow2": dict(kernel=1, split=2),
         "narrow6": dict(kernel=1, split=6), "wide": dict(kernel=2), "wider": dict(kernel=3)}


def form(name, fmt, K):
    kw = dict(FORMS[name])
    if "split" in kw:
        kw["split"] = min(kw["split"], k_blocks(fmt, K))
    return kw


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_product(fmt, M, N, K):
    a = random_matrix(M, K, fmt, 21, pad=16 if M % 2 else 0)
    w = random_matrix(N, K, fmt, 22, pad=32 if N % 2 else 0, scale=0.02)
    va, vw = matrix_values(a), matrix_values(w)
    for name in FORMS:
        out = Rows(M, N, 8 if N % 2 else 0)
        mx.matmul(a.t, w.t, out.t, **form(name, fmt, K))
        torch.cuda.synchronize()
        assert out.intact() and a.intact() and w.intact(), name
        check_product(out.t, va, vw, K)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(2500, 2500, 1120), (777, 9001, 352), (20000, 96, 64), (257, 40000, 288)])
def test_product_of_many_tiles(fmt, M, N, K):
    """More tiles than CTAs at work: the persistent forms' walk and their ring."""
    a, w = mx.quantize(activations(M, K, 31), fmt), mx.quantize((activations(N, K, 32) * 0.02).bfloat16(), fmt)

    def vals(t):
        return torch.from_numpy(R.values(t.data.view(torch.uint8).cpu().numpy(),
                                         t.scales.view(torch.uint8).cpu().numpy().reshape(-1), fmt)).cuda()
    va, vw = vals(a), vals(w)
    for name in ("auto", "narrow1", "wide", "wider"):
        check_product(mx.matmul(a, w, **form(name, fmt, K)), va, vw, K)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("off", [0, 8])
def test_product_rows_off_sector_boundaries(fmt, off):
    """Results whose rows start on 16-byte but not on 32-byte boundaries, and ragged ends."""
    M, K = 300, 256
    a = random_matrix(M, K, fmt, 33)
    for N in (256, 261, 520):
        w = random_matrix(N, K, fmt, 34)
        for name in FORMS:
            buf = torch.zeros(M, 536 + 8, dtype=torch.bfloat16, device="cuda")
            out = buf[:, off:off + N]
            mx.matmul(a.t, w.t, out, **form(name, fmt, K))
            check_product(out, matrix_values(a), matrix_values(w), K)
            assert not buf[:, :off].any() and not buf[:, off + N:].any(), name


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("N", [8, 73, 200, 505, 520, 776])
def test_product_rows_on_and_off_sector_boundaries(fmt, N):
    """Every other row of the result between two 32-byte boundaries."""
    M, K = 300, 256
    a, w = random_matrix(M, K, fmt, 35), random_matrix(N, K, fmt, 36)
    for name in FORMS:
        out = Rows(M, N)
        if out.row % 16 == 0:
            out = Rows(M, N, 8)
        mx.matmul(a.t, w.t, out.t, **form(name, fmt, K))
        torch.cuda.synchronize()
        assert out.intact(), name
        check_product(out.t, matrix_values(a), matrix_values(w), K)
        # rows that the call makes itself start on 16-byte boundaries
        y = mx.matmul(a.t, w.t, **form(name, fmt, K))
        assert y.shape == (M, N) and y.stride(0) % 8 == 0 and torch.equal(y, out.t), name


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M", [1, 5, 40, 130, 600])
def test_product_ignores_what_lies_behind(fmt, M):
    """NaN scale codes of rows that do not exist and codes behind a row's end
    have no part in any output; those behind the last group are zero."""
    K, N = 288, 200
    a, w = random_matrix(M, K, fmt, 23, pad=16), random_matrix(N, K, fmt, 24, pad=16)
    outs = []
    for fill in (0x00, 0x7F if fmt == "nvfp4" else 0xFF):
        for m in (a, w):
            t = m.gs.view.view(mx.scales_shape(fmt, m.rows, K))
            rows = torch.arange(128, device="cuda")
            behind = (t.shape[0] - 1) * 128 + rows >= m.rows
            r = rows[behind]
            t[-1][:, r % 32, r // 32, :] = fill
            m.gd.view.view(m.rows, m.row_bytes)[:, m.used:] = 0x7F if fill else 0
        outs.append([mx.matmul(a.t, w.t, **form(name, fmt, K)) for name in FORMS])
    for x, y in zip(*outs):
        assert torch.equal(x, y)
        assert torch.isfinite(x).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M", [3, 60, 200, 520])
def test_product_of_nan_groups(fmt, M):
    """A group that stands for NaN makes its row's outputs NaN and no others."""
    N, K = 150, 416
    x, v = activations(M, K, 25), activations(N, K, 26)
    x[M // 2, 100] = float("inf")
    v[7, 300] = float("nan")
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[M // 2, :] = True
    bad[:, 7] = True
    a, w = mx.quantize(x, fmt), mx.quantize(v, fmt)
    for name in FORMS:
        assert torch.equal(torch.isnan(mx.matmul(a, w, **form(name, fmt, K))), bad), name


def test_product_tensor_scales():
    M, N, K = 70, 200, 512
    a, w = random_matrix(M, K, "nvfp4", 27, g=0.031), random_matrix(N, K, "nvfp4", 28, scale=0.02, g=0.0007)
    va, vw = matrix_values(a, 0.031), matrix_values(w, 0.0007)
    check_product(mx.matmul(a.t, w.t), va, vw, K)
    # either may be absent
    a1 = mx.MxTensor(a.t.data, a.t.scales, "nvfp4")
    check_product(mx.matmul(a1, w.t), matrix_values(a), vw, K)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_product_far_scales(fmt):
    """Powers of two at both ends of the scales' range multiply exactly."""
    M, N, K = 5, 130, 64
    one = 0x38 if fmt == "mxfp8" else 2  # the element 1
    for sa, sw in ((0, 254), (254, 0), (127, 127), (1, 200), (240, 3)):
        def full(rows, s):
            e = np.full((rows, K), one, dtype=np.uint8)
            return Matrix(rows, K, fmt).set(R.pack(e, fmt), R.tile(np.full((rows, K // 32), s, np.uint8)))
        out = mx.matmul(full(M, sa).t, full(N, sw).t)
        want = K * 2.0 ** (sa + sw - 254)
        assert (out.double() == want).all(), (sa, sw, out[0, 0].item(), want)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M", [1, 48, 129, 900])
def test_product_is_repeatable(fmt, M):
    a, w = random_matrix(M, 1056, fmt, 29), random_matrix(700, 1056, fmt, 30)
    for name in FORMS:
        kw = form(name, fmt, 1056)
        first = mx.matmul(a.t, w.t, **kw)
        for _ in range(5):
            assert torch.equal(mx.matmul(a.t, w.t, **kw), first), name


def test_zero_rows():
    for fmt in FORMATS:
        e = mx.quantize(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), fmt)
        assert e.shape == (0, 64) and mx.dequantize(e).shape == (0, 64)
        w = mx.quantize(activations(40, 64, 1), fmt)
        assert mx.matmul(e, w).shape == (0, 40) and mx.matmul(w, e).shape == (40, 0)


# ---- streams, graphs, chains ------------------------------------------------------------


def layer(prefix, delta, bank, ws, fmt, pdl=False, stream=None):
    """A decoder layer's use of the operators: the mixture's row to a
    projection, its result added to the residual, normed and projected."""
    kw = dict(pdl=pdl, stream=stream)
    mixed = ar.attn_res(prefix, delta, bank, 4, -1, ws["res"], ws["rms"], ws["out"], **kw)
    up = mx.matmul(mx.quantize(mixed, fmt, **kw), ws["up"], **kw)
    q = mx.add_rms_norm(prefix, up, ws["norm"], format=fmt, **kw)
    return mixed, up, q, mx.matmul(q, ws["down"], **kw)


def layer_inputs(T, fmt, seed=0, H=7168):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    ws = {n: (1 + 0.1 * rnd(H).float()).bfloat16() for n in ("rms", "out", "norm")}
    ws["res"] = (0.02 * rnd(H).float()).bfloat16()
    ws["up"] = mx.quantize((0.02 * rnd(H, H).float()).bfloat16(), fmt)
    ws["down"] = mx.quantize((0.02 * rnd(2048, H).float()).bfloat16(), fmt)
    return rnd(T, H), rnd(T, H), rnd(T, 8, H), ws


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 37, 300])
def test_layer(fmt, T):
    """The operators together, each checked on what the one before it gave."""
    prefix, delta, bank, ws = layer_inputs(T, fmt)
    p0, b0 = prefix.clone(), bank.clone()
    mixed, up, q, down = layer(prefix, delta, bank, ws, fmt)
    assert torch.equal(bank, b0)
    H = mixed.shape[1]

    def vals(t):
        r, k = t.shape
        return torch.from_numpy(R.values(t.data.view(torch.uint8).cpu().numpy(),
                                         t.scales.view(torch.uint8).cpu().numpy().reshape(-1), t.format)).cuda()
    data, flat = R.quantize(f64(mixed), fmt)
    a = torch.from_numpy(R.values(data, flat, fmt)).cuda()
    check_product(up, a, vals(ws["up"]), H)
    c1 = (p0.float() + delta.float()).bfloat16()
    c2 = (c1.float() + up.float()).bfloat16()
    assert torch.equal(prefix, c2)
    check_product(down, vals(q), vals(ws["down"]), H)
    y = c2.double() * torch.rsqrt(c2.double().square().mean(-1, keepdim=True) + 1e-6) * ws["norm"].double()
    # the 8- or 4-bit rows stand near the norm: half a step of the elements
    # under the group's scale (its top element at most twice the scale's reach)
    amax = y.view(T, -1, R.GROUP[fmt]).abs().amax(-1, keepdim=True)
    step = 2.0 ** -3 if fmt == "mxfp8" else 2.0 / 6 + (2.0 ** -3 if fmt == "nvfp4" else 0)
    err = (vals(q) - y).view(T, -1, R.GROUP[fmt]).abs()
    if fmt == "nvfp4":
        step = step + 2.0 ** -9 * 6 / amax.clamp(min=1e-3)
    assert (err <= step * amax).all()


@pytest.mark.parametrize("T", [1, 200])
def test_layer_with_programmatic_launches(T):
    """Chains with PDL flags give the same bits, in order and back to back."""
    for fmt in FORMATS:
        prefix, delta, bank, ws = layer_inputs(T, fmt)
        p1, p2 = prefix.clone(), prefix.clone()
        want = [layer(p1, delta, bank, ws, fmt) for _ in range(4)]
        got = [layer(p2, delta, bank, ws, fmt, pdl=True) for _ in range(4)]
        torch.cuda.synchronize()
        assert torch.equal(p1, p2)
        for x, y in zip(want, got):
            assert torch.equal(x[1], y[1]) and torch.equal(x[3], y[3])


@pytest.mark.parametrize("T", [1, 200])
def test_layer_in_a_graph(T):
    """Captured and replayed on new inputs; two graphs replayed side by side."""
    fmt = "mxfp4"
    sets = [layer_inputs(T, fmt, seed) for seed in (1, 2)]
    want = []
    for prefix, delta, bank, ws in sets:
        want.append(layer(prefix.clone(), delta, bank, ws, fmt)[3])
    graphs, outs, statics = [], [], []
    for prefix, delta, bank, ws in sets:
        p = prefix.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(layer(p, delta, bank, ws, fmt)[3])
        graphs.append(g)
        statics.append(p)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for p, (prefix, *_r) in zip(statics, sets):
            p.copy_(prefix)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, x in zip(outs, want):
            assert torch.equal(o, x)


def test_calls_in_flight_together():
    """Products on five streams at once, every form among them."""
    cases = []
    for i, (M, fmt, name) in enumerate([(1, "mxfp4", "auto"), (48, "nvfp4", "narrow6"), (150, "mxfp8", "narrow2"),
                                        (2000, "mxfp4", "wider"), (700, "nvfp4", "wide")]):
        a = mx.quantize(activations(M, 2048, 40 + i), fmt)
        w = mx.quantize(activations(1500, 2048, 50 + i), fmt)
        kw = form(name, fmt, 2048)
        cases.append((a, w, kw, mx.matmul(a, w, **kw), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = [[] for _ in cases]
    for _ in range(8):
        for k, (a, w, kw, _o, s) in enumerate(cases):
            got[k].append(mx.matmul(a, w, stream=s, **kw))
    torch.cuda.synchronize()
    for k, (_a, _w, _kw, o, _s) in enumerate(cases):
        assert all(torch.equal(o, x) for x in got[k])


def test_other_stream_than_the_current():
    s = torch.cuda.Stream()
    x = activations(100, 512, 60)
    torch.cuda.synchronize()
    q = mx.quantize(x, "mxfp4", stream=s)
    y = mx.dequantize(q, stream=s)
    s.synchronize()
    assert torch.equal(y, mx.dequantize(mx.quantize(x, "mxfp4")))


def test_binding_refusals():
    x = activations(4, 64, 1)
    q = mx.quantize(x, "mxfp4")
    with pytest.raises(ValueError):
        mx.quantize(x.t(), "mxfp4")
    with pytest.raises(ValueError):
        mx.quantize(x[:, :48], "mxfp4")
    with pytest.raises(ValueError):
        mx.quantize(x, "mxfp8", out=q)
    with pytest.raises(ValueError):
        mx.matmul(q, mx.quantize(x, "nvfp4"))
    with pytest.raises(ValueError):
        mx.matmul(q, mx.quantize(activations(4, 96, 1), "mxfp4"))
    with pytest.raises(ValueError):
        mx.matmul(q, q, torch.empty(4, 8, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        mx.MxTensor(q.data, q.scales, "mxfp4", torch.ones(1, device="cuda"))
    with pytest.raises(ValueError):
        mx.MxTensor(q.data, q.scales.view(torch.uint8), "mxfp4")
    with pytest.raises(ValueError):
        mx.add_rms_norm(x, x[:2].clone(), x[0])
    with pytest.raises(ar.AttnResError):
        mx.add_rms_norm(x, x, x[0].clone())
    with pytest.raises(ValueError):
        mx.quantize(x, "mxfp5")
    with pytest.raises(ar.AttnResError):
        mx.matmul(q, q, kernel=4)
    with pytest.raises(ar.AttnResError):
        mx.matmul(q, q, kernel=mx.KERNEL_WIDE, split=2)
    with pytest.raises(ValueError):
        mx.matmul(q, q, split=-1)
    with pytest.raises(TypeError):
        mx.matmul(q, q.data)


@pytest.mark.slow
def test_far_offsets():
    """Rows past 2^31 elements and bytes from their buffers' start."""
    row = 1 << 22
    rows = 700  # 2.9e9 elements apart at the end, in 5.9 GB
    buf = torch.zeros(rows * row, dtype=torch.bfloat16, device="cuda").view(rows, row)
    x = buf[:, :256]
    x.copy_(activations(rows, 256, 70))
    # written ranges may not enclose what is read: the results' own buffer
    res = torch.zeros(rows * row, dtype=torch.bfloat16, device="cuda").view(rows, row)
    for fmt in FORMATS:
        near = mx.quantize(x.contiguous(), fmt)
        far = mx.quantize(x, fmt)
        assert torch.equal(near.data.view(torch.uint8), far.data.view(torch.uint8))
        assert torch.equal(near.scales.view(torch.uint8), far.scales.view(torch.uint8))
        w = mx.quantize(activations(200, 256, 71), fmt)
        want = mx.matmul(near, w)
        # the codes' rows far apart, and the product's rows
        big = buf.view(torch.uint8)[:, row:row + near.data.shape[1]]
        big.copy_(near.data.view(torch.uint8))
        a = mx.MxTensor(big.view(near.data.dtype), near.scales, fmt)
        out = res[:, 1024:1224]
        mx.matmul(a, w, out)
        assert torch.equal(out, want)
        assert torch.equal(mx.matmul(w, a)[:5], mx.matmul(w, near)[:5])
        back = res[:, 2048:2304]
        mx.dequantize(a, back)
        assert torch.equal(back, mx.dequantize(near))
        p = res[:, 4096:4352]
        p.copy_(x)
        qn = mx.add_rms_norm(p, x, torch.ones(256, dtype=torch.bfloat16, device="cuda"), format=fmt, out=None)
        pn = x.contiguous()
        qc = mx.add_rms_norm(pn, x.contiguous(), torch.ones(256, dtype=torch.bfloat16, device="cuda"), format=fmt)
        assert torch.equal(p, pn) and torch.equal(qn.data.view(torch.uint8), qc.data.view(torch.uint8))
