"""The activations' accuracy behind the 8-bit codes.

A group with a single value that is not 0 has that value over 448 for its scale, to
fp32.  Here the values lie where token and column agree modulo 128, one to a group of
every result, by rows and transposed.  Bounds in units of 2^-23 (half of one a
rounding), relative; p = 1 / (1 + exp(-z)) is off by (1 - p) times what exp(-z) is off
by, half a unit of the sum and one of the reciprocal (rcp.approx)."""
import pytest
import torch

import attention_residual_fusion_gb300 as ar
from attention_residual_fusion_gb300 import _build, f8
from tests import f8_restatement as R

pytestmark = pytest.mark.gpu

UNIT = 2.0 ** -23
T, F = 512, 1024
ONE = 0x38  # the code of 1


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    ar.device_status(clear=True)
    yield
    assert ar.device_status() == 0


def single(rows, cols):
    """Where a value lies: [rows, cols]."""
    r, c = torch.arange(rows, device="cuda")[:, None], torch.arange(cols, device="cuda")[None, :]
    return r % 128 == c % 128


def gates(n, act, seed=3):
    """Gate values from where z is -85 up to where p is 1."""
    lo, hi = (-85.0, 20.0) if act == "silu" else (-9.8, 6.0)
    g = torch.rand(n, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda") * (hi - lo) + lo
    g[:8] = torch.tensor([lo, hi, -1.0, 1.0, -1e-3, 1e-3, -1e-10, 0.5 * lo], device="cuda")
    return g


def sigmoid_arg(g, act):
    """z, z' and how far z's own roundings in fp32 may take it (relative)."""
    if act == "silu":
        return g, torch.ones_like(g), 0.0
    k = (8 / torch.pi) ** 0.5
    return k * (g + 0.044715 * g ** 3), k * (1 + 3 * 0.044715 * g * g), None


def check(got, want, error, what):
    """Scales of groups with one value: |value| / 448, rounded."""
    v, want = got.double() * 448.0, want.abs()
    bound = error + (want + error) * 2.0 ** -24
    worst = ((v - want).abs() / bound).max()
    assert bool(((v - want).abs() <= bound).all()), f"{what}: {worst.item():.2f} times the bound"


def of_groups(x):
    """The one value of each row and block of 128 columns of [rows, cols], as scales lie: [blocks, rows]."""
    rows, cols = x.shape
    return x.view(rows, cols // 128, 128).sum(2).t()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_backward(act):
    """exp(-z) there is off by 2 units (ex2.approx) and half of one; z (GELU) by its constants', the square's, the
    sum's and the product's roundings, 2 units of z at most."""
    where = single(T, F)
    value = gates(T * F // 128, act).view(T, F // 128)  # of each row and block
    g = f8.F8Tensor(((ONE + 128 * (value < 0)).repeat_interleave(128, 1) * where).to(torch.uint8).view(torch.float8_e4m3fn),
                    value.abs().t().contiguous())
    u = f8.F8Tensor((ONE * where).to(torch.uint8).view(torch.float8_e4m3fn), torch.ones(F // 128, T, device="cuda"))
    dh = where.to(torch.bfloat16)
    dg, du, dgt, dut, ht = f8.gated_backward(dh, g, u, act)
    x = (value.double().repeat_interleave(128, 1) * where)
    a, da = R.act(x, act)
    z, dz, off_z = sigmoid_arg(x, act)
    p = torch.sigmoid(z)
    q = 1 - p
    ep = UNIT * p * (1.5 + q * (2.5 + (2 * z.abs() if off_z is None else 0)))
    ea = x.abs() * ep + 0.5 * UNIT * a.abs()
    # slope = p + t z', t = act (1 - p): 1 - p is off by ep and half a unit, z' (GELU) by three roundings
    et = ea * q + a.abs() * (ep + 0.5 * UNIT * q) + 0.5 * UNIT * (a * q).abs()
    ed = ep + dz * et + (1.5 * UNIT * dz * (a * q).abs() if act == "gelu" else 0) + 0.5 * UNIT * da.abs()
    a, da, ea, ed = (t * where for t in (a, da, ea, ed))
    for got, want, error, what in ((dg, da, ed, "dg"), (du, a, ea, "du")):
        check(got.scales, of_groups(want), of_groups(error), what)
    for got, want, error, what in ((dgt, da, ed, "dg^T"), (dut, a, ea, "du^T"), (ht, a, ea, "h^T")):
        check(got.scales, of_groups(want.t().contiguous()), of_groups(error.t().contiguous()), what)
    for got, want in ((dg, da), (du, a), (dgt, da.t()), (dut, a.t()), (ht, a.t())):
        assert torch.equal(got.data.view(torch.uint8) & 0x7F, (126 * (want != 0)).to(torch.uint8))
        assert torch.equal(got.data.double() < 0, want < 0)


@pytest.mark.parametrize("kernel", [f8.KERNEL_NARROW, f8.KERNEL_WIDE])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_forward(act, kernel):
    """g = u = the token's scale.  exp(-z) there is off by the fast exponential's documented 2 + floor(1.173 |z|) units;
    z (GELU) by its two constants' and four operations' roundings, 3 units of z at most."""
    value = gates(T, act)
    eye = (ONE * single(F, 128)).to(torch.uint8).view(torch.float8_e4m3fn)
    x = f8.F8Tensor(((ONE + 128 * (value < 0))[:, None] * single(T, 128)).to(torch.uint8).view(torch.float8_e4m3fn),
                    value.abs()[None, :].contiguous())
    w = f8.F8Tensor(eye, torch.ones(F // 128, 1, device="cuda"), 128)
    h, g, u = f8.gated(x, w, w, act, save=True, kernel=kernel)
    v = value.double()
    for t in (g, u):
        check(t.scales, v.expand(F // 128, T), 0 * v, "projections")
    a, _ = R.act(v, act)
    z, _, off_z = sigmoid_arg(v, act)
    p = torch.sigmoid(z)
    e = UNIT * (2.0 + (1 - p) * (2 + (1.173 * z.abs()).floor() + (3 * z.abs() if off_z is None else 0)))
    # (a quotient below 2^-126 may lose bits: half a step of 2^-149)
    check(h.scales, (a * v).expand(F // 128, T), ((a * v).abs() * (e + 0.5 * UNIT) + 2.0 ** -149 * v.abs()).expand(F // 128, T), "h")
    # what the header says: SiLU to 2^-16 of itself, GELU to 2^-14
    limit = (2.0 ** -16 if act == "silu" else 2.0 ** -14) + UNIT
    check(h.scales, (a * v).expand(F // 128, T), ((a * v).abs() * limit).expand(F // 128, T), "h, as documented")
