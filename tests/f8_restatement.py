"""The 8-bit format with scales for blocks of 128, its products and the gated
block, restated in 64 bits (torch, on whatever device the inputs are on)."""
import math

import torch

BLOCK = 128
F32 = torch.float32
F64 = torch.float64

# e4m3 values of the codes 0 .. 126, by definition
E4M3 = [m * 2.0 ** -9 for m in range(8)] + [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)][:-1]


def blocks(n):
    return -(-n // BLOCK)


def group_index(rows, cols, block, device):
    """[rows, cols] -> the place of an element's scale in scales.reshape(-1)."""
    r = torch.arange(rows, device=device)[:, None]
    b = torch.arange(cols, device=device)[None, :] // BLOCK
    if block == 1:
        return b * rows + r
    return (r // BLOCK) * blocks(cols) + b


def scales_shape(rows, cols, block):
    return (blocks(cols), rows) if block == 1 else (blocks(rows), blocks(cols))


def nearest_code(x):
    """Codes of the nearest e4m3 values to fp64 x, ties to the even code, saturating; the sign kept."""
    grid = torch.tensor(E4M3, dtype=F64, device=x.device)
    a = x.abs().clamp(max=448.0)
    hi = torch.bucketize(a, grid).clamp(1, len(E4M3) - 1)
    below, above = a - grid[hi - 1], grid[hi] - a
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    code = torch.where(up, hi, hi - 1)
    return (code + 128 * torch.signbit(x)).to(torch.uint8)


def quantize(x, block):
    """(codes uint8 [r, c], scales fp32) of values that fp32 holds: correctly rounded fp32 quotients."""
    r, c = x.shape
    shape = scales_shape(r, c, block)
    idx = group_index(r, c, block, x.device)
    a = x.double().abs()
    bad = torch.zeros(shape, dtype=torch.int64, device=x.device).view(-1)
    bad.scatter_reduce_(0, idx.reshape(-1), (~torch.isfinite(a)).long().reshape(-1), "amax")
    top = torch.zeros(shape, dtype=F64, device=x.device).view(-1)
    top.scatter_reduce_(0, idx.reshape(-1), torch.where(torch.isfinite(a), a, 0.0).reshape(-1), "amax")
    s = (top / 448.0).to(F32)  # (one rounding: top is an fp32 value)
    s = torch.where(top == 0, torch.ones_like(s), s.clamp(min=2.0 ** -126))
    q = x.double() / s.double()[idx]
    # rounded to fp32 first, then to e4m3; an fp64 quotient of fp32 values rounds to the same fp32
    codes = nearest_code(torch.where(torch.isfinite(q), q, 0.0).to(F32).double())
    codes = torch.where(bad[idx] > 0, torch.zeros_like(codes), codes)
    s = torch.where(bad > 0, torch.full_like(s, float("nan")), s)
    return codes, s.view(shape)


def values(codes, scales, block):
    """fp64 values of codes (float8 or uint8) and scales."""
    t = codes if codes.dtype == torch.float8_e4m3fn else codes.view(torch.float8_e4m3fn)
    r, c = t.shape
    s = scales.double().reshape(-1)
    if r == 0 or c == 0:
        return torch.zeros(r, c, dtype=F64, device=t.device)
    return t.double() * s[group_index(r, c, block, t.device)]


def act(g, kind):
    """act(g) and its derivative, fp64."""
    if kind == "silu":
        p = torch.sigmoid(g)
        return g * p, p + g * p * (1 - p)
    # (1 + tanh(y)) / 2 as the sigmoid of 2 y: 1 + tanh loses all of small values
    k = math.sqrt(8 / math.pi)
    p = torch.sigmoid(k * (g + 0.044715 * g ** 3))
    return g * p, p + g * p * (1 - p) * k * (1 + 3 * 0.044715 * g * g)


# ---- bounds ---------------------------------------------------------------------
# Half a step of rounding, relative to the value at most: bf16 2^-8, fp32 2^-24,
# e4m3 2^-4 (and 2^-10 of the scale where the code is subnormal).


def product_bound(magnitudes, cols):
    """Of fp32 sums of products of codes, times scales: magnitudes = |a| |w|^T.
    In a block of K 128 exact products are added, each addition off by a unit of
    fp32 (2^-23: the tensor cores may cut off) of sums no larger than the
    block's magnitudes; the scales' product and the scaled sum are rounded, and
    the blocks' sums added, to fp32 each."""
    return magnitudes * (128 * 2.0 ** -23 + (blocks(cols) + 3) * 2.0 ** -24)


def code_bound(value, error, scale):
    """Of a value rounded to a code from something off by `error`: half a step
    of the value that was rounded, half the smallest step times the scale, and
    the quotient's and the product's roundings."""
    return error + (value.abs() + error) * (2.0 ** -4 + 2.0 ** -22) + scale * 2.0 ** -10
