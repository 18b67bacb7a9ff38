"""The microscaled formats restated in numpy, from the definition in
include/attn_res.h, apart from the CUDA code: every element and scale is
found by searching the list of values that its code can stand for."""
from __future__ import annotations

import numpy as np

FORMATS = ("mxfp8", "mxfp4", "nvfp4")
CODE = {"mxfp8": 1, "mxfp4": 2, "nvfp4": 3}
GROUP = {"mxfp8": 32, "mxfp4": 32, "nvfp4": 16}
TOP = {"mxfp8": 448.0, "mxfp4": 6.0, "nvfp4": 6.0}

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _e4m3_positive() -> np.ndarray:
    v = []
    for code in range(127):
        e, m = code >> 3, code & 7
        v.append(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(v)


E4M3 = _e4m3_positive()  # value of code i; 127 is NaN


def nearest_code(v: np.ndarray, table: np.ndarray) -> np.ndarray:
    """Index of the table value nearest to v >= 0 (at most the last), ties to
    the even index; every table above alternates even and odd significands."""
    v = np.minimum(v, table[-1])
    hi = np.clip(np.searchsorted(table, v), 1, len(table) - 1)
    below, above = v - table[hi - 1], table[hi] - v
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return np.where(up, hi, hi - 1)


def e8m0(codes: np.ndarray) -> np.ndarray:
    c = codes.astype(np.float64)
    return np.where(codes == 255, np.nan, np.exp2(c - 127))


def e4m3(codes: np.ndarray) -> np.ndarray:
    c = codes.astype(int)
    v = np.append(E4M3, np.nan)[c & 127]
    return np.where(c & 128, -v, v)


def tile(codes: np.ndarray) -> np.ndarray:
    """[rows, groups] scale codes -> the tiled bytes, entry by entry."""
    rows, groups = codes.shape
    gt = -(-groups // 4)
    out = np.zeros(-(-rows // 128) * gt * 512, dtype=np.uint8)
    r = np.arange(rows)[:, None]
    j = np.arange(groups)[None, :]
    out[(r // 128 * gt + j // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + j % 4] = codes
    return out


def untile(flat: np.ndarray, rows: int, groups: int) -> np.ndarray:
    gt = -(-groups // 4)
    r = np.arange(rows)[:, None]
    j = np.arange(groups)[None, :]
    return flat[(r // 128 * gt + j // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + j % 4]


def scale_codes(amax: np.ndarray, fmt: str, g=None) -> np.ndarray:
    """Codes of the group scales for the groups' largest magnitudes."""
    if fmt == "nvfp4":
        g = np.float32(1 if g is None else g)
        t = (amax.astype(np.float32) / np.float32(np.float32(6) * g)).astype(np.float64)
        ok = np.isfinite(amax)
        return np.where(ok, nearest_code(np.where(ok, t, 0), E4M3), 127).astype(np.uint8)
    out = np.full(amax.shape, 255, dtype=int)
    for c in range(254, -1, -1):
        out = np.where(amax <= TOP[fmt] * 2.0 ** (c - 127), c, out)
    return np.where(np.isfinite(amax), out, 255).astype(np.uint8)


def element_codes(x: np.ndarray, codes: np.ndarray, fmt: str, g=None) -> np.ndarray:
    """Element codes [rows, cols] of float64 values that are fp32 numbers."""
    xg = x.reshape(x.shape[0], codes.shape[1], GROUP[fmt])
    bad = codes == (127 if fmt == "nvfp4" else 255)
    with np.errstate(all="ignore"):
        if fmt == "nvfp4":
            g = np.float32(1 if g is None else g)
            d = (e4m3(codes).astype(np.float32) * g)[..., None]
            v = np.where(d > 0, xg.astype(np.float32) / d, np.float32(0)).astype(np.float64)
        else:
            v = xg / e8m0(codes)[..., None]
    v = np.where(bad[..., None], 0.0, v)
    table, sign = (E4M3, 128) if fmt == "mxfp8" else (E2M1, 8)
    c = nearest_code(np.abs(v), table) | np.where(np.signbit(v), sign, 0)
    return c.reshape(x.shape).astype(np.uint8)


def pack(codes: np.ndarray, fmt: str) -> np.ndarray:
    return codes if fmt == "mxfp8" else codes[:, ::2] | (codes[:, 1::2] << 4)


def unpack(data: np.ndarray, fmt: str) -> np.ndarray:
    if fmt == "mxfp8":
        return data
    return np.stack([data & 15, data >> 4], axis=-1).reshape(data.shape[0], -1)


def quantize(x: np.ndarray, fmt: str, g=None):
    """float64 [rows, cols] -> (data bytes, tiled scale bytes)."""
    amax = np.abs(x.reshape(x.shape[0], -1, GROUP[fmt])).max(-1)
    amax = np.where(np.isnan(x.reshape(x.shape[0], -1, GROUP[fmt])).any(-1), np.nan, amax)
    s = scale_codes(amax, fmt, g)
    return pack(element_codes(x, s, fmt, g), fmt), tile(s)


def elements(data: np.ndarray, fmt: str) -> np.ndarray:
    c = unpack(data, fmt).astype(int)
    if fmt == "mxfp8":
        return e4m3(c)
    return np.where(c & 8, -1.0, 1.0) * E2M1[c & 7]


def scales(flat: np.ndarray, rows: int, groups: int, fmt: str) -> np.ndarray:
    c = untile(flat, rows, groups)
    return e4m3(c) if fmt == "nvfp4" else e8m0(c)


def values(data: np.ndarray, flat: np.ndarray, fmt: str, g=None) -> np.ndarray:
    """The float64 values that codes and tiled scales stand for."""
    q = elements(data, fmt)
    s = scales(flat, q.shape[0], q.shape[1] // GROUP[fmt], fmt)
    v = (q.reshape(q.shape[0], s.shape[1], -1) * s[..., None]).reshape(q.shape)
    return v if g is None else v * float(np.float32(g))
