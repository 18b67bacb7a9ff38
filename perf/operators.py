"""Measured cases of the microscaled operators (attention_residual_fusion_gb300.mx).

Operators:

* ``norm``     residual addition and root-mean-square norm of token rows, the
               normalised row in 8 bits with a scale for each 32 columns;
* ``quantize`` bf16 rows to a microscaled format and back to bf16 (the two
               directions; in the 8-bit format the codes themselves);
* ``product``  activations [rows, cols] times weights [n, cols], transposed,
               both in a microscaled format, the sums in 32 bits.

Formats: ``mxfp8`` (e4m3 elements, a power-of-two scale for each 32 of a row),
``mxfp4`` (e2m1 elements, the same scales), ``nvfp4`` (e2m1 elements, an e4m3
scale for each 16 and one fp32 scale for the tensor).

Scales lie in tiles of 128 rows x 4 groups: entry [i, j, r, p, g] belongs to
row 128 i + 32 p + r and to group 4 j + g of that row; entries past the last
row or group are zero codes.  4-bit codes lie two to a byte, the even column
in the low half.

``run`` computes the operators in plain torch operations, or with ``own`` set
by the framework's calls.
"""
import math

import torch

own = False

H = 7168  # the row width that the framework's tuned kernels are built for
GROUP = {"mxfp8": 32, "mxfp4": 32, "nvfp4": 16}
TOP = {"mxfp8": 448.0, "mxfp4": 6.0, "nvfp4": 6.0}
EPS = 1e-6


# ---- cases ---------------------------------------------------------------------


def listed():
    norm = lambda name, rows, cols, **more: dict(  # noqa: E731
        name=name, op="norm", rows=rows, cols=cols, **{"delta": True, "pad": 0, "both": False, **more})
    quant = lambda name, fmt, rows, cols, pad=0: dict(  # noqa: E731
        name=name, op="quantize", format=fmt, rows=rows, cols=cols, pad=pad)
    prod = lambda name, fmt, rows, n, cols: dict(  # noqa: E731
        name=name, op="product", format=fmt, rows=rows, n=n, cols=cols)
    return [
        # one token of a decode step: the launch itself counts
        norm("norm one token", 1, H),
        # a decode batch; the bf16 row is kept as well, for a router or a head
        norm("norm decode 256", 256, H, both=True),
        # a row count and a width that nothing divides well, no addend
        norm("norm odd 1003x2080", 1003, 2080, delta=False),
        # long prefill, the framework's largest workload, rows in a padded buffer
        norm("norm prefill 8192", 8192, H, pad=64),
        # the activations of a few speculative tokens before an 8-bit product
        quant("quantize mxfp8 4x16384", "mxfp8", 4, 16384),
        # ragged rows of a mid-sized batch in the finer-grained 4-bit format
        quant("quantize nvfp4 333x4128", "nvfp4", 333, 4128, pad=32),
        # a long prefill's activations, or a weight matrix when it is loaded
        quant("quantize mxfp4 8192x7168", "mxfp4", 8192, H),
        # decode of one token: the product is the reading of the weights
        prod("product mxfp4 1 token", "mxfp4", 1, H, H),
        # a decode batch against a projection
        prod("product nvfp4 64 tokens", "nvfp4", 64, 4096, H),
        # ragged in every direction: a last batch of a chunked prefill, a gate
        prod("product mxfp8 300 odd", "mxfp8", 300, 2050, 7200),
        # prefill against a wide up-projection
        prod("product nvfp4 4096 wide", "nvfp4", 4096, 16384, 2048),
        # long prefill against a square projection
        prod("product mxfp4 8192", "mxfp4", 8192, H, H),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "quantize", "product", "product"])
    if op == "product":
        fmt = rng.choice(["mxfp8", "mxfp4", "nvfp4"])
        rows, n, cols = _log(rng, 1, 8192), _log(rng, 64, 16384), 32 * _log(rng, 4, 512)
        # at most half of the largest listed product (8 bits cost more than 4)
        while rows * n * cols > 8192 * H * H // 2:
            rows = max(1, rows // 2)
        return dict(op=op, format=fmt, rows=rows, n=n, cols=cols)
    rows, cols = _log(rng, 1, 8192), 32 * _log(rng, 8, 512)
    while rows * cols > 8192 * H * 3 // 4:
        rows = max(1, rows // 2)
    pad = rng.choice([0, 0, 16, 64])
    if op == "norm":
        return dict(op=op, rows=rows, cols=cols, delta=rng.random() < 0.75, pad=pad, both=rng.random() < 0.25)
    return dict(op=op, format=rng.choice(["mxfp8", "mxfp4", "nvfp4"]), rows=rows, cols=cols, pad=pad)


def work(case):
    rows, cols = case["rows"], case["cols"]
    if case["op"] == "norm":
        d = int(case["delta"])
        moved = rows * cols * (2 + 4 * d + 1 + 2 * int(case["both"])) + rows * cols // 32 + 2 * cols
        return {"bytes": moved, "flops": (8 + d) * rows * cols}
    fmt = case["format"]
    bits = 8 if fmt == "mxfp8" else 4

    def packed(r):
        return r * cols * bits // 8 + r * cols // GROUP[fmt]

    if case["op"] == "quantize":
        back = 0 if fmt == "mxfp8" else 2 * rows * cols
        return {"bytes": 2 * rows * cols + packed(rows) + back, "flops": 4 * rows * cols}
    return {"bytes": packed(rows) + packed(case["n"]) + 2 * rows * case["n"], "flops": 2 * rows * case["n"] * cols}


# ---- the formats in plain torch ---------------------------------------------------


def _tile(codes):
    """[rows, groups] codes -> [row tiles, group tiles, 32, 4, 4], zero codes behind."""
    r, g = codes.shape
    rt, gt = -(-r // 128), -(-g // 4)
    full = torch.zeros(rt * 128, gt * 4, dtype=codes.dtype, device=codes.device)
    full[:r, :g] = codes
    return full.view(rt, 4, 32, gt, 4).permute(0, 3, 2, 1, 4).contiguous()


def _untile(t, rows, groups):
    rt, gt = t.shape[:2]
    return t.permute(0, 3, 2, 1, 4).reshape(rt * 128, gt * 4)[:rows, :groups]


def _pow2(e):
    return torch.exp2(e.double()).float()


def _mx_codes(amax, top):
    """Codes c of the smallest powers of two 2^(c - 127) with amax <= top * 2^(c - 127);
    255 (no number) where amax is none."""
    m, e = torch.frexp(amax)
    mt, et = math.frexp(top)
    c = (e - et + (m > mt).to(e.dtype) + 127).clamp(min=0)
    c = torch.where(amax == 0, torch.zeros_like(c), c)
    return torch.where(torch.isfinite(amax), c, torch.full_like(c, 255))


def _e2m1(v):
    """Codes of the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (ties to the even code), with the sign."""
    a = v.abs().clamp(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = torch.round(a / step) * step
    code = torch.where(q <= 2, 2 * q, torch.where(q <= 4, q + 2, torch.full_like(q, 7.0)))
    return code.to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)


def _quantize(x, fmt, g):
    """fp32 rows -> (codes, tiled scale codes): e4m3 values, or packed e2m1 bytes."""
    r, k = x.shape
    xg = x.view(r, k // GROUP[fmt], GROUP[fmt])
    amax = xg.abs().amax(-1)
    if fmt == "nvfp4":
        s = (amax / (6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
        d = s.float() * g
        v = torch.where(d[..., None] > 0, xg / d[..., None], torch.zeros_like(xg))
        bad = ~torch.isfinite(amax)
        scales = torch.where(bad, torch.full_like(s.view(torch.uint8), 0x7F), s.view(torch.uint8))
    else:
        c = _mx_codes(amax, TOP[fmt])
        v = xg * _pow2(127 - c)[..., None]
        bad = c == 255
        scales = c.to(torch.uint8)
    v = torch.where(bad[..., None], torch.zeros_like(xg), v).view(r, k)
    kind = torch.float8_e4m3fn if fmt == "nvfp4" else torch.float8_e8m0fnu
    scales = _tile(scales).view(kind)
    if fmt == "mxfp8":
        return v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scales
    q = _e2m1(v).view(r, k // 2, 2)
    return q[..., 0] | (q[..., 1] << 4), scales


_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _values(data, scales, fmt, g):
    """The fp32 values of codes and tiled scales (without the tensor's scale where g is None)."""
    r = data.shape[0]
    if fmt == "mxfp8":
        q = data.float()
    else:
        table = torch.tensor(_E2M1 + [-v for v in _E2M1], device=data.device)
        q = table[torch.stack((data & 15, data >> 4), -1).view(r, -1).int()]
    groups = q.shape[1] // GROUP[fmt]
    if fmt == "nvfp4":
        s = _untile(scales.view(torch.uint8), r, groups).contiguous().view(torch.float8_e4m3fn).float()
    else:
        c = _untile(scales.view(torch.uint8), r, groups).int()
        s = torch.where(c == 255, torch.full((), float("nan"), device=c.device), _pow2(c - 127))
    v = (q.view(r, groups, -1) * s[..., None]).view(r, -1)
    return v if g is None else v * g


# ---- inputs ------------------------------------------------------------------------


def _activations(gen, rows, cols, pad=0):
    """N(0, 1) with one value in a hundred 50 times as large, bf16, rows in a buffer of cols + pad."""
    x = torch.randn(rows, cols + pad, generator=gen, device="cuda")
    x *= 1.0 + 49.0 * (torch.rand(rows, cols + pad, generator=gen, device="cuda") < 0.01)
    return x.to(torch.bfloat16)[:, :cols]


def _tensor_scale(x):
    """The least power of two at which the largest value's group scale is no more than 448
    (a power of two, as a calibration that leaves the elements' roundings alone gives)."""
    return torch.exp2(torch.ceil(torch.log2(x.abs().amax().double() / (448.0 * 6.0)))).float().view(1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rows, cols, op = case["rows"], case["cols"], case["op"]
    s = {"op": op}
    if op == "norm":
        s["prefix"] = _activations(gen, rows, cols, case["pad"])
        s["delta"] = _activations(gen, rows, cols, case["pad"]) if case["delta"] else None
        s["weight"] = (1 + 0.1 * torch.randn(cols, generator=gen, device="cuda")).to(torch.bfloat16)
        s["both"] = case["both"]
        return s
    fmt = s["format"] = case["format"]
    if op == "quantize":
        s["x"] = _activations(gen, rows, cols, case["pad"])
        s["g"] = _tensor_scale(s["x"]) if fmt == "nvfp4" else None
        return s
    for name, r, scale in (("a", rows, 1.0), ("w", case["n"], 0.02)):
        x = _activations(gen, r, cols) if name == "a" else \
            (scale * torch.randn(r, cols, generator=gen, device="cuda")).to(torch.bfloat16)
        g = _tensor_scale(x) if fmt == "nvfp4" else None
        s[name], s[name + "_scales"] = _quantize(x.float(), fmt, g)
        s[name + "_g"] = g
    return s


# ---- the passes ----------------------------------------------------------------------


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from attention_residual_fusion_gb300 import mx

    if s["op"] == "norm":
        out = torch.empty(s["prefix"].shape, dtype=torch.bfloat16, device="cuda") if s["both"] else None
        q = mx.add_rms_norm(s["prefix"], s["delta"], s["weight"], EPS, format="mxfp8", norm_out=out)
        return {"prefix": s["prefix"], "q": q.data, "scales": q.scales, "norm": out}
    fmt = s["format"]
    if s["op"] == "quantize":
        q = mx.quantize(s["x"], fmt, s["g"])
        if fmt == "mxfp8":
            return {"q": q.data, "scales": q.scales}
        return {"values": mx.dequantize(q)}
    a = mx.MxTensor(s["a"], s["a_scales"], fmt, s["a_g"])
    w = mx.MxTensor(s["w"], s["w_scales"], fmt, s["w_g"])
    return {"out": mx.matmul(a, w)}


def _run_plain(s):
    if s["op"] == "norm":
        c = s["prefix"].float()
        if s["delta"] is not None:
            s["prefix"].copy_(c + s["delta"].float())
            c = s["prefix"].float()
        y = c * torch.rsqrt((c * c).mean(-1, keepdim=True) + EPS) * s["weight"].float()
        q, scales = _quantize(y, "mxfp8", None)
        return {"prefix": s["prefix"], "q": q, "scales": scales,
                "norm": y.to(torch.bfloat16) if s["both"] else None}
    fmt = s["format"]
    if s["op"] == "quantize":
        q, scales = _quantize(s["x"].float(), fmt, s["g"])
        if fmt == "mxfp8":
            return {"q": q, "scales": scales}
        return {"values": _values(q, scales, fmt, s["g"]).to(torch.bfloat16)}
    a = _values(s["a"], s["a_scales"], fmt, None)
    w = _values(s["w"], s["w_scales"], fmt, None)
    out = a @ w.t()
    if fmt == "nvfp4":
        out = out * (s["a_g"] * s["w_g"])
    return {"out": out.to(torch.bfloat16)}


# ---- the definitions in 64 bits --------------------------------------------------------


def _nearest(v, grid):
    """The nearest entries of an ascending grid to v >= 0, ties to the even index."""
    grid = torch.tensor(grid, dtype=torch.float64, device=v.device)
    hi = torch.bucketize(v, grid).clamp(1, len(grid) - 1)
    below, above = v - grid[hi - 1], grid[hi] - v
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return grid[torch.where(up, hi, hi - 1)]


def _e4m3_grid():
    return [m * 2.0 ** -9 for m in range(8)] + [
        (8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8) if (e, m) != (15, 7)]


def _exact_scales(x, fmt, g):
    """[rows, groups] scales of 64-bit rows, the tensor's scale left out."""
    amax = x.view(x.shape[0], -1, GROUP[fmt]).abs().amax(-1)
    if fmt == "nvfp4":
        return _nearest((amax / (6.0 * g)).clamp(max=448.0), _e4m3_grid())
    e = torch.ceil(torch.log2(amax / TOP[fmt]))
    # log2 may land a hair beside a whole number: settle it by the definition itself
    e = torch.where(TOP[fmt] * torch.exp2(e - 1) >= amax, e - 1, e)
    e = torch.where(TOP[fmt] * torch.exp2(e) < amax, e + 1, e)
    return torch.exp2(e.clamp(min=-127.0))


def _exact_elements(x, s, fmt):
    q = x.view(x.shape[0], s.shape[1], -1) / s[..., None]
    q = torch.where(s[..., None] > 0, q, torch.zeros_like(q))
    grid = _e4m3_grid() if fmt == "mxfp8" else [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    return torch.sign(q) * _nearest(q.abs().clamp(max=grid[-1]), grid)


def _exact_tiles(s, empty):
    rt, gt = -(-s.shape[0] // 128), -(-s.shape[1] // 4)
    t = torch.full((rt, gt, 32, 4, 4), empty, dtype=torch.float64, device=s.device)
    rows = torch.arange(s.shape[0], device=s.device)[:, None]
    cols = torch.arange(s.shape[1], device=s.device)[None, :]
    t[rows // 128, cols // 4, rows % 32, rows // 32 % 4, cols % 4] = s
    return t


def _exact_decode(data, scales, fmt):
    rows = data.shape[0]
    if fmt == "mxfp8":
        q = data.double()
    else:
        q = torch.empty(rows, 2 * data.shape[1], dtype=torch.float64, device=data.device)
        for half, shift in ((0, 0), (1, 4)):
            c = (data.int() >> shift) & 15
            m = torch.where((c & 6) == 0, 0.5 * (c & 1), (1 + 0.5 * (c & 1)) * torch.exp2(((c & 6) // 2 - 1).double()))
            q[:, half::2] = torch.where(c >= 8, -m, m)
    r = torch.arange(rows, device=data.device)[:, None]
    k = torch.arange(q.shape[1] // GROUP[fmt], device=data.device)[None, :]
    s = scales.double()[r // 128, k // 4, r % 32, r // 32 % 4, k % 4]
    return (q.view(rows, s.shape[1], -1) * s[..., None]).view(rows, -1)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "norm":
        c = s["prefix"].double()
        if s["delta"] is not None:
            c = (c + s["delta"].double()).to(torch.bfloat16).double()
        y = c / torch.sqrt(c.square().mean(-1, keepdim=True) + EPS) * s["weight"].double()
        scale = _exact_scales(y, "mxfp8", None)
        return {"prefix": c, "q": _exact_elements(y, scale, "mxfp8").view(y.shape),
                "scales": _exact_tiles(scale, 2.0 ** -127), "norm": y if s["both"] else None}
    fmt = s["format"]
    if s["op"] == "quantize":
        x = s["x"].double()
        g = s["g"].double() if fmt == "nvfp4" else 1.0
        scale = _exact_scales(x, fmt, g)
        if fmt == "mxfp8":
            return {"q": _exact_elements(x, scale, fmt).view(x.shape), "scales": _exact_tiles(scale, 2.0 ** -127)}
        step = scale * g
        return {"values": (_exact_elements(x, step, fmt) * step[..., None]).view(x.shape)}
    out = _exact_decode(s["a"], s["a_scales"], fmt) @ _exact_decode(s["w"], s["w_scales"], fmt).t()
    if fmt == "nvfp4":
        out = out * (s["a_g"].double() * s["w_g"].double())
    return {"out": out}
