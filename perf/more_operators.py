"""Measured cases of the feed-forward operators in 8 bits (attention_residual_fusion_gb300.f8).

Operators:

* ``quantize``  bf16 rows to e4m3 codes, with a scale for each row and 128 columns ("rows") or for each
                block of 128 x 128 ("square", for weights); with ``both`` the transposed matrix as well;
* ``product``   out = a w^T of two such matrices, the sums in 32 bits: ``square`` (activations times
                weights), ``pair`` (the sum of two such products: the gradient of the input of gate and
                up) and ``rows`` (both with a scale for each row and 128 columns: the gradient of
                weights, summed over tokens, in fp32);
* ``gated``     h = act(x gate^T) * (x up^T), h in codes; with ``save`` gate's and up's projections in
                codes too, for the backward pass;
* ``backward``  from h's gradient and those codes the gradients of both projections in codes, by rows
                and transposed, and the transposed h.

A group of values has the scale amax / 448 (at least 2^-126; 1 for zeros), its codes are the values over
the scale, rounded to e4m3.  Scales of rows lie by groups first, [ceil(cols / 128), rows], those of blocks
[ceil(rows / 128), ceil(cols / 128)].

``run`` computes the operators in plain torch operations, or with ``own`` set by the framework's calls.
"""
import math

import torch

own = False

H = 7168  # the row width that the framework's tuned kernels are built for
BLOCK = 128
TOP = 448.0  # the largest e4m3 value
SMALLEST = 2.0 ** -126
GELU = 2.0 * math.sqrt(2.0 / math.pi)


# ---- cases ---------------------------------------------------------------------


def listed():
    def quant(name, rows, cols, kind="rows", both=False, pad=0):
        return dict(name=name, op="quantize", rows=rows, cols=cols, kind=kind, both=both, pad=pad)

    def product(name, rows, n, cols, kind="square"):
        return dict(name=name, op="product", rows=rows, n=n, cols=cols, kind=kind)

    def gated(name, rows, n, cols, act="silu", save=False):
        return dict(name=name, op="gated", rows=rows, n=n, cols=cols, act=act, save=save)

    def backward(name, rows, n, act="silu"):
        return dict(name=name, op="backward", rows=rows, n=n, act=act)

    return [
        # the activations of a few speculative tokens before a projection
        quant("quantize 4x7168", 4, H),
        # a training step's activations: rows for the projection, transposed for the weights' gradient
        quant("quantize both 8192x7168", 8192, H, both=True),
        # decode of one token: the product is the reading of the weights
        product("product 1 token", 1, H, H),
        # ragged in every direction: the last batch of a chunked prefill
        product("product 333 odd", 333, 2050, 7200),
        # long prefill, the framework's largest number of tokens, against a down-projection
        product("product 8192", 8192, H, 4096),
        # the input's gradient behind gate and up
        product("product pair 4096", 4096, H, 2048, kind="pair"),
        # the gradient of a weight matrix over a ragged number of tokens
        product("product gradient 4096x7168", 4096, H, 8190, kind="rows"),
        # a decode batch against gate and up
        gated("gated 64 tokens", 64, 4096, H),
        # a ragged training batch of a narrow block, the other activation
        gated("gated 1003 odd", 1003, 2000, 2080, act="gelu", save=True),
        # a training step's feed-forward block on a long batch
        gated("gated train 8192", 8192, 4096, H, save=True),
        # the backward pass of the narrow block
        backward("backward 1003 odd", 1003, 2000, act="gelu"),
        # and of the wide one
        backward("backward 8192", 8192, 4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "gated", "backward"])
    rows = _log(rng, 1, 8192)
    act = rng.choice(["silu", "gelu"])
    if op == "quantize":
        cols = 8 * _log(rng, 4, 2048)
        while rows * cols > 8192 * H:
            rows = max(1, rows // 2)
        return dict(op=op, rows=rows, cols=cols, kind=rng.choice(["rows", "square"]), both=rng.random() < 0.5,
                    pad=rng.choice([0, 0, 8, 64]))
    if op == "backward":
        n = 16 * _log(rng, 4, 512)
        while rows * n > 8192 * 4096:
            rows = max(1, rows // 2)
        return dict(op=op, rows=rows, n=n, act=act)
    if op == "gated":
        n, cols = 16 * _log(rng, 4, 512), 16 * _log(rng, 8, 512)
        while rows * n * cols > 8192 * 4096 * H // 2:
            rows = max(1, rows // 2)
        return dict(op=op, rows=rows, n=n, cols=cols, act=act, save=rng.random() < 0.5)
    kind = rng.choice(["square", "square", "pair", "rows"])
    n, cols = _log(rng, 64, 16384), _log(rng, 100, 16384)
    while rows * n * cols > 8192 * 4096 * H // 2:
        rows = max(1, rows // 2)
        cols = cols if rows > 1 else max(100, cols // 2)
    return dict(op=op, rows=rows, n=n, cols=cols, kind=kind)


def _groups(n):
    return -(-n // BLOCK)


def _held(rows, cols, kind):
    """Bytes of a matrix's codes and scales."""
    return rows * cols + 4 * _groups(cols) * (rows if kind == "rows" else _groups(rows))


def work(case):
    rows, op = case["rows"], case["op"]
    if op == "quantize":
        cols, kind = case["cols"], case["kind"]
        moved = 2 * rows * cols + _held(rows, cols, kind) + (_held(cols, rows, kind) if case["both"] else 0)
        return {"bytes": moved, "flops": 4 * rows * cols * (1 + case["both"])}
    n = case["n"]
    if op == "backward":
        moved = 2 * rows * n + 4 * _held(rows, n, "rows") + 3 * _held(n, rows, "rows")
        return {"bytes": moved, "flops": 30 * rows * n}
    cols = case["cols"]
    if op == "gated":
        moved = _held(rows, cols, "rows") + 2 * _held(n, cols, "square") + (3 if case["save"] else 1) * _held(rows, n, "rows")
        return {"bytes": moved, "flops": 4 * rows * n * cols}
    terms = 2 if case["kind"] == "pair" else 1
    moved = terms * (_held(rows, cols, "rows") + _held(n, cols, "rows" if case["kind"] == "rows" else "square"))
    moved += (4 if case["kind"] == "rows" else 2) * rows * n
    return {"bytes": moved, "flops": 2 * terms * rows * n * cols}


# ---- the format in plain torch ---------------------------------------------------


def _filled(x, rows, cols):
    """x with zeros behind its last row and column."""
    full = torch.zeros(rows, cols, dtype=x.dtype, device=x.device)
    full[:x.shape[0], :x.shape[1]] = x
    return full


def _quantize(x, kind):
    """fp32 [r, c] -> (e4m3 codes [r, c], scales in the kind's order)."""
    r, c = x.shape
    tall = 1 if kind == "rows" else BLOCK
    rb, cb = -(-r // tall), _groups(c)
    xb = _filled(x, rb * tall, cb * BLOCK).view(rb, tall, cb, BLOCK)
    amax = xb.abs().amax((1, 3))
    s = (amax / TOP).clamp(min=SMALLEST)
    s = torch.where(amax == 0, torch.ones_like(s), s)
    v = (xb / s[:, None, :, None]).clamp(-TOP, TOP).to(torch.float8_e4m3fn)
    return v.view(rb * tall, cb * BLOCK)[:r, :c].contiguous(), (s.t().contiguous() if kind == "rows" else s)


def _values(codes, scales, kind):
    """The fp32 values of codes and scales."""
    r, c = codes.shape
    s = scales.t() if kind == "rows" else scales.repeat_interleave(BLOCK, 0)[:r]
    return codes.float() * s.repeat_interleave(BLOCK, 1)[:, :c]


def _act(g, act):
    """act(g) and its derivative."""
    z = g if act == "silu" else GELU * (g + 0.044715 * g * g * g)
    dz = 1.0 if act == "silu" else GELU * (1.0 + 3 * 0.044715 * g * g)
    p = 1.0 / (1.0 + torch.exp(-z))
    return g * p, p + g * p * (1.0 - p) * dz


# ---- inputs ------------------------------------------------------------------------


def _activations(gen, rows, cols, pad=0, scale=1.0):
    """N(0, scale) with one value in a hundred 20 times as large, bf16, rows in a buffer of cols + pad."""
    x = scale * torch.randn(rows, cols + pad, generator=gen, device="cuda")
    x *= 1.0 + 19.0 * (torch.rand(rows, cols + pad, generator=gen, device="cuda") < 0.01)
    return x.to(torch.bfloat16)[:, :cols]


def _weights(gen, rows, cols):
    return torch.randn(rows, cols, generator=gen, device="cuda").mul_(cols ** -0.5).to(torch.bfloat16)


def _stored(x, kind):
    """Codes whose rows lie a multiple of 16 bytes apart, as a program allocates them, and scales whose
    rows of groups do as well."""
    codes, scales = _quantize(x.float(), kind)
    r, c = codes.shape
    data = torch.zeros(r, -(-c // 16) * 16, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)[:, :c]
    data.copy_(codes)
    if kind == "rows":
        held = torch.zeros(scales.shape[0], -(-r // 4) * 4, device="cuda")[:, :r]
        scales = held.copy_(scales)
    return data, scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, rows = case["op"], case["rows"]
    s = dict(case)
    if op == "quantize":
        # columns in steps of 8, so that bf16 rows begin on 16-byte boundaries
        s["x"] = _weights(gen, rows, case["cols"] + case["pad"])[:, :case["cols"]] if case["kind"] == "square" else \
            _activations(gen, rows, case["cols"], case["pad"])
        return s
    n = case["n"]
    if op == "backward":
        s["dh"] = _activations(gen, rows, n, scale=1e-3)
        s["gate"] = _stored(_activations(gen, rows, n), "rows")
        s["up"] = _stored(_activations(gen, rows, n), "rows")
        return s
    cols = case["cols"]
    if op == "gated":
        s["x"] = _stored(_activations(gen, rows, cols), "rows")
        s["gate"] = _stored(_weights(gen, n, cols), "square")
        s["up"] = _stored(_weights(gen, n, cols), "square")
        return s
    if case["kind"] == "rows":
        s["a"] = _stored(_activations(gen, rows, cols, scale=1e-3), "rows")
        s["w"] = _stored(_activations(gen, n, cols), "rows")
        return s
    for i in range(2 if case["kind"] == "pair" else 1):
        s["a" + "2" * i] = _stored(_activations(gen, rows, cols), "rows")
        s["w" + "2" * i] = _stored(_weights(gen, n, cols), "square")
    return s


# ---- the passes ----------------------------------------------------------------------


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from attention_residual_fusion_gb300 import f8

    op = s["op"]
    if op == "quantize":
        block = 1 if s["kind"] == "rows" else BLOCK
        if s["both"]:
            q, t = f8.quantize(s["x"], block, transposed=True)
            return {"q": q.data, "scales": q.scales, "t": t.data, "t_scales": t.scales}
        q = f8.quantize(s["x"], block)
        return {"q": q.data, "scales": q.scales}
    if op == "backward":
        dg, du, dgt, dut, ht = f8.gated_backward(s["dh"], f8.F8Tensor(*s["gate"]), f8.F8Tensor(*s["up"]), s["act"])
        return {"dg": dg.data, "dg_scales": dg.scales, "du": du.data, "du_scales": du.scales,
                "dgt": dgt.data, "dgt_scales": dgt.scales, "dut": dut.data, "dut_scales": dut.scales,
                "ht": ht.data, "ht_scales": ht.scales}
    if op == "gated":
        x, gate, up = f8.F8Tensor(*s["x"]), f8.F8Tensor(*s["gate"], BLOCK), f8.F8Tensor(*s["up"], BLOCK)
        if not s["save"]:
            h = f8.gated(x, gate, up, s["act"])
            return {"h": h.data, "h_scales": h.scales}
        h, g, u = f8.gated(x, gate, up, s["act"], save=True)
        return {"h": h.data, "h_scales": h.scales, "g": g.data, "g_scales": g.scales, "u": u.data, "u_scales": u.scales}
    block = 1 if s["kind"] == "rows" else BLOCK
    a, w = f8.F8Tensor(*s["a"]), f8.F8Tensor(*s["w"], block)
    if s["kind"] == "rows":
        return {"out": f8.matmul(a, w, dtype=torch.float32)}
    plus = (f8.F8Tensor(*s["a2"]), f8.F8Tensor(*s["w2"], block)) if s["kind"] == "pair" else None
    return {"out": f8.matmul(a, w, plus=plus)}


def _run_plain(s):
    op = s["op"]
    if op == "quantize":
        x = s["x"].float()
        q, scales = _quantize(x, s["kind"])
        if not s["both"]:
            return {"q": q, "scales": scales}
        t, t_scales = _quantize(x.t(), s["kind"])
        return {"q": q, "scales": scales, "t": t, "t_scales": t_scales}
    if op == "backward":
        g, u, dh = _values(*s["gate"], "rows"), _values(*s["up"], "rows"), s["dh"].float()
        a, da = _act(g, s["act"])
        dg, du, h = dh * u * da, dh * a, a * u
        out = {}
        for name, v in (("dg", dg), ("du", du), ("dgt", dg.t()), ("dut", du.t()), ("ht", h.t())):
            out[name], out[name + "_scales"] = _quantize(v, "rows")
        return out
    if op == "gated":
        x = _values(*s["x"], "rows")
        g, u = x @ _values(*s["gate"], "square").t(), x @ _values(*s["up"], "square").t()
        out = {}
        out["h"], out["h_scales"] = _quantize(_act(g, s["act"])[0] * u, "rows")
        if s["save"]:
            out["g"], out["g_scales"] = _quantize(g, "rows")
            out["u"], out["u_scales"] = _quantize(u, "rows")
        return out
    if s["kind"] == "rows":
        return {"out": _values(*s["a"], "rows") @ _values(*s["w"], "rows").t()}
    out = _values(*s["a"], "rows") @ _values(*s["w"], "square").t()
    if s["kind"] == "pair":
        out += _values(*s["a2"], "rows") @ _values(*s["w2"], "square").t()
    return {"out": out.to(torch.bfloat16)}


# ---- the definitions in 64 bits --------------------------------------------------------


def _e4m3_grid():
    return [m * 2.0 ** -9 for m in range(8)] + [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)][:-1]


def _exact_codes(v, square=False):
    """Element values and scales of fp64 [r, c], a row at a time or (square) a block at a time."""
    r, c = v.shape
    col = torch.arange(c, device=v.device) // BLOCK
    row = torch.arange(r, device=v.device) // (BLOCK if square else 1)
    top = torch.zeros(int(row[-1]) + 1, int(col[-1]) + 1, dtype=torch.float64, device=v.device)
    cell = row[:, None] * top.shape[1] + col[None, :]
    top.view(-1).scatter_reduce_(0, cell.reshape(-1), v.abs().reshape(-1), "amax")
    s = torch.where(top > 0, (top / TOP).clamp(min=SMALLEST), torch.ones_like(top))
    x = v / s.view(-1)[cell]
    grid = torch.tensor(_e4m3_grid(), dtype=torch.float64, device=v.device)
    a = x.abs().clamp(max=TOP)
    hi = torch.bucketize(a, grid).clamp(1, len(grid) - 1)
    below, above = a - grid[hi - 1], grid[hi] - a
    near = grid[torch.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, hi - 1)]
    return torch.sign(x) * near, (s if square else s.t())


def _exact_values(pair, square=False):
    codes, s = pair
    r, c = codes.shape
    row = torch.arange(r, device=codes.device) // (BLOCK if square else 1)
    col = torch.arange(c, device=codes.device) // BLOCK
    return codes.double() * ((s if square else s.t()).double()[row][:, col])


def _exact_act(g, act):
    if act == "silu":
        p = torch.sigmoid(g)
        return g * p, p * (1 + g * (1 - p))
    # (1 + tanh(y)) / 2 as the sigmoid of 2 y: 1 + tanh loses all of small values
    k = math.sqrt(8 / math.pi)
    p = torch.sigmoid(k * (g + 0.044715 * g ** 3))
    return g * p, p + g * p * (1 - p) * k * (1 + 3 * 0.044715 * g * g)


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    out = {}

    def put(name, v, square=False):
        out[name], out[("scales" if name == "q" else name + "_scales")] = _exact_codes(v, square)

    if op == "quantize":
        x = s["x"].double()
        put("q", x, s["kind"] == "square")
        if s["both"]:
            put("t", x.t(), s["kind"] == "square")
        return out
    if op == "backward":
        g, u, dh = _exact_values(s["gate"]), _exact_values(s["up"]), s["dh"].double()
        a, da = _exact_act(g, s["act"])
        put("dg", dh * u * da)
        put("du", dh * a)
        put("dgt", (dh * u * da).t())
        put("dut", (dh * a).t())
        put("ht", (a * u).t())
        return out
    if op == "gated":
        x = _exact_values(s["x"])
        g, u = x @ _exact_values(s["gate"], True).t(), x @ _exact_values(s["up"], True).t()
        put("h", _exact_act(g, s["act"])[0] * u)
        if s["save"]:
            put("g", g)
            put("u", u)
        return out
    square = s["kind"] != "rows"
    out["out"] = _exact_values(s["a"]) @ _exact_values(s["w"], square).t()
    if s["kind"] == "pair":
        out["out"] += _exact_values(s["a2"]) @ _exact_values(s["w2"], True).t()
    return out
