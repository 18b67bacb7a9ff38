"""The 8-bit calls as programs make them: first calls inside a graph capture,
replays on new inputs, other streams, host threads, matrices whose tensors change,
far offsets, random configurations."""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import attention_residual_fusion_gb300 as ar
from attention_residual_fusion_gb300 import _build, f8
from tests import f8_restatement as R
from tests.test_f8_gpu import (BF16_HALF, FORMS, Matrix, Rows, activations, backward_want, check_codes, equal_with_nan,
                               form, gated_want, product_want, quantized, within)

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    ar.device_status(clear=True)
    yield
    assert ar.device_status() == 0


def raw(t):
    return [t.data.view(torch.uint8), t.scales]


def tensors(x):
    """The plain tensors of a call's result."""
    if isinstance(x, torch.Tensor):
        return [x]
    return raw(x) if isinstance(x, f8.F8Tensor) else [t for y in x for t in tensors(y)]


CALLS = {
    "rows": lambda s: f8.quantize(s["x"]),
    "both": lambda s: f8.quantize(s["x"], transposed=True),
    "square": lambda s: f8.quantize(s["x"], 128, transposed=True),
    "back": lambda s: f8.dequantize(s["a"]),
    "narrow": lambda s: f8.matmul(s["a"], s["w"], kernel=f8.KERNEL_NARROW),
    "wide": lambda s: f8.matmul(s["a"], s["w"], kernel=f8.KERNEL_WIDE, dtype=torch.float32),
    "gradient": lambda s: f8.matmul(s["a"], s["a"], dtype=torch.float32),
    "pair": lambda s: f8.matmul(s["a"], s["w"], plus=(s["a"], s["v"])),
    "gated": lambda s: f8.gated(s["a"], s["w"], s["v"], save=True),
    "gated wide": lambda s: f8.gated(s["a"], s["w"], s["v"], "gelu", kernel=f8.KERNEL_WIDE, dtype=torch.bfloat16),
    "backward": lambda s: f8.gated_backward(s["x"], s["a"], s["b"]),
}


def state(T=200, H=512, F=260, seed=1):
    s = {"x": activations(T, H, seed)}
    s["a"], s["b"] = (f8.quantize(activations(T, H, seed + i)) for i in (1, 2))
    s["w"], s["v"] = (f8.quantize(activations(F, H, seed + i, 0.05), 128) for i in (3, 4))
    return s


CHILD = r"""
import sys
import torch
import attention_residual_fusion_gb300 as ar
from attention_residual_fusion_gb300 import f8
torch.manual_seed(5)
T, H, F = 200, 512, 260
def made(rows, cols, block=1):  # by hand, so that the captured call is the process's first
    codes = torch.randint(0, 120, (rows, cols), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    return f8.F8Tensor(codes, torch.rand(f8.scales_shape(rows, cols, block), device="cuda") + 0.01, block)
s = dict(x=torch.randn(T, H, device="cuda").bfloat16(), a=made(T, H), b=made(T, H), w=made(F, H, 128), v=made(F, H, 128))
CALLS = {
    "both": lambda: f8.quantize(s["x"], transposed=True),
    "narrow": lambda: f8.matmul(s["a"], s["w"], kernel=1),
    "wide": lambda: f8.matmul(s["a"], s["w"], kernel=2),
    "gated": lambda: f8.gated(s["a"], s["w"], s["v"], save=True),
    "gated wide": lambda: f8.gated(s["a"], s["w"], s["v"], save=True, kernel=2),
    "backward": lambda: f8.gated_backward(s["x"], s["a"], s["b"]),
}
def tensors(x):
    if isinstance(x, torch.Tensor):
        return [x]
    return [x.data.view(torch.uint8), x.scales] if isinstance(x, f8.F8Tensor) else [t for y in x for t in tensors(y)]
call = CALLS[sys.argv[1]]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = tensors(call())
g.replay()
torch.cuda.synchronize()
want = tensors(call())
torch.cuda.synchronize()
assert all(torch.equal(x, y) for x, y in zip(got, want))
assert ar.device_status() == 0
print("ok")
"""


@pytest.mark.parametrize("what", ["both", "narrow", "wide", "gated", "gated wide", "backward"])
def test_first_call_inside_graph_capture(what):
    r = subprocess.run([sys.executable, "-c", CHILD, what], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stderr[-3000:]


@pytest.mark.parametrize("what", CALLS)
def test_replays_read_what_the_inputs_then_hold(what):
    """A captured call on other contents of the same buffers, between eager calls, twice; and two graphs at once."""
    s, other = state(seed=1), state(seed=50)
    keep = {k: [t.clone() for t in tensors(v)] for k, v in s.items()}
    want_one = [t.clone() for t in tensors(CALLS[what](s))]
    want_two = [t.clone() for t in tensors(CALLS[what](other))]
    graphs, got = [], []
    for st in (s, other):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(tensors(CALLS[what](st)))
        graphs.append(g)
    for _ in range(2):
        for t in got[0] + got[1]:
            t.zero_()
        for g in graphs:
            g.replay()
        assert all(torch.equal(a, b) for a, b in zip(got[0], want_one))
        assert all(torch.equal(a, b) for a, b in zip(got[1], want_two))
    # on two streams, as far as they overlap
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(5):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got[0] + got[1], want_one + want_two))
    # the first graph's buffers given the second's contents
    for k in s:
        for a, b in zip(tensors(s[k]), tensors(other[k])):
            a.copy_(b)
    graphs[0].replay()
    assert all(torch.equal(a, b) for a, b in zip(got[0], want_two))
    for k in s:
        for a, b in zip(tensors(s[k]), keep[k]):
            a.copy_(b)
    graphs[0].replay()
    assert all(torch.equal(a, b) for a, b in zip(got[0], want_one))


@pytest.mark.parametrize("what", CALLS)
def test_on_a_given_stream(what):
    """The stream argument is where the call runs: behind the stream's earlier work, results seen through it."""
    s = state()
    want = [t.clone() for t in tensors(CALLS[what](s))]
    stream = torch.cuda.Stream()
    name = {"rows": "x", "both": "x", "square": "x", "backward": "x"}.get(what, "a")
    source = [t.clone() for t in tensors(s[name])]
    torch.cuda.synchronize()
    calls = dict(quantize=f8.quantize, dequantize=f8.dequantize, matmul=f8.matmul, gated=f8.gated,
                 gated_backward=f8.gated_backward)
    with torch.cuda.stream(stream):  # a long fill first, then the inputs
        big = torch.empty(1 << 30, dtype=torch.uint8, device="cuda")
        for t in tensors(s[name]):
            t.zero_()
        big.fill_(1)
        for t, v in zip(tensors(s[name]), source):
            t.copy_(v)
    try:  # the same call with stream=, from the default stream
        for k, fn in calls.items():
            setattr(f8, k, lambda *a, fn=fn, **kw: fn(*a, stream=stream, **kw))
        got = tensors(CALLS[what](s))
    finally:
        for k, fn in calls.items():
            setattr(f8, k, fn)
    stream.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_chained_with_pdl():
    """A block's chain with every call allowed to start early."""
    s2 = {k: f8.quantize(activations(768, 768, 20 + i, 0.04), 128) for i, k in enumerate("wvd")}

    def chain(pdl):
        x = f8.quantize(activations(64, 768, 9), pdl=pdl)
        out = []
        for _ in range(4):
            h = f8.gated(x, s2["w"], s2["v"], pdl=pdl)
            y = f8.matmul(h, s2["d"], pdl=pdl)
            x = f8.quantize(y, pdl=pdl)
            out += tensors(h) + [y]
        return out
    torch.cuda.synchronize()
    want = chain(False)
    got = chain(True)
    # bit for bit (the chain's values may grow out of range)
    assert all(torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)) for a, b in zip(got, want))
    assert torch.isfinite(want[1]).all() and bool((want[2].float() != 0).any())


def test_calls_from_concurrent_host_threads():
    errors = []

    def worker(i):
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                s = state(T=100 + 60 * i, seed=10 * i)
                want = {k: [t.clone() for t in tensors(c(s))] for k, c in CALLS.items()}
                for _ in range(10):
                    for k, c in CALLS.items():
                        got = tensors(c(s))
                        st.synchronize()
                        assert all(torch.equal(a, b) for a, b in zip(got, want[k])), k
        except Exception as e:  # reported on the main thread
            errors.append(repr(e))

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(5)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


# ---- matrices -------------------------------------------------------------------------


def test_parts_replaced_between_calls():
    """A matrix keeps its tensors, not their addresses."""
    a, b = (f8.quantize(activations(200, 512, i)) for i in (1, 2))
    w = f8.quantize(activations(70, 512, 3), 128)
    want = f8.matmul(b, w)
    old = f8.matmul(a, w)
    a.data.set_(b.data.clone())
    a.scales.set_(b.scales.clone())
    got = f8.matmul(a, w)
    assert torch.equal(got, want) and not torch.equal(got, old)
    a.scales.untyped_storage().resize_(16)
    with pytest.raises(ValueError):
        f8.matmul(a, w)


def test_views_of_larger_matrices():
    """Rows, and column blocks from 128-column and 16-byte boundaries on, of one buffer."""
    q = f8.quantize(activations(300, 1024, 1))
    w = f8.quantize(activations(256, 1024, 2), 128)
    part = f8.F8Tensor(q.data[64:200, 256:768], q.scales[2:6, 64:200])
    wpart = f8.F8Tensor(w.data[128:, 256:768], w.scales[1:, 2:6], 128)
    va, vw = R.values(q.data, q.scales, 1)[64:200, 256:768], R.values(w.data, w.scales, 128)[128:, 256:768]
    for kw in (dict(kernel=f8.KERNEL_NARROW), dict(kernel=f8.KERNEL_WIDE)):
        want = va @ vw.t()
        bound = R.product_bound(va.abs() @ vw.abs().t(), 512)
        within(f8.matmul(part, wpart, dtype=torch.float32, **kw), want, bound)
    with pytest.raises(ar.AttnResError):  # rows of scales that start between 16-byte boundaries
        f8.matmul(f8.F8Tensor(q.data[1:200], q.scales[:, 1:200]), w)


@pytest.mark.parametrize("bad", [
    lambda q: f8.F8Tensor(q.data.t(), q.scales), lambda q: f8.F8Tensor(q.data.view(torch.uint8), q.scales),
    lambda q: f8.F8Tensor(q.data, q.scales.double()), lambda q: f8.F8Tensor(q.data, q.scales[:, :-1]),
    lambda q: f8.F8Tensor(q.data, q.scales, 128), lambda q: f8.F8Tensor(q.data, q.scales, 2),
    lambda q: f8.F8Tensor(q.data, q.scales.cpu()), lambda q: f8.F8Tensor(q.data[0], q.scales),
    lambda q: f8.F8Tensor(q.data, torch.empty(q.scales.shape[::-1], device="cuda").t())])
def test_matrices_that_are_none(bad):
    with pytest.raises(ValueError):
        bad(f8.quantize(activations(40, 256, 1)))


def test_refusals_of_the_binding():
    q, w = f8.quantize(activations(40, 256, 1)), f8.quantize(activations(72, 256, 2), 128)
    x = activations(40, 256, 3)
    empty = f8.F8Tensor.empty
    for call in (
            lambda: f8.quantize(x.float()), lambda: f8.quantize(x.t()), lambda: f8.quantize(x, 64),
            lambda: f8.quantize(x, out=empty(40, 255)), lambda: f8.quantize(x, out=empty(40, 256, 128)),
            lambda: f8.quantize(x, transposed=empty(40, 256)), lambda: f8.quantize(x, out=x),
            lambda: f8.dequantize(q, x[:39]), lambda: f8.matmul(w, q), lambda: f8.matmul(q, empty(72, 255, 128)),
            lambda: f8.matmul(q, w, dtype=torch.float16), lambda: f8.matmul(q, w, dtype="bf16"),
            lambda: f8.matmul(q, w, add=True), lambda: f8.matmul(q, w, torch.empty(40, 72, device="cuda").bfloat16(), add=True),
            lambda: f8.matmul(q, w, torch.empty(40, 71, device="cuda")), lambda: f8.matmul(q, w, plus=(q, q)),
            lambda: f8.matmul(q, w, plus=(empty(41, 256), w)), lambda: f8.matmul(q, w, kernel=16),
            lambda: f8.gated(q, w, q), lambda: f8.gated(q, w, empty(71, 256, 128)), lambda: f8.gated(q, w, w, "relu"),
            lambda: f8.gated(q, w, w, save=(empty(40, 72),)), lambda: f8.gated(q, w, w, out=empty(40, 72), dtype=torch.bfloat16),
            lambda: f8.gated(q, w, w, dtype=torch.float32), lambda: f8.gated(q, w, w, out="here"),
            lambda: f8.gated_backward(x, q, w), lambda: f8.gated_backward(x[:39], q, q),
            lambda: f8.gated_backward(x, q, q, out=[empty(40, 256)] * 2), lambda: f8.gated_backward(x.float(), q, q),
            lambda: f8.matmul(q, w, stream="s")):
        with pytest.raises(ValueError):
            call()
    for call in (
            lambda: f8.matmul(q, w, kernel=3), lambda: f8.matmul(q, w, split=2), lambda: f8.matmul(q, w, kernel=2, split=1),
            lambda: f8.matmul(q, w, kernel=1, split=3), lambda: f8.gated(q, w, w, kernel=9),
            lambda: f8.gated_backward(x, q, q, out=[q, empty(40, 256)], transposed=False)):
        with pytest.raises(ar.AttnResError):
            call()


def test_far_offsets():
    """Codes and rows beyond 2^31 elements and bytes of their buffers' starts."""
    rows, cols = 70000, 65536
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    some = [0, 32767, 32768, 65535, 69999]
    x[some] = activations(len(some), cols, 1)
    q = f8.quantize(x)
    back = f8.dequantize(q)
    codes, scales = R.quantize(x[some], 1)
    assert torch.equal(q.data[some].view(torch.uint8), codes) and equal_with_nan(q.scales[:, some], scales)
    assert torch.equal(back[some].double(), R.values(codes, scales, 1).float().bfloat16().double())
    del back, x
    w = quantized(130, cols, 2, 128, scale=0.01)
    va = R.values(codes, scales.contiguous(), 1)
    want = va @ w.values().t()
    bound = R.product_bound(va.abs() @ w.values().abs().t(), cols)
    out = f8.matmul(q, w.t, dtype=torch.float32)  # [70000, 130]: rows of the operand far behind its start
    within(out[some], want, bound)
    assert bool((out[1:100] == 0).all())
    # as weights too: 70000 columns of a result
    a = quantized(40, cols, 3, scale=0.01)
    out = f8.matmul(a.t, q, dtype=torch.float32)
    within(out[:, some], a.values() @ va.t(), R.product_bound(a.values().abs() @ va.abs().t(), cols))
    # and results beyond 2^32 bytes, from rows that lie far apart
    far = torch.empty(5, 1 << 30, dtype=torch.uint8, device="cuda")[:, :256].view(torch.float8_e4m3fn)
    src = f8.quantize(activations(5, 256, 4))
    far.view(torch.uint8).copy_(src.data.view(torch.uint8))
    b = f8.F8Tensor(far, src.scales)
    v = f8.quantize(activations(300, 256, 5), 128)
    for kw in (dict(kernel=1), dict(kernel=2)):
        assert torch.equal(f8.matmul(b, v, **kw), f8.matmul(src, v, **kw))
    wide = torch.empty(5, 1 << 29, dtype=torch.bfloat16, device="cuda")[:, :300]
    f8.matmul(b, v, wide)
    assert torch.equal(wide, f8.matmul(src, v))


# ---- random configurations ------------------------------------------------------------


def log_int(rng, lo, hi):
    return int(round(np.exp(rng.uniform(np.log(lo), np.log(hi)))))


@pytest.mark.parametrize("seed", range(40))
def test_random_products(seed):
    rng = np.random.default_rng(1000 + seed)
    m, n, k = (log_int(rng, 1, 1500) for _ in range(3))
    block = 1 if seed % 3 == 0 else 128
    pairs = []
    for i in range(1 + seed % 2):
        kk = k if i == 0 else log_int(rng, 1, 1500)
        pairs.append((quantized(m, kk, seed + i, pad=int(rng.integers(3))),
                      quantized(n, kk, seed + 50 + i, block, pad=int(rng.integers(3)), scale=0.05)))
    cols = sum(128 * R.blocks(a.cols) for a, _ in pairs)
    want, bound = product_want(pairs, cols)
    plus = None if len(pairs) == 1 else (pairs[1][0].t, pairs[1][1].t)
    for kw in (dict(), form(FORMS[int(rng.integers(len(FORMS) - 1))], cols)):
        out = Rows(m, n, 8 * int(rng.integers(3)))
        f8.matmul(pairs[0][0].t, pairs[0][1].t, out.t, plus=plus, pdl=bool(rng.integers(2)), **kw)
        within(out.t, want, bound + BF16_HALF * (want.abs() + bound))
        assert out.intact()


@pytest.mark.parametrize("seed", range(30))
def test_random_blocks(seed):
    rng = np.random.default_rng(2000 + seed)
    T, F, H = log_int(rng, 1, 700), log_int(rng, 1, 700), log_int(rng, 1, 900)
    act = ["silu", "gelu"][seed % 2]
    x = quantized(T, H, seed, pad=int(rng.integers(3)))
    wg, wu = (quantized(F, H, seed + i, 128, pad=int(rng.integers(3)), scale=H ** -0.5) for i in (1, 2))
    g, u, h, eg, eu, eh = gated_want(x, wg, wu, act)
    out = [Matrix(T, F, 1, int(rng.integers(3))) for _ in range(3)]
    f8.gated(x.t, wg.t, wu.t, act, out[0].t, save=(out[1].t, out[2].t), pdl=bool(rng.integers(2)))
    for got, want, e in zip(out, (h, g, u), (eh, eg, eu)):
        check_codes(got, want, e, "gated")
    dh = Rows(T, F, 8 * int(rng.integers(3)), activations(T, F, seed + 7, 10.0 ** rng.uniform(-5, 1)))
    grads = [Matrix(T, F, 1, int(rng.integers(3))) for _ in range(2)] + [Matrix(F, T, 1, int(rng.integers(3))) for _ in range(3)]
    f8.gated_backward(dh.t, out[1].t, out[2].t, act, [t.t for t in grads])
    (dg, e1), (du, e2), (hh, e3) = backward_want(dh.t, out[1].values(), out[2].values(), act)
    for got, want, e in zip(grads, (dg, du, dg.t(), du.t(), hh.t()), (e1, e2, e1.t(), e2.t(), e3.t())):
        check_codes(got, want.contiguous(), e.contiguous(), "backward")


@pytest.mark.parametrize("seed", range(30))
def test_random_rows(seed):
    rng = np.random.default_rng(3000 + seed)
    rows, cols = log_int(rng, 1, 600), log_int(rng, 1, 2000)
    block = [1, 128][seed % 2]
    x = Rows(rows, cols, 8 * int(rng.integers(4)), activations(rows, cols, seed, scale=10.0 ** rng.uniform(-30, 30)))
    q, t = Matrix(rows, cols, block, int(rng.integers(3))), Matrix(cols, rows, block, int(rng.integers(3)))
    both = bool(rng.integers(2))
    f8.quantize(x.t, block, q.t, transposed=t.t if both else None)
    for got, src in ((q, x.t), (t, x.t.t()))[:1 + both]:
        codes, scales = R.quantize(src, block)
        assert equal_with_nan(got.scales, scales) and torch.equal(got.codes, codes)
        assert got.intact()
    assert x.intact()
