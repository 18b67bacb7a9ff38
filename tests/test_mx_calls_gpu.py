"""The microscaled calls as programs make them: first calls inside a graph
capture, calls from several host threads, and random configurations."""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import attention_residual_fusion_gb300 as ar
from attention_residual_fusion_gb300 import _build, mx
from tests import mx_restatement as R
from tests.test_mx_gpu import (FORMATS, FORMS, Matrix, Rows, activations, check_norm, check_product, f64, form,
                               matrix_values, random_matrix)

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    ar.device_status(clear=True)
    yield
    assert ar.device_status() == 0


CHILD = r"""
import sys
import torch
import attention_residual_fusion_gb300 as ar
from attention_residual_fusion_gb300 import mx
what, fmt, m, n, k, kernel = sys.argv[1], sys.argv[2], *(int(a) for a in sys.argv[3:7])
torch.manual_seed(5)
if what == "matmul":  # codes made by hand, so that the captured call is the process's first
    def matrix(rows):
        cols = k if fmt == "mxfp8" else k // 2
        data = torch.randint(0, 120, (rows, cols), dtype=torch.uint8, device="cuda")
        shape = mx.scales_shape(fmt, rows, k)
        scales = torch.randint(50, 60, shape, dtype=torch.uint8, device="cuda") + (0 if fmt == "nvfp4" else 70)
        if fmt == "mxfp8":
            data = data.view(torch.float8_e4m3fn)
        kind = torch.float8_e4m3fn if fmt == "nvfp4" else torch.float8_e8m0fnu
        return mx.MxTensor(data, scales.view(kind), fmt)
    a, w = matrix(m), matrix(n)
    def call():
        return [mx.matmul(a, w, kernel=kernel)]
else:
    x = torch.randn(m, k, device="cuda").bfloat16()
    wt = torch.ones(k, dtype=torch.bfloat16, device="cuda")
    def call():
        if what == "norm":
            y = torch.empty_like(x)
            q = mx.add_rms_norm(x, None, wt, format=fmt, norm_out=y)
            return [q.data.view(torch.uint8), q.scales.view(torch.uint8), y]
        q = mx.quantize(x, fmt)
        return [q.data.view(torch.uint8), q.scales.view(torch.uint8), mx.dequantize(q)]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = call()
g.replay()
torch.cuda.synchronize()
want = call()
torch.cuda.synchronize()
for x, y in zip(got, want):
    assert torch.equal(x, y)
assert ar.device_status() == 0
print("ok")
"""


@pytest.mark.parametrize("what,fmt,m,n,k,kernel", [
    ("matmul", "mxfp4", 1, 300, 1024, 0), ("matmul", "nvfp4", 100, 300, 1024, 1), ("matmul", "mxfp8", 600, 700, 512, 2),
    ("matmul", "mxfp4", 600, 700, 512, 3), ("norm", "mxfp8", 5, 0, 7168, 0), ("quantize", "nvfp4", 200, 0, 1056, 0)])
def test_first_call_inside_graph_capture(what, fmt, m, n, k, kernel):
    r = subprocess.run([sys.executable, "-c", CHILD, what, fmt, str(m), str(n), str(k), str(kernel)], cwd=ROOT,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stderr[-3000:]


def test_calls_from_concurrent_host_threads():
    """Five host threads with streams and inputs of their own, twenty rounds each."""
    errors = []

    def worker(i):
        try:
            s = torch.cuda.Stream()
            fmt = FORMATS[i % 3]
            name = list(FORMS)[i]
            with torch.cuda.stream(s):
                x, v = activations(100 + 60 * i, 1056, i), activations(333, 1056, 50 + i)
                kw = form(name, fmt, 1056)
                want = mx.matmul(mx.quantize(x, fmt), mx.quantize(v, fmt), **kw)
                one = torch.ones(1056, dtype=torch.bfloat16, device="cuda")
                n0 = mx.add_rms_norm(x, None, one, format=fmt)
                for _ in range(20):
                    got = mx.matmul(mx.quantize(x, fmt), mx.quantize(v, fmt), **kw)
                    n1 = mx.add_rms_norm(x, None, one, format=fmt)
                    s.synchronize()
                    assert torch.equal(got, want), name
                    assert torch.equal(n0.data.view(torch.uint8), n1.data.view(torch.uint8))
        except Exception as e:  # reported on the main thread
            errors.append(repr(e))

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(5)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def log_int(rng, lo, hi):
    return int(round(np.exp(rng.uniform(np.log(lo), np.log(hi)))))


@pytest.mark.parametrize("seed", range(40))
def test_random_product(seed):
    rng = np.random.default_rng(1000 + seed)
    fmt = FORMATS[seed % 3]
    M, N, K = log_int(rng, 1, 1500), log_int(rng, 1, 1500), 32 * log_int(rng, 1, 64)
    g = 0.01 if fmt == "nvfp4" and rng.random() < 0.5 else None
    a = random_matrix(M, K, fmt, seed, pad=16 * int(rng.integers(3)), g=g)
    w = random_matrix(N, K, fmt, seed + 500, pad=16 * int(rng.integers(3)), scale=0.05)
    va, vw = matrix_values(a, g), matrix_values(w)
    for name in ("auto", rng.choice(list(FORMS))):
        out = Rows(M, N, 8 * int(rng.integers(3)))
        mx.matmul(a.t, w.t, out.t, pdl=bool(rng.integers(2)), **form(name, fmt, K))
        torch.cuda.synchronize()
        assert out.intact(), name
        check_product(out.t, va, vw, K)


@pytest.mark.parametrize("seed", range(30))
def test_random_rows(seed):
    rng = np.random.default_rng(2000 + seed)
    fmt = FORMATS[seed % 3]
    rows, cols = log_int(rng, 1, 400), 32 * log_int(rng, 1, 300)
    pad = 8 * int(rng.integers(4))
    x = Rows(rows, cols, pad, activations(rows, cols, seed, scale=10.0 ** rng.uniform(-6, 6)))
    g = float(np.float32(10.0 ** rng.uniform(-8, 4))) if fmt == "nvfp4" else None
    q = Matrix(rows, cols, fmt, 16 * int(rng.integers(3)), None if g is None else torch.tensor([g], device="cuda"))
    mx.quantize(x.t, fmt, out=q.t)
    want = R.quantize(f64(x.t), fmt, g)
    data, flat, _ = q.host()
    np.testing.assert_array_equal(flat, want[1])
    np.testing.assert_array_equal(data, want[0])
    assert x.intact() and q.intact()
    check_norm(rows, cols, fmt, bool(rng.integers(2)), pad, bool(rng.integers(2)), 3000 + seed,
               scale=10.0 ** rng.uniform(-4, 4), g=None if g is None else 0.004)


@pytest.mark.parametrize("fmt", FORMATS)
def test_same_matrix_on_both_sides(fmt):
    """a and w may be one matrix; in-place chains reuse outputs as inputs."""
    q = mx.quantize(activations(200, 512, 8), fmt)
    v = torch.from_numpy(R.values(q.data.view(torch.uint8).cpu().numpy(),
                                  q.scales.view(torch.uint8).cpu().numpy().reshape(-1), fmt)).cuda()
    out = mx.matmul(q, q)
    check_product(out, v, v, 512)
    again = mx.quantize(mx.dequantize(q), fmt, out=q)  # a format's values quantise to themselves
    assert again is q or again.data.data_ptr() == q.data.data_ptr()
    check_product(mx.matmul(q, q), v, v, 512)
