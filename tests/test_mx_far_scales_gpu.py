"""Products under tensor scales whose product fp32 does not hold."""
import numpy as np
import pytest
import torch

import attention_residual_fusion_gb300 as ar
from attention_residual_fusion_gb300 import _build, mx
from tests import mx_restatement as R
from tests.test_mx_gpu import BF16_HALF, FORMS, Matrix, Rows, form, matrix_values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    ar.device_status(clear=True)
    yield
    assert ar.device_status() == 0


def matrix(x, g):
    return Matrix(*x.shape, "nvfp4", 0, torch.tensor([g], device="cuda")).set(*R.quantize(x, "nvfp4", g))


def check(out, a, w, K):
    """fp32 sums as in the other products' tests, every factor rounded once, and half a
    step of the smallest bf16 numbers."""
    ref, mag = a @ w.t(), a.abs() @ w.abs().t()
    assert torch.isfinite(ref.to(torch.float32)).all()
    tol = BF16_HALF * ref.abs() + (1 + BF16_HALF) * (K / 32 + 4) * 2.0 ** -22 * mag + 2.0 ** -134 + 2.0 ** -147
    worst = ((out.double() - ref).abs() / tol).max().item()
    assert worst <= 1, f"worst error {worst} of the tolerance"


@pytest.mark.parametrize("M", [3, 60, 200])
@pytest.mark.parametrize("ga,gw", [(1e-24, 1e-20), (1e-20, 1e-25), (3e-30, 2e-16), (1e-38, 1e-9), (2.0 ** -149, 2.0 ** 60),
                                   (1e-23, 1e-22)])
def test_small_scales_under_large_sums(M, ga, gw):
    """Every form; sums of 1e9 and more, whose results are numbers although the scales' product is hardly one."""
    N, K = 200, 4128
    rng = np.random.default_rng(7)
    a, w = (matrix(np.abs(rng.standard_normal((r, K))) * 900 * float(np.float32(g)), g) for r, g in ((M, ga), (N, gw)))
    va, vw = matrix_values(a, ga), matrix_values(w, gw)
    for name in FORMS:
        out = Rows(M, N)
        mx.matmul(a.t, w.t, out.t, **form(name, "nvfp4", K))
        torch.cuda.synchronize()
        assert out.intact(), name
        check(out.t, va, vw, K)


@pytest.mark.parametrize("M", [3, 60, 200])
@pytest.mark.parametrize("ga,gw", [(1e30, 1e10), (3e25, 1e14), (1e2, 3e37), (5e37, 3e2)])
def test_large_scales_over_small_sums(M, ga, gw):
    """One small element a row: the scales' product is infinite, the results are not."""
    N, K = 200, 288
    rng = np.random.default_rng(8)

    def rows(r, g):
        x = np.zeros((r, K))
        x[:, 40] = np.round(rng.uniform(6, 24, r)) * 2.0 ** -9 * float(np.float32(g))
        return matrix(x, g)
    a, w = rows(M, ga), rows(N, gw)
    va, vw = matrix_values(a, ga), matrix_values(w, gw)
    assert bool((va != 0).any(1).all()) and bool((vw != 0).any(1).all())
    for name in FORMS:
        out = Rows(M, N)
        mx.matmul(a.t, w.t, out.t, **form(name, "nvfp4", K))
        torch.cuda.synchronize()
        check(out.t, va, vw, K)
        assert torch.isfinite(out.t).all() and bool((out.t != 0).all())


def test_results_out_of_range():
    """What is out of range itself is infinite or zero."""
    x = np.full((40, 64), 100.0)
    big, small = matrix(x * 1e30, 1e30), matrix(x * 1e-30, 1e-30)
    one = matrix(x, 1.0)
    for name in ("narrow1", "wide", "wider"):
        kw = form(name, "nvfp4", 64)
        assert torch.isinf(mx.matmul(big.t, big.t, **kw)).all()
        assert (mx.matmul(small.t, small.t, **kw) == 0).all()
        assert torch.isfinite(mx.matmul(big.t, one.t, **kw)).all()
        check(mx.matmul(big.t, small.t, **kw), matrix_values(big, 1e30), matrix_values(small, 1e-30), 64)


@pytest.mark.parametrize("M", [3, 60, 200])
def test_scales_that_are_no_numbers(M):
    """A tensor scale of NaN makes every result NaN, on either side; a negative one negates."""
    N, K = 130, 288
    rng = np.random.default_rng(9)
    a, w = (R.quantize(rng.standard_normal((r, K)), "nvfp4", 1.0) for r in (M, N))

    def at(codes, rows, g):
        return Matrix(rows, K, "nvfp4", 0, torch.tensor([g], device="cuda")).set(*codes).t
    for name in FORMS:
        kw = form(name, "nvfp4", K)
        for ga, gw in ((float("nan"), 0.5), (0.5, float("nan")), (float("nan"), float("nan"))):
            assert torch.isnan(mx.matmul(at(a, M, ga), at(w, N, gw), **kw)).all(), name
        want = mx.matmul(at(a, M, 0.5), at(w, N, 0.25), **kw)
        assert torch.equal(mx.matmul(at(a, M, -0.5), at(w, N, 0.25), **kw), -want), name
        far = mx.matmul(at(a, M, 1e30), at(w, N, 1e6), **kw)
        assert torch.equal(mx.matmul(at(a, M, 1e30), at(w, N, -1e6), **kw), -far), name
        tiny = mx.matmul(at(a, M, 1e-30), at(w, N, 1e-9), **kw)
        assert torch.equal(mx.matmul(at(a, M, -1e-30), at(w, N, 1e-9), **kw), -tiny) and bool((tiny != 0).any()), name
