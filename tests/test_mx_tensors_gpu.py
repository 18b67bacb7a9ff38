"""Matrices whose tensors change between two calls: an MxTensor's parts are the
caller's tensors, so a call takes them as they then are."""
import pytest
import torch

import attention_residual_fusion_gb300 as ar
from attention_residual_fusion_gb300 import _build, mx
from tests.test_mx_gpu import FORMATS, activations

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    ar.device_status(clear=True)
    yield
    assert ar.device_status() == 0


def raw(t):
    return t.view(torch.uint8)


def matrices(fmt, rows=200, cols=512):
    """Two matrices of one shape; nvfp4's with tensor scales of their own."""
    g = [torch.tensor([v], device="cuda") if fmt == "nvfp4" else None for v in (0.5, 0.03)]
    return [mx.quantize(activations(rows, cols, 80 + i), fmt, g[i]) for i in range(2)]


def by_data(t, other):
    t.data = other


def by_set(t, other):
    t.set_(other)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("replace", [by_data, by_set])
def test_parts_replaced_between_calls(fmt, replace):
    """Each part given other storage: every call reads the new one."""
    a, b = matrices(fmt)
    x = mx.quantize(activations(70, 512, 83), fmt)
    old = [mx.matmul(x, a), mx.matmul(a, x), mx.dequantize(a)]
    want = [mx.matmul(x, b), mx.matmul(b, x), mx.dequantize(b)]
    keep = [t.detach() for t in (a.data, a.scales)]  # the old storage stays alive
    replace(a.data, b.data.clone())
    replace(a.scales, b.scales.clone())
    if fmt == "nvfp4":
        keep.append(a.global_scale.detach())
        replace(a.global_scale, b.global_scale.clone())
    got = [mx.matmul(x, a), mx.matmul(a, x), mx.dequantize(a)]
    for o, w, g in zip(old, want, got):
        assert torch.equal(g, w) and not torch.equal(g, o)
    assert len(keep) >= 2


@pytest.mark.parametrize("fmt", FORMATS)
def test_results_go_to_the_new_storage(fmt):
    x = activations(130, 352, 84)
    want = mx.quantize(x, fmt)
    out = mx.MxTensor.empty(130, 352, fmt)
    for call in (lambda: mx.quantize(x, fmt, out=out),
                 lambda: mx.add_rms_norm(x, None, torch.ones(352, dtype=torch.bfloat16, device="cuda"), format=fmt,
                                         out=out)):
        raw(out.data).fill_(0x11)
        raw(out.scales).fill_(0x22)
        old = [raw(out.data).clone(), raw(out.scales).clone()]
        keep = [out.data.detach(), out.scales.detach()]
        out.data.data = torch.empty_like(out.data)
        out.scales.data = torch.empty_like(out.scales)
        assert call() is out
        assert torch.equal(raw(keep[0]), old[0]) and torch.equal(raw(keep[1]), old[1])
        assert not torch.equal(raw(out.data), old[0]) and not torch.equal(raw(out.scales), old[1])
    mx.quantize(x, fmt, out=out)
    assert torch.equal(raw(out.data), raw(want.data)) and torch.equal(raw(out.scales), raw(want.scales))


def test_another_row_stride_and_shape():
    """Rows further apart, and a smaller matrix, in the place of the first."""
    fmt, (a, b) = "mxfp4", matrices("mxfp4")
    x = mx.quantize(activations(70, 512, 83), fmt)
    wide = torch.zeros(200, 256 + 64, dtype=torch.uint8, device="cuda")
    wide[:, :256] = b.data
    a.data.data = wide[:, :256]
    a.scales.data = b.scales.clone()
    assert torch.equal(mx.matmul(x, a), mx.matmul(x, b))
    small = mx.quantize(activations(40, 512, 85), fmt)
    a.data.data, a.scales.data = small.data.clone(), small.scales.clone()
    assert a.shape == (40, 512) and torch.equal(mx.matmul(x, a), mx.matmul(x, small))


def test_storage_that_shrank():
    """Weights moved away (their storage emptied) are refused until they are back."""
    a, _ = matrices("mxfp8")
    x = activations(70, 512, 83)
    q = mx.quantize(x, "mxfp8")
    want = mx.matmul(q, a)
    for part in (a.data, a.scales):
        saved, size = raw(part).clone(), part.untyped_storage().nbytes()
        torch.cuda.synchronize()
        part.untyped_storage().resize_(0)
        for call in (lambda: mx.matmul(q, a), lambda: mx.matmul(a, q), lambda: mx.dequantize(a),
                     lambda: mx.quantize(activations(200, 512, 1), "mxfp8", out=a)):
            with pytest.raises(ValueError, match="storage"):
                call()
        part.untyped_storage().resize_(size)
        raw(part).copy_(saved)
        assert torch.equal(mx.matmul(q, a), want)
    # rows, of which the last few alone are gone, too
    y = torch.empty(70, 200, dtype=torch.bfloat16, device="cuda")
    for t, call in ((x, lambda: mx.quantize(x, "mxfp8")), (y, lambda: mx.matmul(q, a, y))):
        call()
        torch.cuda.synchronize()
        t.untyped_storage().resize_(t.untyped_storage().nbytes() - 2)
        with pytest.raises(ValueError, match="storage"):
            call()


def test_parts_that_no_longer_fit():
    """A part of another type, shape or layout is refused at the next call."""
    x = mx.quantize(activations(70, 512, 83), "nvfp4")
    changes = [
        lambda a: setattr(a.data, "data", a.data[:199]),  # the scales fit 129 to 256 rows still
        lambda a: setattr(a.data, "data", a.data[:100]),
        lambda a: setattr(a.data, "data", a.data.t()),
        lambda a: setattr(a.data, "data", a.data.view(-1)),
        lambda a: setattr(a.scales, "data", a.scales[:1]),
        lambda a: setattr(a.scales, "data", a.scales.transpose(2, 3)),
        lambda a: setattr(a.global_scale, "data", torch.ones(2, device="cuda")),
    ]
    for i, change in enumerate(changes):
        a, _ = matrices("nvfp4")
        change(a)
        if i == 0:
            assert mx.matmul(x, a).shape == (70, 199)
            continue
        for call in (lambda: mx.matmul(x, a), lambda: mx.matmul(a, x), lambda: mx.dequantize(a)):
            with pytest.raises(ValueError):
                call()


def test_wrong_types():
    """What is no matrix, no stream or no tensor is refused as documented."""
    x = activations(4, 64, 1)
    one = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    q = mx.quantize(x, "mxfp8")
    for bad in (x, "q", 3, q.data):
        with pytest.raises(ValueError, match="out"):
            mx.quantize(x, "mxfp8", out=bad)
        with pytest.raises(ValueError, match="out"):
            mx.add_rms_norm(x, None, one, out=bad)
    for bad in ("s", 0, x, torch.cuda.current_stream().cuda_stream):
        with pytest.raises(ValueError, match="stream"):
            mx.matmul(q, q, stream=bad)
        with pytest.raises(ValueError, match="stream"):
            mx.dequantize(q, stream=bad)
    for call in (lambda: mx.dequantize(x), lambda: mx.matmul(q, x), lambda: mx.quantize(q), lambda: mx.quantize(x, 3)):
        with pytest.raises(TypeError):
            call()
    assert torch.equal(mx.matmul(q, q, stream=torch.cuda.current_stream()), mx.matmul(q, q))
