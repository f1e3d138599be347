"""The norm, the routing and the 8-bit form where offsets pass 32 bits and launches more workgroups than fit
along x."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import error_bounded_lossy_amd as ec  # noqa: E402
import layerref as R  # noqa: E402


@pytest.fixture(autouse=True)
def freed():
    yield
    torch.cuda.empty_cache()


def ends(n, count=40):
    """Rows from the start, the end and between."""
    return torch.cat([torch.arange(count), torch.arange(n // 2, n // 2 + count), torch.arange(n - count, n)]).cuda()


def test_arrays_of_more_than_2_to_the_32_elements():
    rows, cols = 1050000, 4100
    g = torch.Generator("cuda").manual_seed(1)
    part = torch.randn(1000, cols, generator=g, device="cuda").bfloat16()
    x = part.repeat(rows // 1000, 1)
    at, w = ends(rows), torch.randn(cols, generator=g, device="cuda").bfloat16()
    q = ec.i8_quantize(x)
    want = ec.i8_quantize(part[at % 1000])
    assert torch.equal(q.codes[at], want.codes) and torch.equal(q.scales[at], want.scales)
    y = ec.i8_dequantize(q, torch.bfloat16)
    assert torch.equal(y[at], ec.i8_dequantize(want, torch.bfloat16))
    del y
    n, saved = ec.rms_norm_forward(x, w)
    assert torch.equal(n[at], ec.rms_norm(part[at % 1000], w))
    dx, _ = ec.rms_norm_backward(x, saved)
    assert torch.equal(dx[at], ec.rms_norm_backward(part[at % 1000], ec.rms_norm_forward(part[at % 1000], w)[1])[0])
    del n, dx, saved
    q2 = ec.rms_norm_i8(x, w)
    assert torch.equal(q2.codes[at], ec.rms_norm_i8(part[at % 1000], w).codes)
    del q2, x
    b = ec.i8_quantize(torch.randn(4097, cols, generator=g, device="cuda"))
    y = ec.i8_product(q, b, torch.bfloat16)  # 4.3e9 results
    assert torch.equal(y[at], R.i8_product(q.codes[at], q.scales[at], b.codes, b.scales, torch.bfloat16))
    del y
    ids = torch.randint(-1, 8, (rows, 1), generator=g, device="cuda", dtype=torch.int32)
    r = ec.expert_sort(ids, 8)
    xs = ec.expert_dispatch_i8(q, r)
    kept = int(r.offsets[-1])
    at = ends(kept)
    token = r.order[at].long()
    assert torch.equal(xs.codes[at], q.codes[token]) and torch.equal(xs.scales[at], q.scales[token])
    assert not xs.codes[kept:].any()


def test_more_workgroups_than_fit_along_x():
    tokens = (1 << 28) + 77
    l = torch.randn(tokens, 1, device="cuda", dtype=torch.bfloat16)
    ids, weights = ec.expert_route(l, 1, "sigmoid", renormalize=False)
    at = ends(tokens)
    assert not ids.any() and torch.allclose(weights[at], torch.sigmoid(l[at].float()))
    d = ec.expert_route_backward(weights, l, ids, "sigmoid", renormalize=False)
    s = torch.sigmoid(l[at].double())
    assert torch.allclose(d[at].double(), weights[at].double() * s * (1 - s), rtol=2.0 ** -8)
    del l, ids, weights, d
    rows = (1 << 26) + 21
    x = torch.randn(rows, 3, device="cuda", dtype=torch.bfloat16)
    w = torch.randn(3, device="cuda")
    y, saved = ec.rms_norm_forward(x, w)
    at = ends(rows)
    assert torch.equal(y[at], ec.rms_norm(x[at], w))
    dx, dw = ec.rms_norm_backward(y, saved)
    assert torch.equal(dx[at], ec.rms_norm_backward(y[at], ec.rms_norm_forward(x[at], w)[1])[0])
    terms = y.double() * x.double() * saved.rstd.double()[:, None]
    assert ((dw.double() - terms.sum(0)).abs() <= terms.abs().sum(0) * 2.0 ** -24 * 9000).all()  # 8192 rows a slot, then its parts
    del y, saved, dx, terms
    q = ec.i8_quantize(x)
    assert torch.equal(q.codes[at], ec.i8_quantize(x[at]).codes) and torch.equal(ec.i8_dequantize(q)[at], ec.i8_dequantize(ec.i8_quantize(x[at])))
