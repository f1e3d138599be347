"""The root-mean-square norm and its gradients against 64 bits.

Tolerances: a lane adds up to 64 terms a round one after the other and the lanes' sums are joined in at
most 8 steps, so a sum of n terms is off by at most (64 rounds + 8) 2^-24 of its terms' magnitudes (rounds:
every 16384 elements), 1 / sqrt of a mean by half of that and 4 roundings more; a product has one
rounding more for each factor, and a result half a step of its type."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import error_bounded_lossy_amd as ec  # noqa: E402
import layerref as R  # noqa: E402

TYPES = [torch.float32, torch.float16, torch.bfloat16]
ids = lambda v: str(v).replace("torch.", "") if isinstance(v, torch.dtype) else None  # noqa: E731
U = 2.0 ** -24
SIZES = [(1, 1), (1, 8192), (2, 7), (3, 128), (40, 129), (5, 500), (33, 1111), (300, 2048), (1000, 64), (9, 5120),
         (4, 16384), (3, 16385), (2, 50000)]


def step(dtype):
    return torch.finfo(dtype).eps / 2


def values(seed, *shape, dtype=torch.float32, size=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(*shape, generator=g, device="cuda") * size
    return (x * torch.exp(torch.randn(*shape[:-1], 1, generator=g, device="cuda"))).to(dtype)


def weights(seed, cols, dtype):
    return (1 + 0.3 * torch.randn(cols, generator=torch.Generator("cuda").manual_seed(seed), device="cuda")).to(dtype)


def of_sum(cols):
    return (64 * math.ceil(cols / 16384) + 8) * U


def least(dtype):
    """Results below the type's smallest normal number are off by half of its smallest step."""
    return torch.finfo(dtype).tiny * torch.finfo(dtype).eps


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_norm(rows, cols, dtype):
    x, r = values(1, rows, cols, dtype=dtype), values(2, rows, cols, dtype=dtype)
    x[0, :] = 0
    r[0, :] = 0
    for wtype in TYPES:
        w = weights(3, cols, wtype)
        y, h = ec.rms_norm(x, w, 1e-5, residual=r)
        assert torch.equal(h, (x.float() + r.float()).to(dtype))
        for got, of in ((y, h), (ec.rms_norm(x, w, 1e-5), x)):
            want = R.norm(of, w, 1e-5)
            assert got.dtype == dtype
            assert ((got.double() - want).abs() <= want.abs() * (of_sum(cols) / 2 + 6 * U + step(dtype)) + least(dtype)).all()
        y2, saved = ec.rms_norm_forward(x, w, 1e-5, residual=r)
        assert torch.equal(y2, y) and torch.equal(saved.h, h)
        assert ((saved.rstd.double() * (h.double().square().mean(1) + 1e-5).sqrt() - 1).abs() <= of_sum(cols) / 2 + 4 * U).all()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_norm_in_8_bits(rows, cols, dtype):
    x, r = values(1, rows, cols, dtype=dtype), values(2, rows, cols, dtype=dtype)
    x[0, :] = 0
    r[0, :] = 0
    w = weights(3, cols, dtype)
    q, h = ec.rms_norm_i8(x, w, 1e-5, residual=r)
    assert torch.equal(h, (x.float() + r.float()).to(dtype))
    alone = ec.rms_norm_i8(h, w, 1e-5)
    assert torch.equal(q.codes, alone.codes) and torch.equal(q.scales, alone.scales)
    assert q.shape == x.shape and not q.codes[:, cols:].any()
    want = R.norm(h, w, 1e-5)
    off = of_sum(cols) / 2 + 6 * U  # of y before its rounding
    top = want.abs().amax(1)
    assert ((q.scales.double() - top / 127).abs() <= top / 127 * (off + U) + least(torch.float32)).all()
    # half a step of the scale, and what y and the quotient are off by before
    got = ec.i8_dequantize(q).double()
    assert ((got - want).abs() <= q.scales.double()[:, None] * (0.5 + 127 * (2 * off + 3 * U))).all()
    assert (q.codes.abs().amax(1)[top > 0] == 127).all()


def gradients(dy, h, w, dh, eps):
    h, w = h.double().requires_grad_(), w.double().requires_grad_()
    y = R.norm(h, w, eps)
    dx, dw = torch.autograd.grad(y, (h, w), dy.double())
    return dx + (0 if dh is None else dh.double()), dw


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,cols", SIZES + [(5000, 100), (2100, 1030)])
def test_gradients(rows, cols, dtype):
    x, r = values(1, rows, cols, dtype=dtype), values(2, rows, cols, dtype=dtype)
    if rows > 1:
        x[0, :] = 0
        r[0, :] = 0
    dy, dh = values(4, rows, cols, dtype=dtype, size=0.1), values(5, rows, cols, dtype=dtype, size=0.1)
    for wtype in {dtype, torch.float32}:
        w = weights(3, cols, wtype)
        y, saved = ec.rms_norm_forward(x, w, 1e-5, residual=r)
        for after in (None, dh):
            dx, dw = ec.rms_norm_backward(dy, saved, after)
            want, want_w = gradients(dy, saved.h, w, after, 1e-5)
            assert dx.dtype == dtype and dw.dtype == wtype and dw.shape == (cols,)
            # dx is a difference: its parts' magnitudes count
            f, g = saved.h.double(), dy.double() * w.double()
            rstd = (f.square().mean(1, keepdim=True) + 1e-5).rsqrt()
            parts = rstd * (g.abs() + (f * rstd).abs() * (g * f * rstd).abs().mean(1, keepdim=True))
            parts = parts + (0 if after is None else after.double().abs())
            off = 2.5 * of_sum(cols) + 12 * U
            assert ((dx.double() - want).abs() <= parts * off + want.abs() * step(dtype) + least(dtype)).all()
            # a slot's rows one after the other (at most rows / 2 of them), then the parts in slices
            terms = (dy.double() * f * rstd).abs().sum(0)
            assert ((dw.double() - want_w).abs() <= terms * (of_sum(cols) / 2 + (8 + rows) * U) + want_w.abs() * step(wtype) + least(wtype)).all()


def test_gradients_against_differences():
    rows, cols, eps, d = 3, 40, 1e-3, 1e-5
    x, w, dy = (values(i, *s, dtype=torch.float32) for i, s in ((1, (rows, cols)), (2, (1, cols)), (3, (rows, cols))))
    w = w[0]
    _, saved = ec.rms_norm_forward(x, w, eps)
    dx, dw = ec.rms_norm_backward(dy, saved)
    loss = lambda x, w: (R.norm(x, w, eps) * dy.double()).sum()  # noqa: E731
    for (i, j) in ((0, 0), (1, 17), (2, 39)):
        e = torch.zeros(rows, cols, dtype=torch.float64, device="cuda")
        e[i, j] = d
        slope = (loss(x.double() + e, w.double()) - loss(x.double() - e, w.double())) / (2 * d)
        assert abs(slope - dx[i, j].double()) <= 1e-5 * dx.abs().max()
        slope = (loss(x.double(), w.double() + e.sum(0)) - loss(x.double(), w.double() - e.sum(0))) / (2 * d)
        assert abs(slope - dw[j].double()) <= 1e-5 * dw.abs().max()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_rows_that_are_not_finite_stay_among_themselves(dtype):
    x = values(1, 6, 300, dtype=dtype)
    clean = x.clone()
    x[1, 5], x[2, 299], x[4, 0] = math.nan, math.inf, -math.inf
    w = weights(2, 300, dtype)
    good = [0, 3, 5]
    y = ec.rms_norm(x, w)
    assert torch.equal(y[good], ec.rms_norm(clean, w)[good])
    assert torch.isnan(y[1]).all() and torch.isnan(y[2, 299]) and torch.isnan(y[4, 0])
    q = ec.rms_norm_i8(x, w)
    assert torch.isnan(q.scales[[1, 2, 4]]).all() and not q.codes[[1, 2, 4]].any()
    assert torch.equal(q.codes[good], ec.rms_norm_i8(clean, w).codes[good])
    dx, dw = ec.rms_norm_backward(clean, ec.rms_norm_forward(x, w)[1])
    assert torch.isnan(dx[1]).all() and torch.isnan(dw).any()
    assert torch.equal(dx[good], ec.rms_norm_backward(clean, ec.rms_norm_forward(clean, w)[1])[0][good])


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_strides_shapes_and_no_rows(dtype):
    base, other = values(3, 40, 300, dtype=dtype), values(4, 40, 300, dtype=dtype)
    for cut in (lambda b: b[:, 7:207], lambda b: b[::3, :200], lambda b: b.t()[:100], lambda b: b[:1, 1:2],
                lambda b: b.view(4, 10, 300)[:, :, 5:105], lambda b: b[3], lambda b: b[:0]):
        x, r = cut(base), cut(other)
        w = weights(1, x.shape[-1], dtype)
        for f in (ec.rms_norm, ec.rms_norm_i8):
            got, h = f(x, w, residual=r)
            want, h2 = f(x.contiguous().clone(), w, residual=r.contiguous().clone())
            assert got.shape == x.shape and h.shape == x.shape and torch.equal(h, h2)
            for a, b in ((got, want),) if f is ec.rms_norm else ((got.codes, want.codes), (got.scales, want.scales)):
                assert torch.equal(a, b)
        y, saved = ec.rms_norm_forward(x, w)
        dx, dw = ec.rms_norm_backward(r, saved, dh=x)
        dx2, dw2 = ec.rms_norm_backward(r.contiguous().clone(), ec.rms_norm_forward(x.contiguous().clone(), w)[1], dh=x.contiguous().clone())
        assert dx.shape == x.shape and torch.equal(dx, dx2) and torch.equal(dw, dw2)
        if x.numel() == 0:
            assert not dw.any()


def test_sums_of_large_and_small_rows():
    # squares within fp32's range: 1e18 and 1e-15 (below eps)
    w = torch.ones(256, device="cuda")
    x = torch.randn(4, 256, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    for size in (1e18, 1e-15):
        y = ec.rms_norm(x * size, w, 1e-6)
        want = R.norm(x * size, w, 1e-6)
        assert ((y.double() - want).abs() <= want.abs() * (of_sum(256) / 2 + 7 * U)).all()
