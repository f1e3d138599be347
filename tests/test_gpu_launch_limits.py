"""Calls within the documented limits whose workgroups do not fit along x of a launch, which holds
less than 2^32 threads."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import error_bounded_lossy_amd as ec  # noqa: E402
import mxref as R  # noqa: E402

ROWS = 2 ** 30 + 77  # of 64 rows a workgroup: 2^24 workgroups of 256 threads and two


def marks(rows, per):
    """Some rows: the first ones, those around the borders of 2^22 workgroups, the last ones."""
    step = per << 22
    at = [0, 1] + [b + d for b in range(step, rows, step) for d in (-1, 0, 1)] + list(range(rows - 80, rows))
    return torch.tensor(sorted({a for a in at if 0 <= a < rows}), device="cuda")


def test_quantization_of_many_narrow_rows():
    at = marks(ROWS, 64)
    x = torch.zeros(ROWS, 1, dtype=torch.bfloat16, device="cuda")
    x[at, 0] = torch.randn(len(at), generator=torch.Generator("cuda").manual_seed(1), device="cuda").bfloat16()
    q = ec.mx_quantize(x)
    code, s = R.quantize(x[at])
    assert torch.equal(R.unpack(q.codes[at]), code.int()) and torch.equal(q.scales[at].int(), s.int())
    y = ec.mx_dequantize(q, torch.bfloat16)
    assert torch.equal(y[at], R.near(x[at]).to(torch.bfloat16))
    assert int(torch.count_nonzero(y)) == int(torch.count_nonzero(y[at]))
    del y
    q.codes[at] = 0
    q.scales[at] = 0
    for part in q.home.split(1 << 31):  # every other row is zeros
        assert not part.any()


def test_columns_of_a_product_of_one_row():
    cols = 2 ** 27 + 21  # 16 or 32 columns a workgroup, in other products of 512 threads
    g = torch.Generator("cuda").manual_seed(2)
    base = ec.mx_quantize(torch.randn(977, 100, generator=g, device="cuda").bfloat16())
    at = torch.arange(cols, device="cuda", dtype=torch.int32) % 977
    w = ec.MXTensor(base.codes[at], base.scales[at], 100)
    x = torch.randn(1, 100, generator=g, device="cuda").bfloat16()
    want = ec.mx_linear(x, base)[:, at]
    assert torch.equal(ec.mx_linear(x, w), want)
    assert torch.equal(ec.mx_product(ec.mx_quantize(x), w), want)


def test_exchange_of_many_narrow_tokens():
    tokens = 2 ** 28 + 37  # 16 tokens a workgroup of 256 threads
    g = torch.Generator("cuda").manual_seed(3)
    ids = torch.randint(-1, 3, (tokens, 1), generator=g, device="cuda", dtype=torch.int32)
    r = ec.expert_sort(ids, 3)
    counts = torch.bincount((ids.reshape(-1) + 1).long(), minlength=4)
    assert r.offsets.tolist() == [0, *counts[1:].cumsum(0).tolist()]
    kept = int(r.offsets[-1])
    order = torch.cat([torch.nonzero(ids.reshape(-1) == e).reshape(-1) for e in range(3)])
    assert torch.equal(r.order[:kept], order.int()) and bool((r.order[kept:] == -1).all())
    here = (ids >= 0).reshape(-1)
    assert torch.equal(r.place.reshape(-1)[order], torch.arange(kept, device="cuda", dtype=torch.int32))
    assert bool((r.place.reshape(-1)[~here] == -1).all())

    x = torch.randn(tokens, 1, generator=g, device="cuda").bfloat16()
    xs = ec.expert_dispatch(x, r)
    assert torch.equal(xs[:kept], x[order]) and not xs[kept:].any()
    back = torch.where(here[:, None], x, torch.zeros_like(x))
    assert torch.equal(ec.expert_dispatch_backward(xs, r), back)
    one = torch.ones(tokens, 1, device="cuda")
    assert torch.equal(ec.expert_combine(xs, r, one), back)
    dys, dw = ec.expert_combine_backward(x, xs, r, one)
    assert torch.equal(dys, xs)
    # a product of two bf16 values is exact in fp32
    assert torch.equal(dw, back.float() * x.float())
    q = ec.expert_dispatch_mx(x, r)
    at = marks(tokens, 16)
    at = at[at < kept]
    code, s = R.quantize(xs[at])
    assert torch.equal(R.unpack(q.codes[at]), code.int()) and torch.equal(q.scales[at].int(), s.int())
    assert not q.codes[kept:].any() and not q.scales[kept:].any()


def test_training_over_the_longest_row_of_tokens():
    # ones among zeros: every sum is a whole number that fp32 holds
    rows, depth, cols = 2 ** 24, 8, 8
    g = torch.Generator("cuda").manual_seed(4)
    x = (torch.rand(rows, depth, generator=g, device="cuda") < 0.3).bfloat16()
    dy = (torch.rand(rows, cols, generator=g, device="cuda") < 0.3).bfloat16()
    w = torch.ones(3, cols, depth, dtype=torch.bfloat16, device="cuda")
    at = [0, 5_000_001, 5_000_002, rows]
    offsets = torch.tensor(at, dtype=torch.int32, device="cuda")
    y, saved = ec.mx_experts_forward(x, w, offsets)
    dx, dw = ec.mx_experts_backward(dy, saved)
    assert torch.equal(y.float(), x.float().sum(1, keepdim=True).expand(-1, cols))
    assert torch.equal(dx.float(), dy.float().sum(1, keepdim=True).expand(-1, depth))
    for e, (a, b) in enumerate(zip(at, at[1:])):
        want = (dy[a:b].t().contiguous().double() @ x[a:b].double()).float().bfloat16()
        assert torch.equal(dw[e], want)
