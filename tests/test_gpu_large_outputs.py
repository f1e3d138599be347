"""Outputs large enough to be stored past the caches (256 MiB in rows of whole lines, values and weight
gradients 32 MiB, products of large tiles in any rows 512 MiB), and as large ones in ragged rows: the
same bits as in parts, and as moved."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import error_bounded_lossy_amd as ec  # noqa: E402
import mxref as R  # noqa: E402

MIB = 1 << 20


def values(seed, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(dtype)


def part(q, a, b):
    return ec.MXTensor(q.codes[a:b], q.scales[a:b], q.cols)


def large(t):
    row = t.shape[-1] * t.element_size()
    return t.numel() * t.element_size() >= (256 if row % 128 == 0 else 512) * MIB


@pytest.mark.parametrize("rows,cols,dtype", [(32768, 4096, torch.bfloat16), (70000, 4090, torch.float16), (16384, 4096, torch.float32),
                                             (1100000, 123, torch.float32), (4300000, 64, torch.bfloat16)])
def test_values(rows, cols, dtype):
    q = ec.mx_quantize(values(1, rows, cols))
    y = ec.mx_dequantize(q, dtype)
    assert large(y)
    step = rows // 7
    for a in range(0, rows, step):
        p = ec.mx_dequantize(part(q, a, min(a + step, rows)), dtype)
        assert torch.equal(y[a:a + step], p)


@pytest.mark.parametrize("rows,depth,cols,dtype", [(16384, 300, 8192, torch.bfloat16), (16500, 256, 16389, torch.float16), (8200, 256, 8192, torch.float32),
                                                   (16400, 128, 8190, torch.float32), (40000, 640, 3520, torch.bfloat16)])
def test_products(rows, depth, cols, dtype):
    a, b = ec.mx_quantize(values(1, rows, depth)), ec.mx_quantize(values(2, cols, depth))
    y = ec.mx_product(a, b, dtype)
    assert large(y)
    for first in (0, rows // 3, rows - 1100):
        p = ec.mx_product(part(a, first, first + 1100), b, dtype)
        assert not large(p) and torch.equal(y[first:first + 1100], p)


@pytest.mark.parametrize("cols,dtype", [(4096, torch.bfloat16), (8190, torch.float16), (4096, torch.float32)])
def test_experts_rows(cols, dtype):
    counts = [9000, 0, 1, 17000, 7000, 100]
    rows = sum(counts) + 70
    offsets = torch.tensor([0] + counts).cumsum(0).int().cuda()
    x, w = values(1, rows, 200), ec.mx_quantize(values(2, len(counts), cols, 200))
    q = ec.mx_quantize(x)
    y = ec.mx_experts_product(q, w, offsets, dtype)
    assert large(y)
    at = offsets.tolist()
    for e, (a, b) in enumerate(zip(at, at[1:])):
        for first in range(a, b, 3000):
            last = min(first + 3000, b)
            if last - first > 16:  # the kernel for few rows adds up in another order
                p = ec.mx_product(part(q, first, last), ec.MXTensor(w.codes[e], w.scales[e], 200), dtype)
                assert torch.equal(y[first:last], p)
    assert not y[at[-1]:].any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("depth,cols", [(1200, 1024), (1111, 1030)])
def test_weight_gradients(depth, cols, dtype):
    counts = [100, 0, 130, 7, 300] * 4
    offsets = torch.tensor([0] + counts).cumsum(0).int().cuda()
    rows = sum(counts)
    x, dy = values(1, rows, depth, dtype=dtype), values(2, rows, cols, dtype=dtype)
    w = values(3, len(counts), cols, depth, dtype=dtype)
    _, dw = ec.mx_experts_backward(dy, ec.mx_experts_forward(x, w, offsets)[1])
    assert dw.numel() * dw.element_size() > 32 * MIB
    at = offsets.tolist()
    for e, (a, b) in enumerate(zip(at, at[1:])):
        if a == b:
            assert not dw[e].any()
        else:
            R.check(dw[e], *R.mm_bound(R.near(dy[a:b].t()), R.near(x[a:b].t()), dtype), f"dw {e}")


@pytest.mark.parametrize("tokens,k,cols,dtype", [(16384, 4, 2048, torch.bfloat16), (17000, 4, 4100, torch.float16), (16384, 2, 4096, torch.float32)])
def test_exchange(tokens, k, cols, dtype):
    g = torch.Generator("cuda").manual_seed(tokens + k)
    ids = torch.randint(-1, 24, (tokens, k), generator=g, device="cuda", dtype=torch.int32)
    r = ec.expert_sort(ids, 24)
    x = values(1, tokens, cols, dtype=dtype)
    xs = ec.expert_dispatch(x, r)
    assert large(xs)
    kept = int(r.offsets[-1])
    assert torch.equal(xs[:kept], x[(r.order[:kept] // k).long()]) and not xs[kept:].any()


@pytest.mark.parametrize("tokens,cols,dtype", [(33000, 4096, torch.bfloat16), (66000, 4090, torch.float16), (16500, 4096, torch.float32)])
def test_tokens_brought_back(tokens, cols, dtype):
    # one choice of weight one: the rows themselves
    g = torch.Generator("cuda").manual_seed(tokens)
    ids = torch.randint(-1, 9, (tokens, 1), generator=g, device="cuda", dtype=torch.int32)
    r = ec.expert_sort(ids, 9)
    ys = values(1, tokens, cols, dtype=dtype)
    want = torch.where(ids >= 0, ys[r.place.reshape(-1).clamp(min=0).long()], torch.zeros((), dtype=dtype, device="cuda"))
    y = ec.expert_combine(ys, r, torch.ones(tokens, 1, device="cuda"))
    assert large(y) and torch.equal(y, want)
    assert torch.equal(ec.expert_dispatch_backward(ys, r), want)
