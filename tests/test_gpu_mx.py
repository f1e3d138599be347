"""The 4-bit format and its products on the GPU against their definitions in 64 bits."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import error_bounded_lossy_amd as ec  # noqa: E402
import mxref as R  # noqa: E402

TYPES = [torch.bfloat16, torch.float16, torch.float32]
ids = lambda v: str(v).replace("torch.", "") if isinstance(v, torch.dtype) else None  # noqa: E731


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def activations(seed, *shape, dtype=torch.bfloat16, spread=3.0):
    g = gen(seed)
    x = torch.randn(*shape, generator=g, device="cuda")
    x = x * torch.exp2(spread * torch.randn(*shape[:-1], 1, generator=g, device="cuda"))
    if x.numel() > 64:
        x.view(-1)[5::97] = 0
    return x.to(dtype)


def same_form(q, x, what=""):
    code, s = R.quantize(x)
    assert torch.equal(R.unpack(q.codes), code.int()), f"{what}: codes"
    assert torch.equal(q.scales.int(), s.int()), f"{what}: scales"


# ---------------------------------------------------------------- the form


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 32), (3, 31), (2, 33), (5, 127), (4, 128), (7, 129),
                                       (1, 8192), (33, 1111), (300, 520), (129, 2500), (2100, 4096)])
def test_quantize_rows_and_values(rows, cols, dtype):
    x = activations(rows * 7 + cols, rows, cols, dtype=dtype)
    q = ec.mx_quantize(x)
    assert q.shape == (rows, cols) and q.codes.shape == (rows, R.pad(cols) // 2)
    same_form(q, x)
    v = R.near(x)
    for out in TYPES:
        assert torch.equal(ec.mx_dequantize(q, out), v.to(out)), out


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_every_pattern_and_every_border(dtype):
    if dtype == torch.float32:
        e = torch.arange(0, 255, device="cuda", dtype=torch.int64)
        m = torch.arange(0, 64, device="cuda", dtype=torch.int64) << 17
        near = torch.tensor([-1, 0, 1], device="cuda", dtype=torch.int64)
        bits = (e[:, None, None] << 23) + m[None, :, None] + near
        x = bits.clamp(min=0, max=0x7f7fffff).to(torch.int32).reshape(-1).view(torch.float32)
    else:
        x = torch.arange(0x10000, device="cuda", dtype=torch.int32).to(torch.int16).view(dtype)
        x = x[torch.isfinite(x.float())]
    x = torch.cat([x, -x])
    x = x[: x.numel() // 16 * 16].reshape(-1, 16)
    # every value beside the largest of its block, over the binades around it
    f = x.float().abs()
    for shift in (0, 1, 2, 3):
        lead = torch.full_like(f, 0)
        lead[:, 0] = f.amax(-1) * 2.0 ** shift
        top = torch.finfo(dtype).max
        b = torch.cat([x, lead.clamp(max=top).to(dtype)], -1)
        same_form(ec.mx_quantize(b), b, f"{dtype} shift {shift}")


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_blocks_that_are_not_finite(dtype):
    x = activations(3, 6, 256, dtype=dtype)
    x[1, 40] = float("inf")
    x[2, 70] = float("nan")
    x[3, 255] = -float("inf")
    x[4] = 0
    x[5] = -0.0
    rows, cols = ec.mx_quantize_both(x)
    want = R.near(x)
    for q, w in ((ec.mx_quantize(x), want), (rows, want), (cols, R.near(x.t()))):
        v = ec.mx_dequantize(q, dtype)
        assert torch.equal(torch.isnan(v), torch.isnan(w))
        assert torch.equal(v.nan_to_num(0.0), w.to(dtype).nan_to_num(0.0))
    # a product over such a block is NaN, the other rows are not
    w = ec.mx_quantize(activations(4, 40, 256, dtype=dtype))
    for rep in (1, 8):  # few rows, and tiles
        y = ec.mx_linear(x.repeat(rep, 1), w)
        assert torch.equal(torch.isnan(y), torch.isnan(want).any(-1).repeat(rep)[:, None].expand_as(y))


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("shape", [(1, 1), (32, 32), (31, 33), (127, 65), (128, 128), (129, 130), (300, 77),
                                   (1000, 260), (3, 70, 90), (2, 256, 512), (5, 1, 129)])
def test_quantize_both(shape, dtype):
    x = activations(sum(shape), *shape, dtype=dtype)
    rows, cols = ec.mx_quantize_both(x)
    same_form(rows, x, "rows")
    same_form(cols, x.transpose(-1, -2), "columns")
    assert cols.shape == (*shape[:-2], shape[-1], shape[-2])


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_strides_and_alignment(dtype):
    big = activations(11, 70, 1031, dtype=dtype)
    for x in (big[:, 3:900], big[5:60, 1:130], big[::2, :77], big.t()[:100, :50], big[:1, 7:8]):
        same_form(ec.mx_quantize(x), x)
        a, b = ec.mx_quantize_both(x)
        same_form(a, x)
        same_form(b, x.t())
        w = ec.mx_quantize(activations(12, 19, x.shape[1], dtype=dtype))
        y, bound = R.mm_bound(R.near(x), ec.mx_dequantize(w, torch.float32).double(), dtype)
        R.check(ec.mx_linear(x, w), y, bound)
    batch = big[:60].reshape(2, 30, 1031)[:, :, 9:200]
    same_form(ec.mx_quantize_both(batch)[1], batch.transpose(1, 2))


def test_strides_of_sizes_of_one():
    # a single row or column: its stride may be anything, here 1
    row = activations(1, 200, 1).t()
    assert row.shape == (1, 200) and row.stride(0) == 1
    w = ec.mx_quantize(activations(2, 30, 200))
    want, bound = R.mm_bound(R.near(row), ec.mx_dequantize(w, torch.float32).double(), torch.bfloat16)
    R.check(ec.mx_linear(row, w), want, bound)
    offsets = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    y, saved = ec.mx_experts_forward(row, activations(3, 1, 30, 200), offsets)
    assert y.shape == (1, 30) and ec.mx_experts_backward(y, saved)[0].shape == (1, 200)
    for x in (row, row.t(), row.unsqueeze(0), row.t().unsqueeze(0), activations(4, 5, 7, 1).transpose(0, 2)):
        same_form(ec.mx_quantize(x), x)
        a, b = ec.mx_quantize_both(x)
        same_form(a, x)
        same_form(b, x.transpose(-1, -2))


def test_empty_rows_and_leading_dimensions():
    x = activations(1, 2, 3, 40)
    same_form(ec.mx_quantize(x), x)
    assert ec.mx_dequantize(ec.mx_quantize(x)).shape == (2, 3, 40)
    e = x.reshape(6, 40)[:0]
    q = ec.mx_quantize(e)
    assert q.shape == (0, 40) and ec.mx_dequantize(q).shape == (0, 40)
    w = ec.mx_quantize(activations(2, 9, 40))
    assert ec.mx_linear(e, w).shape == (0, 9) and ec.mx_linear(x, w).shape == (2, 3, 9)
    y, saved = ec.mx_linear_forward(e, activations(3, 9, 40))
    dx, dw = ec.mx_linear_backward(y, saved)
    assert dx.shape == (0, 40) and dw.shape == (9, 40) and not dw.any()


def test_offsets_past_32_bits():
    rows, cols = 16500, 132000  # 2.2e9 elements: byte and element offsets leave 32 bits
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    tail = activations(5, 130, cols)
    x[-130:] = tail
    q = ec.mx_quantize(x)
    same_form(ec.MXTensor(q.codes[-130:].contiguous(), q.scales[-130:].contiguous(), cols), tail)
    assert not q.codes[:-130].any()
    a, b = ec.mx_quantize_both(x)
    assert torch.equal(a.codes, q.codes) and torch.equal(a.scales, q.scales)
    del a
    last = ec.MXTensor(b.codes[-9:].contiguous(), b.scales[-9:].contiguous(), rows)
    same_form(last, x[:, -9:].t())
    del b
    y = ec.mx_dequantize(q, torch.bfloat16)
    assert torch.equal(y[-130:], R.near(tail).to(torch.bfloat16)) and not y[:-130].any()


# ---------------------------------------------------------------- products


PRODUCTS = [(1, 1, 1), (1, 128, 128), (1, 8192, 300), (2, 33, 17), (7, 640, 100), (8, 2500, 65), (9, 128, 16),
            (15, 1111, 33), (16, 512, 1111), (17, 513, 64), (33, 4096, 65), (64, 128, 64), (65, 200, 129),
            (77, 2500, 1111), (300, 384, 500), (130, 8192, 60)]


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,depth,cols", PRODUCTS)
def test_linear(rows, depth, cols, dtype):
    x = activations(rows + depth, rows, depth, dtype=dtype, spread=1.0)
    w = activations(cols, cols, depth, dtype=dtype, spread=1.0)
    q = ec.mx_quantize(w)
    y, bound = R.mm_bound(R.near(x), R.near(w), dtype)
    R.check(ec.mx_linear(x, q), y, bound, "linear")
    R.check(ec.mx_product(ec.mx_quantize(x), q, dtype), y, bound, "product")


# each tile size: enough tiles of 128 and of 256 rows and columns, ragged at both ends
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,depth,cols", [(1500, 128, 1700), (1409, 896, 1537), (3500, 384, 3600),
                                             (3457, 1100, 3401), (4000, 640, 3330)])
def test_linear_tiles(rows, depth, cols, dtype):
    x = activations(rows, rows, depth, dtype=dtype, spread=1.0)
    w = activations(cols, cols, depth, dtype=dtype, spread=1.0)
    y, bound = R.mm_bound(R.near(x), R.near(w), dtype)
    R.check(ec.mx_linear(x, ec.mx_quantize(w)), y, bound)


# rows past whole tiles that would start another round of them: few, and some
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,depth,cols", [(4100, 200, 4096), (2125, 300, 8190), (4111, 128, 4001)])
def test_linear_rows_past_whole_tiles(rows, depth, cols, dtype):
    x = activations(rows, rows, depth, dtype=dtype, spread=1.0)
    w = activations(cols, cols, depth, dtype=dtype, spread=1.0)
    y, bound = R.mm_bound(R.near(x), R.near(w), dtype)
    R.check(ec.mx_linear(x, ec.mx_quantize(w)), y, bound)


@pytest.mark.parametrize("rows,depth,cols", [(4111, 2100, 4096), (4226, 2000, 4090), (8200, 1500, 2040)])
def test_linear_rows_past_whole_tiles_of_long_contractions(rows, depth, cols):
    x = activations(rows, rows, depth, spread=1.0)
    w = activations(cols, cols, depth, spread=1.0)
    y, bound = R.mm_bound(R.near(x), R.near(w), torch.bfloat16)
    R.check(ec.mx_linear(x, ec.mx_quantize(w)), y, bound)


def test_scales_at_their_ends():
    # blocks near 2^-127 against blocks near 2^120, and results that are subnormal
    x = torch.randn(20, 256, generator=gen(1), device="cuda")
    w = torch.randn(40, 256, generator=gen(2), device="cuda")
    for a, b in ((2.0 ** -120, 2.0 ** 110), (2.0 ** -70, 2.0 ** -60)):
        y, bound = R.mm_bound(R.near(x * a), R.near(w * b), torch.float32)
        for rows in (x, x.repeat(4, 1)):
            R.check(ec.mx_linear(rows * a, ec.mx_quantize(w * b)), y.repeat(len(rows) // 20, 1),
                    bound.repeat(len(rows) // 20, 1))


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,depth,cols", [(1, 5, 3), (40, 64, 100), (33, 130, 127), (257, 300, 64),
                                             (700, 1111, 520), (1800, 1600, 1500)])
def test_training_step(rows, depth, cols, dtype):
    x = activations(1, rows, depth, dtype=dtype, spread=1.0)
    w = activations(2, cols, depth, dtype=dtype, spread=1.0)
    dy = activations(3, rows, cols, dtype=dtype, spread=1.0)
    y, saved = ec.mx_linear_forward(x, w)
    dx, dw = ec.mx_linear_backward(dy, saved)
    t = lambda v: R.near(v.t())  # noqa: E731
    R.check(y, *R.mm_bound(R.near(x), R.near(w), dtype), "y")
    R.check(dx, *R.mm_bound(R.near(dy), t(w), dtype), "dx")
    R.check(dw, *R.mm_bound(t(dy), t(x), dtype), "dw")


def on_grid(seed, rows, cols):
    """Values that the form holds exactly in both directions: 4 in every block."""
    x = torch.randint(-3, 4, (rows, cols), generator=gen(seed), device="cuda").float()
    x[torch.arange(rows)[:, None] % 32 == torch.arange(cols) % 32] = 4.0
    return x


def test_gradients_against_differences():
    # values and values one step off are exact in the form, so the loss is linear there
    x, w, dy = on_grid(1, 64, 96), on_grid(2, 32, 96), on_grid(3, 64, 32)
    y, saved = ec.mx_linear_forward(x, w)
    dx, dw = ec.mx_linear_backward(dy, saved)
    loss = lambda a, b: (ec.mx_linear_forward(a, b)[0].double() * dy.double()).sum().item()  # noqa: E731
    for i, j in ((0, 1), (5, 40), (33, 2), (63, 95), (20, 70)):
        if abs(x[i, j]) > 2:
            x[i, j] = 1.0
            _, saved = ec.mx_linear_forward(x, w)
            dx, dw = ec.mx_linear_backward(dy, saved)
        up, down = x.clone(), x.clone()
        up[i, j] += 1
        down[i, j] -= 1
        assert (loss(up, w) - loss(down, w)) / 2 == dx[i, j].item()
        k = i % 32
        if abs(w[k, j]) <= 2:
            up, down = w.clone(), w.clone()
            up[k, j] += 1
            down[k, j] -= 1
            assert (loss(x, up) - loss(x, down)) / 2 == dw[k, j].item()


# ---------------------------------------------------------------- groups


GROUPS = [[0], [5], [0, 0, 3], [1, 0, 40, 0, 16, 17], [300, 0, 2, 128, 129], [64] * 8, [3] * 70,
          [1000, 1, 500, 0], [130] * 16]


def grouped(counts, dropped, seed, depth, dtype):
    offsets = torch.tensor([0] + counts).cumsum(0).int().cuda()
    return activations(seed, sum(counts) + dropped, depth, dtype=dtype, spread=1.0), offsets


def parts(offsets):
    at = offsets.tolist()
    return list(zip(at, at[1:]))


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("depth,cols", [(130, 70), (640, 256)])
@pytest.mark.parametrize("dropped", [0, 9])
@pytest.mark.parametrize("counts", GROUPS, ids=lambda c: f"{len(c)}x{sum(c)}")
def test_experts(counts, dropped, depth, cols, dtype):
    x, offsets = grouped(counts, dropped, 1, depth, dtype)
    w = activations(2, len(counts), cols, depth, dtype=dtype, spread=1.0)
    dy = activations(3, len(x), cols, dtype=dtype, spread=1.0)
    used = sum(counts)
    x[used:] = float("nan")   # rows of no expert take no part
    dy[used:] = float("inf")
    y1 = ec.mx_experts_linear(x, ec.mx_quantize(w), offsets)
    y2, saved = ec.mx_experts_forward(x, w, offsets)
    dx, dw = ec.mx_experts_backward(dy, saved)
    for e, (a, b) in enumerate(parts(offsets)):
        if a == b:
            assert not dw[e].any()
            continue
        want = R.mm_bound(R.near(x[a:b]), R.near(w[e]), dtype)
        R.check(y1[a:b], *want, f"linear {e}")
        R.check(y2[a:b], *want, f"forward {e}")
        R.check(dx[a:b], *R.mm_bound(R.near(dy[a:b]), R.near(w[e].t()), dtype), f"dx {e}")
        R.check(dw[e], *R.mm_bound(R.near(dy[a:b].t()), R.near(x[a:b].t()), dtype), f"dw {e}")
    for v in (y1, y2, dx):
        assert v.shape[0] == used + dropped and not v[used:].any()


@pytest.mark.parametrize("dtype", [torch.bfloat16], ids=ids)
def test_experts_large_tiles(dtype):
    counts = [700, 0, 1300, 256, 255, 900]
    x, offsets = grouped(counts, 300, 1, 384, dtype)
    w = activations(2, 6, 4100, 384, dtype=dtype, spread=1.0)
    dy = activations(3, len(x), 4100, dtype=dtype, spread=1.0)
    y, saved = ec.mx_experts_forward(x, w, offsets)
    dx, dw = ec.mx_experts_backward(dy, saved)
    for e, (a, b) in enumerate(parts(offsets)):
        if a < b:
            R.check(y[a:b], *R.mm_bound(R.near(x[a:b]), R.near(w[e]), dtype), f"y {e}")
            R.check(dx[a:b], *R.mm_bound(R.near(dy[a:b]), R.near(w[e].t()), dtype), f"dx {e}")
            R.check(dw[e], *R.mm_bound(R.near(dy[a:b].t()), R.near(x[a:b].t()), dtype), f"dw {e}")
    assert not y[sum(counts):].any() and not dx[sum(counts):].any() and not dw[1].any()


@pytest.mark.parametrize("counts", [[0, 90, 0, 1, 17, 0, 0, 4] + [0] * 12, [500] + [0] * 63, [0] * 1023 + [40]],
                         ids=lambda c: f"{len(c)}x{sum(c)}")
@pytest.mark.parametrize("depth", [200, 9000])
def test_experts_few_rows_on_average(counts, depth):
    # few rows an expert on average, many for some: several workgroups share its columns
    x, offsets = grouped(counts, 5, 1, depth, torch.bfloat16)
    cols = 40 if len(counts) < 100 else 3
    w = activations(2, len(counts), cols, depth, spread=1.0)
    q = ec.mx_quantize(w)
    stored = ec.mx_experts_product(ec.mx_quantize(x), q, offsets)
    y = ec.mx_experts_linear(x, q, offsets)
    for e, (a, b) in enumerate(parts(offsets)):
        if a < b:
            want = R.mm_bound(R.near(x[a:b]), R.near(w[e]), torch.bfloat16)
            R.check(y[a:b], *want, f"y {e}")
            R.check(stored[a:b], *want, f"stored {e}")
    assert not y[sum(counts):].any() and not stored[sum(counts):].any()


def test_experts_tiles_of_256():
    # enough rows and columns for the largest tile, in one round of workgroups
    counts = [2000, 1, 0, 1700, 300]
    x, offsets = grouped(counts, 60, 1, 384, torch.bfloat16)
    w = activations(2, 5, 3001, 384, spread=1.0)
    y = ec.mx_experts_linear(x, ec.mx_quantize(w), offsets)
    for e, (a, b) in enumerate(parts(offsets)):
        if a < b:
            R.check(y[a:b], *R.mm_bound(R.near(x[a:b]), R.near(w[e]), torch.bfloat16), f"y {e}")
    assert not y[sum(counts):].any()


def test_experts_training_with_tiles_of_256():
    # contractions long enough for the largest tile in all three products
    x, offsets = grouped([2400, 2500], 0, 1, 2600, torch.bfloat16)
    w = activations(2, 2, 2500, 2600, spread=1.0)
    dy = activations(3, 4900, 2500, spread=1.0)
    y, saved = ec.mx_experts_forward(x, w, offsets)
    dx, dw = ec.mx_experts_backward(dy, saved)
    for e, (a, b) in enumerate(parts(offsets)):
        R.check(y[a:b], *R.mm_bound(R.near(x[a:b]), R.near(w[e]), torch.bfloat16), f"y {e}")
        R.check(dx[a:b], *R.mm_bound(R.near(dy[a:b]), R.near(w[e].t()), torch.bfloat16), f"dx {e}")
        R.check(dw[e], *R.mm_bound(R.near(dy[a:b].t()), R.near(x[a:b].t()), torch.bfloat16), f"dw {e}")


@pytest.mark.parametrize("offsets", [[0, 50, 20, 90], [-5, 10, 400, 90], [70, 70, 10, 0], [0, 0, 0, 500]],
                         ids=str)
def test_offsets_out_of_order_stay_in_bounds(offsets):
    # wrong rows, but nothing outside the arrays: the ends of each hold their values
    x = activations(1, 90, 256)
    w = activations(2, 3, 64, 256)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    y = ec.mx_experts_linear(x, ec.mx_quantize(w), off)
    y2, saved = ec.mx_experts_forward(x, w, off)
    dx, dw = ec.mx_experts_backward(y2, saved)
    torch.cuda.synchronize()
    assert y.shape == y2.shape == (90, 64) and dx.shape == x.shape and dw.shape == w.shape


# ---------------------------------------------------------------- how calls run


def test_other_stream_and_repeats():
    x = activations(1, 700, 1000)
    w = activations(2, 900, 1000)
    q = ec.mx_quantize(w)
    want = ec.mx_linear(x, q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = ec.mx_linear(x, q, stream=s)
    a, b = ec.mx_quantize_both(x, stream=s)
    y, saved = ec.mx_linear_forward(x, w, stream=s)
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(y, want)
    same_form(b, x.t())
    for _ in range(5):  # the same inputs give the same bits
        assert torch.equal(ec.mx_linear(x, q), want)


def test_graph_replays_equal_eager_calls():
    x, w = activations(1, 300, 512), activations(2, 4, 256, 512)
    dy = activations(3, 300, 256)
    offsets = torch.tensor([0, 100, 100, 250, 280], dtype=torch.int32, device="cuda")

    def step():
        y, saved = ec.mx_experts_forward(x, w, offsets)
        dx, dw = ec.mx_experts_backward(dy, saved)
        q = ec.mx_quantize(w)
        return y, dx, dw, ec.mx_experts_linear(x, q, offsets), ec.mx_dequantize(ec.mx_quantize(x))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        x.copy_(activations(10 + k, 300, 512))
        offsets.copy_(torch.tensor([0, 10 * k, 60, 200, 300 - k], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, step()):
            assert torch.equal(a, b), k


def test_refusals_on_the_gpu():
    x = activations(1, 4, 64)
    w = ec.mx_quantize(activations(2, 8, 64))
    w3 = ec.mx_quantize(activations(2, 3, 8, 64))
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    for call in (
        lambda: ec.mx_quantize(x.double()),
        lambda: ec.mx_quantize(x.cpu()),
        lambda: ec.mx_quantize(x[:, :0]),
        lambda: ec.mx_quantize_both(x[0]),
        lambda: ec.mx_dequantize(w, torch.float64),
        lambda: ec.mx_linear(x[:, :32], w),
        lambda: ec.mx_linear(x, w3),
        lambda: ec.mx_experts_linear(x, w, off),
        lambda: ec.mx_experts_linear(x, w3, off[:3]),
        lambda: ec.mx_experts_linear(x, w3, off.long()),
        lambda: ec.mx_experts_linear(x, w3, off.cpu()),
        lambda: ec.mx_linear_forward(x, activations(2, 8, 64).float()),
        lambda: ec.mx_linear_backward(x, ec.mx_linear_forward(x, activations(2, 8, 64))[1]),
        lambda: ec.MXTensor(w.codes, w.scales, 129),
        lambda: ec.MXTensor(w.codes[:, ::2], w.scales, 64),
        lambda: ec.mx_product(w, ec.mx_quantize(activations(2, 8, 32))),
    ):
        with pytest.raises(ec.ECError) as e:
            call()
        assert e.value.status == ec.EC_ERR_INVALID
