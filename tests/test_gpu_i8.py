"""The 8-bit integer form and its products against their definitions.  Codes, scales and products
are defined bit for bit (quotients and sums are exact or correctly rounded), so they have to be equal."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import error_bounded_lossy_amd as ec  # noqa: E402
import layerref as R  # noqa: E402

TYPES = [torch.float32, torch.float16, torch.bfloat16]
ids = lambda v: str(v).replace("torch.", "") if isinstance(v, torch.dtype) else None  # noqa: E731


def values(seed, *shape, dtype=torch.bfloat16):
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(*shape, generator=g, device="cuda")
    x *= torch.exp(torch.randn(*shape[:-1], 1, generator=g, device="cuda"))
    return x.to(dtype)


def codes(seed, *shape, extreme=False):
    """Any codes, -128 among them, with zeros in the padding, and scales."""
    g = torch.Generator("cuda").manual_seed(seed)
    *lead, cols = shape
    c = torch.randint(-128, 128, shape, generator=g, device="cuda")
    if extreme:
        c = torch.where(c < 0, -128, 127)
    c = torch.nn.functional.pad(c.to(torch.int8), (0, -cols % 128))
    return ec.I8Tensor(c, torch.rand(lead, generator=g, device="cuda") * 0.1, cols)


def same(got, want):
    return torch.equal(got.view(torch.uint8) if got.dtype == torch.int8 else got.nan_to_num(12345.0),
                       want.view(torch.uint8) if want.dtype == torch.int8 else want.nan_to_num(12345.0))


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 8192), (3, 127), (5, 128), (70, 129), (33, 500), (9, 2049),
                                       (257, 1111), (4, 16384), (3, 16385), (2, 40000), (5000, 64)])
def test_quantization_and_its_inverse(rows, cols, dtype):
    x = values(rows * cols, rows, cols, dtype=dtype)
    x[0] = 0
    q = ec.i8_quantize(x)
    want, scales = R.i8_quantize(x.cpu())
    assert q.shape == x.shape and same(q.codes.cpu(), want) and torch.equal(q.scales.cpu(), scales)
    for to in TYPES:
        y = ec.i8_dequantize(q, to)
        assert torch.equal(y.cpu(), (scales[:, None] * want[:, :cols].float()).to(to))


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_rounding_ties_and_borders(dtype):
    # scale 1: halves are ties, and the largest magnitude is 127
    x = torch.arange(-254, 255, device="cuda").float()[None] / 2
    x = torch.cat([x, torch.full((1, 1), 127.0, device="cuda")], 1).to(dtype)
    q = ec.i8_quantize(x)
    want, scales = R.i8_quantize(x.cpu())
    assert scales.item() == 1 and same(q.codes.cpu(), want)
    if dtype == torch.float32:  # subnormal rows: their scales have few digits, or none
        tiny = torch.tensor([[1e-45, -3e-45, 0, 0], [2e-43, -1e-43, 1e-45, 0], [1.2e-38, -1e-38, 1e-39, 1e-45],
                             [3e38, -3.4e38, 1.0, -0.0]], device="cuda")
        q = ec.i8_quantize(tiny)
        want, scales = R.i8_quantize(tiny.cpu())
        assert same(q.codes.cpu(), want) and torch.equal(q.scales.cpu(), scales)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("cols", [5, 700, 20000])
def test_rows_that_are_not_finite_read_as_nan(cols, dtype):
    x = values(1, 6, cols, dtype=dtype)
    x[1, cols - 1], x[2, 0], x[3, cols // 2], x[4, 1] = math.nan, math.inf, -math.inf, -math.nan
    q = ec.i8_quantize(x)
    bad = [1, 2, 3, 4]
    assert torch.isnan(q.scales[bad]).all() and not q.codes[bad].any()
    want, scales = R.i8_quantize(x[[0, 5]].cpu())
    assert same(q.codes[[0, 5]].cpu(), want) and torch.equal(q.scales[[0, 5]].cpu(), scales)
    y = ec.i8_dequantize(q, dtype)
    assert torch.isnan(y[bad]).all() and torch.isfinite(y[[0, 5]]).all()
    p = ec.i8_product(q, ec.i8_quantize(values(2, 40, cols, dtype=dtype)), torch.float32)
    assert torch.isnan(p[bad]).all() and torch.isfinite(p[[0, 5]]).all()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_strides_and_shapes(dtype):
    base = values(3, 40, 300, dtype=dtype)
    for x in (base[:, 7:207], base[::3, :200], base.t()[:100], base[:1, 1:2], base.view(4, 10, 300)[:, :, 5:105],
              base[3], base[:0], base.view(4, 10, 300)[2:3, ::2]):
        q = ec.i8_quantize(x)
        want = ec.i8_quantize(x.contiguous().clone())
        assert q.shape == x.shape and torch.equal(q.codes, want.codes) and torch.equal(q.scales, want.scales)
        assert ec.i8_dequantize(q, dtype).shape == x.shape


SIZES = [(1, 1, 1), (1, 8192, 300), (2, 128, 16), (7, 129, 17), (16, 1000, 100), (17, 128, 64), (40, 300, 65),
         (64, 64, 64), (65, 700, 129), (77, 2500, 1111), (300, 256, 900), (1030, 200, 2100), (500, 520, 5000)]


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,depth,cols", SIZES)
def test_product(rows, depth, cols, dtype):
    a, b = codes(rows, rows, depth), codes(cols + 7, cols, depth)
    y = ec.i8_product(a, b, dtype)
    assert torch.equal(y, R.i8_product(a.codes, a.scales, b.codes, b.scales, dtype))


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_product_of_the_largest_tiles(dtype):
    rows, depth, cols = 3400, 4990, 3700  # ragged tiles of 256 in both directions
    assert ec.lib().ec_i8_product_tile(rows, cols, 5120, 0, 0) == 256
    a, b = codes(1, rows, depth), codes(2, cols, depth)
    assert torch.equal(ec.i8_product(a, b, dtype), R.i8_product(a.codes, a.scales, b.codes, b.scales, dtype))


@pytest.mark.parametrize("rows", [3, 100])
def test_sums_of_the_deepest_contraction_are_exact(rows):
    depth = 130944  # the longest that is taken: 2^14 times it stays below 2^31
    a, b = codes(1, rows, depth, extreme=True), codes(2, 70, depth, extreme=True)
    a.codes[0], b.codes[0], b.codes[1] = -128, -128, 127
    y = ec.i8_product(a, b, torch.float32)
    assert torch.equal(y, R.i8_product(a.codes, a.scales, b.codes, b.scales, torch.float32))


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows", [4097, 4112, 4200, 4351])
def test_rows_past_whole_tiles(rows, dtype):  # some in a launch of their own
    a, b = codes(1, rows, 2000), codes(2, 4100, 2000)
    assert torch.equal(ec.i8_product(a, b, dtype), R.i8_product(a.codes, a.scales, b.codes, b.scales, dtype))


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,depth,cols", [(1, 12200, 5), (1, 40000, 2000), (16, 16384, 4100), (17, 5120, 1), (33, 20000, 40), (64, 6000, 130), (64, 8192, 8100), (65, 8100, 1000),
                                             (200, 9000, 501), (256, 16384, 250), (256, 5249, 66)])
def test_product_in_parts_of_the_contraction(rows, depth, cols, dtype):
    a, b = codes(rows, rows, depth), codes(cols + 7, cols, depth)
    assert ec.lib().ec_i8_product_parts_bytes(rows, cols, a.padded) > 0
    want = R.i8_product(a.codes, a.scales, b.codes, b.scales, dtype)
    assert torch.equal(ec.i8_product(a, b, dtype), want)
    x = values(1, rows, depth + 3, dtype=dtype)[:, :depth]
    q = ec.i8_quantize(x)
    assert torch.equal(ec.i8_linear(x, b), R.i8_product(q.codes, q.scales, b.codes, b.scales, dtype))


def test_what_is_not_finite_in_parts_of_the_contraction():
    x, w = values(1, 40, 9000, dtype=torch.float32), ec.i8_quantize(values(2, 50, 9000))
    assert ec.lib().ec_i8_product_parts_bytes(40, 50, 9088) > 0
    x[3, 8999], x[7, 0], x[11] = math.nan, -math.inf, 0
    y = ec.i8_linear(x, w)
    bad = torch.zeros(40, dtype=torch.bool, device="cuda")
    bad[[3, 7]] = True
    assert torch.equal(y.isnan(), bad[:, None].expand(40, 50)) and not y[11].any()
    q = ec.i8_quantize(x)
    assert same(y, R.i8_product(q.codes, q.scales, w.codes, w.scales, torch.float32))


def split(rows, experts, seed, left=0):
    g = torch.Generator().manual_seed(seed)
    cuts = torch.randint(0, rows - left + 1, (experts - 1,), generator=g).sort().values
    return torch.cat([torch.zeros(1, dtype=torch.long), cuts, torch.tensor([rows - left])]).int().cuda()


def by_expert(a, b, offsets, dtype):
    y = torch.zeros(a.codes.shape[0], b.codes.shape[1], dtype=dtype, device="cuda")
    at = offsets.tolist()
    for e, (i, j) in enumerate(zip(at, at[1:])):
        y[i:j] = R.i8_product(a.codes[i:j], a.scales[i:j], b.codes[e], b.scales[e], dtype)
    return y


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,experts,depth,cols,left", [(1, 1, 5, 9, 0), (5, 32, 300, 40, 2), (128, 32, 2048, 100, 0),
                                                          (200, 3, 129, 65, 50), (900, 8, 256, 700, 1), (3, 1024, 64, 20, 0),
                                                          (2600, 5, 200, 4500, 300), (40, 2, 500, 33, 40)])
def test_products_by_expert(rows, experts, depth, cols, left, dtype):
    a, b = codes(1, rows, depth), codes(2, experts, cols, depth)
    for seed in range(2):
        offsets = split(rows, experts, seed, left)
        y = ec.i8_experts_product(a, b, offsets, dtype)
        assert torch.equal(y, by_expert(a, b, offsets, dtype))
    if experts > 1:  # all rows at one expert, the others have none
        offsets = torch.tensor([0] * experts + [rows], dtype=torch.int32, device="cuda")
        assert torch.equal(ec.i8_experts_product(a, b, offsets, dtype), by_expert(a, b, offsets, dtype))


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,depth,cols", [(1, 8192, 500), (4, 33, 20), (16, 3000, 70), (17, 3000, 70), (100, 257, 300),
                                             (2, 20000, 40), (1, 100000, 40), (0, 100, 10)])
def test_linear_is_quantization_and_product(rows, depth, cols, dtype):
    x, w = values(1, rows, depth + 3, dtype=dtype)[:, :depth], ec.i8_quantize(values(2, cols, depth, dtype=dtype))
    y = ec.i8_linear(x, w)
    q = ec.i8_quantize(x)
    assert y.dtype == dtype and torch.equal(y, R.i8_product(q.codes, q.scales, w.codes, w.scales, dtype))
    three = ec.i8_linear(x[None], w)
    assert three.shape == (1, rows, cols) and torch.equal(three[0], y)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,experts", [(6, 8), (64, 8), (300, 8), (2000, 8)])
def test_experts_linear_is_quantization_and_product(rows, experts, dtype):
    x, w = values(1, rows, 400, dtype=dtype), ec.i8_quantize(values(2, experts, 270, 400, dtype=dtype))
    offsets = split(rows, experts, 5, rows // 6)
    y = ec.i8_experts_linear(x, w, offsets)
    assert torch.equal(y, by_expert(ec.i8_quantize(x), w, offsets, dtype))


def test_dense_rows_are_near_the_values_they_stand_for():
    # each code is off by half a step at most: |y - x w| <= sum |x| s_w / 2 + |w| s_x / 2 + s_x s_w / 4, and three
    # roundings of fp32 on what the form computes
    x, w = values(5, 50, 600, dtype=torch.float32), values(6, 80, 600, dtype=torch.float32)
    q = ec.i8_quantize(w)
    y = ec.i8_linear(x, q).double()
    sx, sw = ec.i8_quantize(x).scales.double()[:, None], q.scales.double()[None]
    xd, wd = x.double(), w.double()
    bound = xd.abs().sum(1, keepdim=True) * sw / 2 + wd.abs().sum(1)[None] * sx / 2 + 600 * sx * sw / 4
    assert ((y - xd @ wd.t()).abs() <= bound * (1 + 1e-5) + y.abs() * 4 * 2.0 ** -24).all()


@pytest.mark.parametrize("tokens,k,experts,cols", [(1, 1, 1, 1), (33, 4, 8, 700), (300, 2, 64, 129), (7, 64, 64, 128), (50, 3, 5, 5000)])
def test_dispatch(tokens, k, experts, cols):
    g = torch.Generator("cuda").manual_seed(tokens)
    r = ec.expert_sort(torch.randint(-1, experts, (tokens, k), generator=g, device="cuda"), experts)
    q = codes(1, tokens, cols)
    xs = ec.expert_dispatch_i8(q, r)
    kept = int(r.offsets[-1])
    token = r.order[:kept].long() // k
    assert xs.shape == (tokens * k, cols)
    assert torch.equal(xs.codes[:kept], q.codes[token]) and torch.equal(xs.scales[:kept], q.scales[token])
    assert not xs.codes[kept:].any() and not xs.scales[kept:].any()
