"""Products of 8-bit operands by the tiles that they run as: each test asks the library which it takes.
They are defined bit for bit."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import error_bounded_lossy_amd as ec  # noqa: E402
import layerref as R  # noqa: E402
from test_gpu_i8 import by_expert, codes  # noqa: E402

KINDS = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
TYPES = list(KINDS)
ids = lambda v: str(v).replace("torch.", "") if isinstance(v, torch.dtype) else None  # noqa: E731


def tile(rows, cols, depth, dtype, experts=0):
    return ec.lib().ec_i8_product_tile(rows, cols, R.pad(depth), KINDS[dtype], experts)


def count(side, rows, cols):
    return -(-rows // side) * -(-cols // side)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,depth,cols,side,stages", [
    (300, 128, 500, 64, 4), (300, 640, 501, 64, 4), (1999, 512, 1900, 128, 4), (2000, 1000, 1903, 128, 4), (600, 8192, 8100, 128, 2), (4900, 129, 1000, 128, 2),
    (4700, 380, 1111, 128, 2), (3400, 4990, 3700, 256, 2), (4900, 2048, 2500, 256, 2), (3840, 2048, 4352, 256, 2)])
def test_tiles(rows, depth, cols, side, stages, dtype):
    assert tile(rows, cols, depth, dtype) == side and ec.lib().ec_i8_product_rows_first(rows, cols, R.pad(depth), KINDS[dtype]) == 0
    if side == 128:  # four stages where each tile has a unit of its own
        assert (count(128, rows, cols) <= 256) == (stages == 4)
    a, b = codes(rows, rows, depth), codes(cols, cols, depth)
    assert torch.equal(ec.i8_product(a, b, dtype), R.i8_product(a.codes, a.scales, b.codes, b.scales, dtype))


# Rows past whole tiles of 256 in a launch of their own: by the kernel for few rows, and as tiles.
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,depth,cols,rest", [(4097, 4096, 4096, 16), (4100, 8060, 4096, 16), (4300, 8000, 3900, 64), (2200, 8064, 8190, 64)])
def test_rows_in_two_launches(rows, depth, cols, rest, dtype):
    first = ec.lib().ec_i8_product_rows_first(rows, cols, R.pad(depth), KINDS[dtype])
    assert first == rows // 256 * 256 and tile(first, cols, depth, dtype) == 256 and tile(rows - first, cols, depth, dtype) == rest
    a, b = codes(rows, rows, depth), codes(cols, cols, depth)
    want = R.i8_product(a.codes, a.scales, b.codes, b.scales, dtype)
    assert torch.equal(ec.i8_product(a, b, dtype), want)
    x = (a.codes[:, :depth].float() * a.scales[:, None]).to(dtype)
    q = ec.i8_quantize(x)
    assert torch.equal(ec.i8_linear(x, b), R.i8_product(q.codes, q.scales, b.codes, b.scales, dtype))


# Empty groups first, between and last, groups of one row, whole tiles, and rows of no expert.
GROUPS = [([0, 2300, 1, 0, 2300, 256, 0], 43, 2600, 2500, 256), ([1700, 1600, 1600], 0, 2601, 2500, 256), ([4900], 5, 4000, 2800, 256),
          ([2048, 2048, 1], 700, 300, 2000, 128), ([1, 0, 4000, 800, 99, 0], 0, 250, 1200, 128), ([3, 64, 0, 65, 168], 20, 500, 300, 64)]


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("counts,left,depth,cols,side", GROUPS, ids=lambda v: "-".join(map(str, v)) if isinstance(v, list) else str(v))
def test_tiles_of_experts(counts, left, depth, cols, side, dtype):
    rows, experts = sum(counts) + left, len(counts)
    assert tile(rows, cols, depth, dtype, experts) == side
    a, b = codes(1, rows, depth), codes(2, experts, cols, depth)
    offsets = torch.tensor([0] + counts).cumsum(0).int().cuda()
    assert torch.equal(ec.i8_experts_product(a, b, offsets, dtype), by_expert(a, b, offsets, dtype))


# Outputs of 256 MiB in whole lines are stored past the caches; of other rows of that size they are not.
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=ids)
@pytest.mark.parametrize("depth,side", [(200, 128), (4096, 256)])
def test_outputs_past_the_caches(depth, side, dtype):
    wide = 8192 * 2 // (4 if dtype == torch.float32 else 2)
    for cols in (wide, wide - 1):
        rows = -(-(1 << 28) // (cols * (4 if dtype == torch.float32 else 2))) + 3
        first = ec.lib().ec_i8_product_rows_first(rows, cols, R.pad(depth), KINDS[dtype])
        assert tile(first or rows, cols, depth, dtype) == side and tile(rows, cols, depth, dtype, 3) == side
        a, b = codes(1, rows, depth), codes(2, cols, depth)
        y = ec.i8_product(a, b, dtype)
        assert torch.equal(y, R.i8_product(a.codes, a.scales, b.codes, b.scales, dtype))
        counts = [rows // 2 + 9, 0, rows - rows // 2 - 400]
        w = codes(3, 3, cols, depth)
        offsets = torch.tensor([0] + counts).cumsum(0).int().cuda()
        y = ec.i8_experts_product(a, w, offsets, dtype)
        assert torch.equal(y, by_expert(a, w, offsets, dtype))
