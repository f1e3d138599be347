"""Products on the GPU by the tiles that they run as: each test asks the library which it takes."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import error_bounded_lossy_amd as ec  # noqa: E402
import mxref as R  # noqa: E402

KINDS = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
TYPES = list(KINDS)
ids = lambda v: str(v).replace("torch.", "") if isinstance(v, torch.dtype) else None  # noqa: E731


def values(seed, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(dtype)


# Rows past whole tiles of 256 that go to a launch of their own: by the kernel for few rows, and as
# tiles of each size.
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,depth,cols,rest", [(4100, 8000, 4096, 16), (4300, 7999, 3900, 64), (2200, 8064, 8190, 128)])
def test_rows_in_two_launches(rows, depth, cols, rest, dtype):
    first = ec.lib().ec_mx_product_rows_first(rows, cols, R.pad(depth), KINDS[dtype])
    assert first == rows // 256 * 256
    assert ec.lib().ec_mx_product_tile(first, cols, R.pad(depth), KINDS[dtype], 0, 0) == 256
    assert ec.lib().ec_mx_product_tile(rows - first, cols, R.pad(depth), KINDS[dtype], 0, 0) == rest
    x, w = values(rows, rows, depth, dtype=dtype), values(cols, cols, depth, dtype=dtype)
    y, bound = R.mm_bound(R.near(x), R.near(w), dtype)
    R.check(ec.mx_linear(x, ec.mx_quantize(w)), y, bound)
