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


def spread(experts, rows, seed, empty):
    """Unequal counts that add up to rows: one for the first expert, none for some."""
    g = torch.Generator().manual_seed(seed)
    share = torch.rand(experts, generator=g) ** 2
    share[torch.randperm(experts, generator=g)[:empty]] = 0
    share[0] = 0
    counts = (share / share.sum() * rows).int()
    counts[0] = 1
    counts[int(counts.argmax())] += rows - int(counts.sum())
    return counts.tolist()


# The largest tile in each product of an expert layer: y (which a forward computes), dx and dw. Few
# experts and more than 64 (found in two rounds), empty ones first, between and last, rows of no
# expert, contractions of 1 and 2 stages past four, and of none (an empty expert's dw).
EXPERTS = [("y", spread(70, 6000, 1, 9), 60, 2700, 1000), ("y", [0, 2300, 1, 0, 2700, 256, 0], 300, 2600, 2000),
           ("dx", spread(70, 6000, 2, 9), 60, 1000, 2600), ("dx", [2300, 0, 1, 2900], 0, 2100, 2700),
           ("dw", [0, 5000, 1], 0, 2000, 2000), ("dw", [1, 0, 130, 9000, 0], 77, 1700, 1500),
           ("dw", spread(70, 140000, 3, 5), 500, 700, 250)]


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("which,counts,dropped,depth,cols", EXPERTS, ids=lambda v: f"{len(v)}x{sum(v)}" if isinstance(v, list) else str(v))
def test_experts_in_the_largest_tiles(which, counts, dropped, depth, cols, dtype):
    experts, used = len(counts), sum(counts)
    rows, kind = used + dropped, KINDS[dtype]
    sizes = {"y": (rows, cols, R.pad(depth), kind, experts, 0), "dx": (rows, depth, R.pad(cols), kind, experts, 0),
             "dw": (cols, depth, 0, kind, experts, rows)}
    assert ec.lib().ec_mx_product_tile(*sizes[which]) == 256
    offsets = torch.tensor([0] + counts).cumsum(0).int().cuda()
    x, dy = values(1, rows, depth, dtype=dtype), values(3, rows, cols, dtype=dtype)
    w = values(2, experts, cols, depth, dtype=dtype)
    x[used:] = float("nan")  # rows of no expert take no part
    dy[used:] = float("inf")
    y, saved = ec.mx_experts_forward(x, w, offsets)
    dx, dw = ec.mx_experts_backward(dy, saved)
    y1 = ec.mx_experts_linear(x, ec.mx_quantize(w), offsets)
    assert torch.equal(y, y1)
    at = offsets.tolist()
    for e, (a, b) in enumerate(zip(at, at[1:])):
        if a == b:
            assert not dw[e].any()
            continue
        R.check(y[a:b], *R.mm_bound(R.near(x[a:b]), R.near(w[e]), dtype), f"y {e}")
        R.check(dx[a:b], *R.mm_bound(R.near(dy[a:b]), R.near(w[e].t()), dtype), f"dx {e}")
        R.check(dw[e], *R.mm_bound(R.near(dy[a:b].t()), R.near(x[a:b].t()), dtype), f"dw {e}")
    assert not y[used:].any() and not dx[used:].any()


def test_which_tiles_the_expert_tests_reach():
    # every tile in every kind of product, in one file or another
    tile = ec.lib().ec_mx_product_tile
    assert tile(3711, 4100, 384, 2, 6, 0) == 128 and tile(40, 70, 256, 2, 1, 0) == 64
    assert tile(4100, 384, 0, 2, 6, 3711) == 128 and tile(70, 130, 0, 2, 1, 5) == 64
    assert tile(4900, 2500, 2688, 2, 2, 0) == tile(2500, 2600, 0, 2, 2, 4900) == 256
