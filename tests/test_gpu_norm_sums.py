"""The sums over the rows that make the gradient of a norm's weights, against 64 bits.

Tolerances: h rstd and its product with dy are two roundings, and rstd is off by half of what a sum of a row
is (64 terms one after the other in a lane, whose sums are joined in 8 steps) and 4 more.  A lane adds what
256 rows give one after the other, then such sums; the parts are joined in 64 bits."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import error_bounded_lossy_amd as ec  # noqa: E402

U = 2.0 ** -24
FACTORS = 2 + 4 + (64 + 8) / 2


def dweight(x, dy, dtype=torch.float32):
    """The gradient, its exact value and the sum of its terms' magnitudes."""
    _, saved = ec.rms_norm_forward(x, torch.ones(x.shape[1], device="cuda", dtype=dtype))
    _, dw = ec.rms_norm_backward(dy, saved)
    h = x.double()
    terms = dy.double() * h * (h.square().mean(1, keepdim=True) + 1e-6).rsqrt()
    return dw.double(), terms.sum(0), terms.abs().sum(0)


# Small terms behind a large one: 8192 parts (512 workgroups of 16 rows), the first of them 1, the others 2^-25, which
# 32 bits lose one by one.
def test_parts_are_joined_in_64_bits():
    rows = 1 << 20
    dy = torch.full((rows, 64), 2.0 ** -25 / 128, device="cuda")
    dy[0] = 1
    got, want, size = dweight(torch.ones(rows, 64, device="cuda"), dy)
    assert ((got - want).abs() <= size * U * (FACTORS + 1)).all()


# The same in a lane: a large term first, then 2^-25 from up to 2047 rows, of which 255 are lost and not all. Whole runs,
# one row more, and none behind the first.
@pytest.mark.parametrize("rows", [1 << 24, (1 << 24) - 5, 256 * 8192, 256 * 8192 + 1, 512 * 8192])
def test_rows_of_a_lane_are_added_in_runs(rows):
    dy = torch.full((rows, 8), 2.0 ** -25, device="cuda")
    dy[:8192] = 1
    got, want, size = dweight(torch.ones(rows, 8, device="cuda"), dy)
    assert ((got - want).abs() <= size * U * (FACTORS + 256 + 8 + 1)).all()


@pytest.mark.parametrize("rows,cols", [(1, 64), (65, 1111), (5000, 200), (1001, 1111), (16384, 1024), (300, 20000), (70000, 8192), (1 << 22, 65)])
def test_sums_of_equal_signs(rows, cols):
    g = torch.Generator("cuda").manual_seed(rows)
    x = 0.5 + torch.rand(rows, cols, generator=g, device="cuda")
    got, want, size = dweight(x, torch.rand(rows, cols, generator=g, device="cuda"))
    # up to 1024 rows of a lane, in 4 runs; a row longer than 16384 is summed in two rounds
    assert ((got - want).abs() <= size * U * (FACTORS + 32 + min(rows, 256) + 4 + 1)).all()
