"""The sums over the rows that make the gradient of a norm's weights, against 64 bits.

Tolerances: h rstd and its product with dy are two roundings, and rstd is off by half of what a sum of a row
is (64 terms one after the other in a lane, whose sums are joined in 8 steps) and 4 more.  A lane adds what
its rows give one after the other (here up to 64); the parts are joined in 64 bits."""
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


@pytest.mark.parametrize("rows,cols", [(1, 64), (65, 1111), (5000, 200), (1001, 1111), (16384, 1024), (300, 20000)])
def test_sums_of_equal_signs(rows, cols):
    g = torch.Generator("cuda").manual_seed(rows)
    x = 0.5 + torch.rand(rows, cols, generator=g, device="cuda")
    got, want, size = dweight(x, torch.rand(rows, cols, generator=g, device="cuda"))
    # (a row longer than 16384 is summed in two rounds)
    assert ((got - want).abs() <= size * U * (FACTORS + 32 + 64 + 1)).all()
