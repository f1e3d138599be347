"""Parts of 4-bit tensors as tensors of their own: one expert's weights, one rank's rows."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import error_bounded_lossy_amd as ec  # noqa: E402


def randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").bfloat16()


def part(q, a, b):
    return ec.MXTensor(q.codes[a:b], q.scales[a:b], q.cols)


def copied(q):
    return ec.MXTensor(q.codes.clone(), q.scales.clone(), q.cols)


# scales of a row: 4, 8, 12, 16, 36 bytes; rows and products of each kernel
@pytest.mark.parametrize("depth", [100, 130, 300, 512, 1100])
@pytest.mark.parametrize("first", [1, 2, 3])
def test_rows_from_the_middle(first, depth):
    a, b = ec.mx_quantize(randn(1, 340, depth)), ec.mx_quantize(randn(2, 203, depth))
    w = part(b, first, 201)
    w2 = copied(w)
    for rows in (1, 9, 40, 300):
        q = part(a, first, first + rows)
        q2 = copied(q)
        assert torch.equal(ec.mx_dequantize(q), ec.mx_dequantize(q2))
        assert torch.equal(ec.mx_product(q, w), ec.mx_product(q2, w2))
        x = randn(3, rows, depth)
        assert torch.equal(ec.mx_linear(x, w), ec.mx_linear(x, w2))


@pytest.mark.parametrize("tokens", [6, 300])
def test_experts_from_the_middle(tokens):
    # experts of 3 rows of 4 bytes of scales: the second starts at 12 bytes
    w = ec.mx_quantize(randn(1, 4, 3, 100))
    x = randn(2, tokens, 100)
    q = ec.mx_quantize(randn(2, tokens + 1, 100))
    offsets = torch.tensor([0, tokens // 3, tokens - 1], dtype=torch.int32, device="cuda")
    mine = ec.MXTensor(w.codes[1:3], w.scales[1:3], 100)
    sent = part(q, 1, tokens + 1)
    assert torch.equal(ec.mx_experts_linear(x, mine, offsets), ec.mx_experts_linear(x, copied(mine), offsets))
    assert torch.equal(ec.mx_experts_product(sent, mine, offsets),
                       ec.mx_experts_product(copied(sent), copied(mine), offsets))
    one = ec.MXTensor(w.codes[1], w.scales[1], 100)
    assert torch.equal(ec.mx_linear(x, one), ec.mx_linear(x, copied(one)))
