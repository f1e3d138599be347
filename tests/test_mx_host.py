"""Host-side checks of the 4-bit format's and the token exchange's entry points: sizes, and
refusals before anything is enqueued (no GPU)."""
import pytest

import error_bounded_lossy_amd as ec

OK, INVALID, CAPACITY, UNSUPPORTED = (ec.EC_OK, ec.EC_ERR_INVALID, ec.EC_ERR_CAPACITY, ec.EC_ERR_UNSUPPORTED)
F = 1 << 20  # a pointer that is never dereferenced: every call below fails its checks or has no work
BF16 = 2


@pytest.fixture(scope="module")
def L():
    return ec.lib()


def test_sizes(L):
    assert [L.ec_mx_padded(n) for n in (0, 1, 128, 129)] == [0, 128, 128, 256]
    # every nonempty group may round up by 127
    for rows, groups in ((0, 4), (1, 4), (5, 3), (128, 1), (1000, 16), (4, 1000)):
        p = L.ec_mx_padded_groups(rows, groups)
        most = 0
        used = min(groups, rows)
        if used:
            # the worst split: all but one group hold one row
            most = (used - 1) * 128 + -(-(rows - used + 1) // 128) * 128
        assert p % 128 == 0 and most <= p <= rows + 127 * used
    assert L.ec_mx_linear_workspace_bytes(0, 4096, 10, 0) == 0
    assert L.ec_mx_linear_workspace_bytes(1, 4096, 10, 0) == 0
    assert L.ec_mx_linear_workspace_bytes(100, 4096, 10, 0) == 100 * (2048 + 128)
    assert L.ec_mx_linear_workspace_bytes(101, 100, 10, 0) == 101 * 64 + 101 * 4
    assert L.ec_expert_sort_workspace_bytes(100, 8) == 0
    assert L.ec_expert_sort_workspace_bytes(1 << 20, 8) % (9 * 4) == 0


def test_quantize_refusals(L):
    q = L.ec_mx_quantize
    assert q(None, BF16, 0, 8, 8, F, F, None) == OK
    assert q(F, 3, 1, 8, 8, F, F, None) == INVALID
    assert q(F, -1, 1, 8, 8, F, F, None) == INVALID
    assert q(F, BF16, 1, 0, 8, F, F, None) == INVALID
    assert q(F, BF16, 1, 8, 7, F, F, None) == INVALID
    assert q(None, BF16, 1, 8, 8, F, F, None) == INVALID
    assert q(F + 1, BF16, 1, 8, 8, F, F, None) == INVALID
    assert q(F + 2, 0, 1, 8, 8, F, F, None) == INVALID
    assert q(F, BF16, 1, 8, 8, F + 8, F, None) == INVALID
    assert q(F, BF16, 1, 8, 8, F, None, None) == INVALID
    assert q(F, BF16, 1, (1 << 24) + 1, 1 << 25, F, F, None) == UNSUPPORTED
    assert q(F, BF16, 1 << 31, 8, 8, F, F, None) == UNSUPPORTED
    b = L.ec_mx_quantize_both
    assert b(F, BF16, 1, 4, 8, 0, 8, None, None, None, None, None) == INVALID
    assert b(F, BF16, 1, 4, 8, 0, 8, F, None, F, F, None) == INVALID
    assert b(F, BF16, 1, 4, 8, 0, 8, F, F, F, F + 4, None) == INVALID
    assert b(F, BF16, 1, 1 << 25, 8, 0, 8, F, F, F, F, None) == UNSUPPORTED
    assert b(F, BF16, 1025, 4, 8, 32, 8, F, F, F, F, None) == UNSUPPORTED
    assert b(F, BF16, 0, 4, 8, 32, 8, F, F, F, F, None) == OK
    g = L.ec_mx_quantize_groups
    assert g(F, BF16, 4, 8, 8, None, 2, F, F, F, F, None) == INVALID
    assert g(F, BF16, 4, 8, 8, F + 2, 2, F, F, F, F, None) == INVALID
    assert g(F, BF16, 4, 8, 8, F, 0, F, F, F, F, None) == INVALID
    assert g(F, BF16, 4, 8, 8, F, 1025, F, F, F, F, None) == UNSUPPORTED
    d = L.ec_mx_dequantize
    assert d(F, F, 0, 8, F, BF16, 8, None) == OK
    assert d(F, F, 1, 8, None, BF16, 8, None) == INVALID
    assert d(F, F, 1, 8, F + 1, BF16, 8, None) == INVALID
    assert d(F, F + 1, 1, 8, F, BF16, 8, None) == INVALID
    assert d(F, F, 1, 8, F, 7, 8, None) == INVALID
    assert d(F, F, 1, 8, F, BF16, 4, None) == INVALID


def test_product_refusals(L):
    p = L.ec_mx_product
    assert p(F, F, 0, F, F, 8, 128, F, BF16, None) == OK
    assert p(F, F, 1, F, F, 0, 128, F, BF16, None) == INVALID
    assert p(F, F, 1, F, F, 8, 100, F, BF16, None) == INVALID
    assert p(F, F, 1, F, F, 8, 0, F, BF16, None) == INVALID
    assert p(F, F, 1, F, F, 8, 128, F, 5, None) == INVALID
    assert p(F, F, 1, F, F, 8, 128, None, BF16, None) == INVALID
    assert p(F + 4, F, 1, F, F, 8, 128, F, BF16, None) == INVALID
    assert p(F, F, 1, None, F, 8, 128, F, BF16, None) == INVALID
    assert p(F, F, 1, F, F, 8, (1 << 24) + 128, F, BF16, None) == UNSUPPORTED
    assert p(F, F, 1 << 31, F, F, 8, 128, F, BF16, None) == UNSUPPORTED
    e = L.ec_mx_product_experts
    assert e(F, F, 1, F, F, 8, 128, None, 2, F, BF16, None) == INVALID
    assert e(F, F, 1, F, F, 8, 128, F, 0, F, BF16, None) == INVALID
    assert e(F, F, 1, F, F, 8, 128, F, 1025, F, BF16, None) == UNSUPPORTED
    t = L.ec_mx_product_tokens
    assert t(F, F, 0, F, F, 8, 10, F, 2, F, BF16, None) == OK
    assert t(F, F, 8, F, F, 8, 10, F + 1, 2, F, BF16, None) == INVALID
    assert t(F, None, 8, F, F, 8, 10, F, 2, F, BF16, None) == INVALID
    assert t(F, F, 8, F, F, 8, 1 << 25, F, 2, F, BF16, None) == UNSUPPORTED
    lin = L.ec_mx_linear
    need = L.ec_mx_linear_workspace_bytes(100, 64, 8, 0)
    assert lin(F, BF16, 0, 64, 64, F, F, 8, None, 0, F, None, 0, None) == OK
    assert lin(F, BF16, 100, 64, 64, F, F, 8, None, 0, F, None, 0, None) == INVALID
    assert lin(F, BF16, 100, 64, 64, F, F, 8, None, 0, F, F, need - 1, None) == CAPACITY
    assert lin(F, BF16, 100, 64, 64, F, F, 8, None, 0, F, F + 8, need, None) == INVALID
    assert lin(F, BF16, 1, 64, 63, F, F, 8, None, 0, F, None, 0, None) == INVALID
    assert lin(F, BF16, 1, 64, 64, F, F, 8, F, 0, F, None, 0, None) == INVALID
    assert lin(F, BF16, 1, 64, 64, F, F, 8, None, 3, F, None, 0, None) == INVALID
    assert lin(F, BF16, 1, 64, 64, F, F, 0, None, 0, F, None, 0, None) == INVALID
    assert lin(F, BF16, 1, 64, 64, F, F, 8, F, 1025, F, None, 0, None) == UNSUPPORTED


def test_exchange_refusals(L):
    s = L.ec_expert_sort
    assert s(F, 4, 10, 0, F, F, F, None, 0, None) == INVALID
    assert s(F, 4, 10, 1025, F, F, F, None, 0, None) == UNSUPPORTED
    assert s(F, 2, 10, 4, F, F, F, None, 0, None) == INVALID
    assert s(F + 4, 8, 10, 4, F, F, F, None, 0, None) == INVALID
    assert s(F, 4, 10, 4, None, F, F, None, 0, None) == INVALID
    assert s(F, 4, 10, 4, F, F, None, None, 0, None) == INVALID
    assert s(F, 4, 1 << 31, 4, F, F, F, F, 1 << 30, None) == UNSUPPORTED
    assert s(F, 4, 1 << 20, 4, F, F, F, None, 0, None) == INVALID
    assert s(F, 4, 1 << 20, 4, F, F, F, F, 16, None) == CAPACITY
    d = L.ec_expert_dispatch
    assert d(F, BF16, 0, 8, F, 2, F, 4, F, None) == OK
    assert d(F, BF16, 1, 0, F, 2, F, 4, F, None) == INVALID
    assert d(F, BF16, 1, 8, F, 0, F, 4, F, None) == INVALID
    assert d(F, BF16, 1, 8, F, 65, F, 4, F, None) == UNSUPPORTED
    assert d(F, BF16, 1 << 30, 8, F, 4, F, 4, F, None) == UNSUPPORTED
    assert d(F, BF16, 1, 8, None, 2, F, 4, F, None) == INVALID
    assert d(F, BF16, 1, 8, F, 2, None, 4, F, None) == INVALID
    assert d(F, BF16, 1, 8, F, 2, F, 0, F, None) == INVALID
    assert d(F, 9, 1, 8, F, 2, F, 4, F, None) == INVALID
    m = L.ec_expert_dispatch_mx
    assert m(F, BF16, 1, 8, F, 2, F, 4, F + 8, F, None) == INVALID
    assert m(F, BF16, 1, 8, F, 2, F, 4, F, None, None) == INVALID
    b = L.ec_expert_dispatch_backward
    assert b(F + 1, BF16, 1, 8, F, 2, F, None) == INVALID
    assert b(F, BF16, 1, 8, F, 2, None, None) == INVALID
    c = L.ec_expert_combine
    assert c(F, BF16, 1, 8, F, 2, F, 4, F, None) == INVALID
    assert c(F, BF16, 1, 8, F, 2, None, 0, F, None) == INVALID
    assert c(F, BF16, 1, 8, F, 2, F + 2, 0, F, None) == INVALID
    assert c(F, BF16, 0, 8, F, 2, None, 0, None, None) == OK
    k = L.ec_expert_combine_backward
    assert k(F, F, BF16, 1, 8, F, 2, F, 0, None, 4, F, F, None) == INVALID
    assert k(F, F, BF16, 1, 8, F, 2, F, 0, F, 4, F, None, None) == INVALID
    assert k(F, None, BF16, 1, 8, F, 2, F, 0, F, 4, F, F, None) == INVALID
    assert k(F, F, BF16, 1, 8, F, 2, F, 3, F, 4, F, F, None) == INVALID


def test_binding_refuses_tensors_of_the_host():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 64)
    q = ec.MXTensor(torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8), 64)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: ec.mx_quantize(x), lambda: ec.mx_quantize_both(x), lambda: ec.mx_dequantize(q),
                 lambda: ec.mx_linear(x, q), lambda: ec.mx_product(q, q), lambda: ec.mx_linear_forward(x, x),
                 lambda: ec.expert_sort(ids, 4), lambda: ec.mx_quantize(x, stream=object())):
        with pytest.raises(ec.ECError) as e:
            call()
        assert e.value.status == INVALID
    for codes, scales, cols in ((q.codes, q.scales, 129), (q.codes[:, ::2], q.scales, 64),
                                (q.codes.int(), q.scales, 64), (q.codes[:3], q.scales, 64)):
        with pytest.raises(ec.ECError):
            ec.MXTensor(codes, scales, cols)


def test_scales_that_are_read_start_at_words(L):
    # (4-byte aligned ones are taken: a part of a tensor's rows, tested on the GPU)
    for off in (1, 2, 3, 6):
        assert L.ec_mx_dequantize(F, F + off, 1, 8, F, BF16, 8, None) == INVALID
        assert L.ec_mx_product(F, F + off, 1, F, F, 8, 128, F, BF16, None) == INVALID
        assert L.ec_mx_product(F, F, 1, F, F + off, 8, 128, F, BF16, None) == INVALID
        assert L.ec_mx_linear(F, BF16, 1, 64, 64, F, F + off, 8, None, 0, F, None, 0, None) == INVALID
    for off in (4, 8, 12):  # codes, and scales that are written
        assert L.ec_mx_dequantize(F + off, F, 1, 8, F, BF16, 8, None) == INVALID
        assert L.ec_mx_quantize(F, BF16, 1, 8, 8, F, F + off, None) == INVALID
        assert L.ec_expert_dispatch_mx(F, BF16, 1, 8, F, 2, F, 4, F, F + off, None) == INVALID


F32 = 0


def test_tiles_of_products(L):
    tile = L.ec_mx_product_tile
    assert [tile(r, 8192, 8192, BF16, 0, 0) for r in (1, 16, 17, 64, 8192)] == [16, 16, 64, 64, 256]
    assert tile(1024, 4096, 4096, BF16, 0, 0) == 128 and tile(1024, 4096, 4096, BF16, 4, 0) == 128
    assert tile(0, 8, 128, BF16, 0, 0) == tile(8, 8, 128, 7, 0, 0) == tile(8, 8, 128, BF16, 0, 5) == 0
    # stores weigh more in fp32: 8192 x 8192 of a contraction of 2048 take 117 us with tiles of 128, 143
    # with tiles of 256, in bf16 112 and 98
    assert tile(8192, 8192, 2048, F32, 0, 0) == 128 and tile(8192, 8192, 2048, BF16, 0, 0) == 256
    assert tile(8192, 8192, 8192, F32, 0, 0) == 256
    # where rounds and starts weigh the same, a few experts change nothing
    assert tile(32768, 2048, 4096, BF16, 64, 0) == 256 and tile(2500, 2600, 0, BF16, 2, 4900) == 256


def test_rows_that_go_first_depend_on_the_columns(L):
    first = L.ec_mx_product_rows_first
    # the rest's launch is cheap, and saves most of a round: 66 us in one, 52 in two
    assert first(4100, 4096, 4096, BF16) == 4096 and first(4346, 16384, 2048, BF16) == 4096
    # its 250 rows are a round of large tiles themselves: 152 us in one, 166 in two; 82 and 95 in fp32
    assert first(506, 57344, 8192, BF16) == 0 and first(4346, 16384, 1024, F32) == 0
    # short contractions: 38 us in one, 44 in two
    assert first(4100, 8190, 1024, BF16) == 0
    # whole tiles, or none
    assert first(4096, 4096, 4096, BF16) == first(255, 57344, 8192, BF16) == 0


def test_tokens_of_the_longest_row_in_groups(L):
    # what quantization per group takes, the product over the tokens takes too: the missing y is
    # what these calls are refused for
    for experts in (1, 16, 1024):
        assert L.ec_mx_product_tokens(F, F, 8, F, F, 8, 1 << 24, F, experts, None, BF16, None) == INVALID
        assert L.ec_mx_product_tokens(F, F, 8, F, F, 8, (1 << 24) + 1, F, experts, None, BF16, None) == UNSUPPORTED
        assert L.ec_mx_quantize_groups(None, BF16, 1 << 24, 8, 8, F, experts, F, F, F, F, None) == INVALID
        assert L.ec_mx_quantize_groups(None, BF16, (1 << 24) + 1, 8, 8, F, experts, F, F, F, F, None) == UNSUPPORTED
