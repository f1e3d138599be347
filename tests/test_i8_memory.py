"""An 8-bit tensor whose memory was replaced, on the CPU: what has its form is read where it is, what has
another is refused before a kernel would read it."""
import pytest

torch = pytest.importorskip("torch")

import error_bounded_lossy_amd as ec  # noqa: E402
from test_mx_binding import gpu, stub  # noqa: E402, F401


def form(rows=6, cols=200):
    codes, scales = torch.zeros(rows, -(-cols // 128) * 128, dtype=torch.int8), torch.zeros(rows)
    return ec.I8Tensor(gpu(codes), gpu(scales), cols)


def half_scales(q):
    q.scales.data = q.scales.data.half()


def doubled_scales(q):
    q.scales.data = q.scales.data.double()


# (on a GPU these come from .data too; a tensor on the CPU takes none of another device)
def scales_elsewhere(q):
    q._scales = torch.zeros(q.scales.shape, device="meta")


def codes_elsewhere(q):
    q.home = torch.zeros(q.codes.shape, dtype=torch.int8, device="meta")


def other_codes(q):
    q.codes.data = q.codes.data.to(torch.int16)


def unsigned_codes(q):
    q.codes.data = q.codes.data.to(torch.uint8)


def reordered_codes(q):
    q.codes.data = torch.zeros(q.codes.shape[::-1], dtype=torch.int8)


def strided_codes(q):
    q.codes.data = torch.zeros(q.codes.shape[::-1], dtype=torch.int8).t()


def strided_scales(q):
    q.scales.data = torch.zeros(2 * q.scales.numel())[::2]


def fewer_scales(q):
    q.scales.data = torch.zeros(q.scales.numel() - 1)


def reshaped_scales(q):
    q.scales.data = torch.zeros(q.scales.numel(), 1)


@pytest.mark.parametrize("change", [half_scales, doubled_scales, scales_elsewhere, codes_elsewhere, other_codes, unsigned_codes,
                                    reordered_codes, strided_codes, strided_scales, fewer_scales, reshaped_scales], ids=lambda f: f.__name__)
def test_memory_of_another_form_is_refused(stub, change):  # noqa: F811
    s = stub()
    q = form()
    ec.i8_dequantize(q)
    calls = len(s.calls)
    change(q)
    for call in (q.pointers, lambda: ec.i8_dequantize(q), lambda: ec.i8_product(q, form(3)), lambda: ec.i8_product(form(3), q)):
        with pytest.raises(ec.ECError) as e:
            call()
        assert e.value.status == ec.EC_ERR_INVALID
    assert len(s.calls) == calls


def test_scales_of_another_type_where_the_right_ones_were(stub):  # noqa: F811
    stub()
    q = form()
    q.pointers()
    q.scales.data = q.scales.data.view(torch.int32)  # the same address and count
    with pytest.raises(ec.ECError):
        q.pointers()
    q = ec.I8Tensor(gpu(torch.zeros(3, 0, dtype=torch.int8)), gpu(torch.zeros(3)), 0)
    q.scales.data = q.scales.data.half()
    with pytest.raises(ec.ECError):
        q.pointers()


def test_memory_of_the_same_form_is_read_where_it_is(stub):  # noqa: F811
    stub()
    q = form()
    q.codes.data, q.scales.data = torch.ones(6, 256, dtype=torch.int8), torch.ones(6)
    assert q.pointers() == (q.codes.data_ptr(), q.scales.data_ptr()) == q.pointers()


@pytest.mark.parametrize("home", [torch.zeros(6 * 260 - 1, dtype=torch.int8), torch.zeros(6 * 260, dtype=torch.uint8), torch.zeros(6 * 260),
                                  torch.zeros(12 * 260, dtype=torch.int8)[::2]], ids=["short", "unsigned", "floats", "strided"])
def test_one_allocation_replaced_by_another(stub, home):  # noqa: F811
    stub()
    q = ec.i8_quantize(gpu(torch.zeros(6, 200)))
    q.home.data = torch.zeros(6 * 260, dtype=torch.int8)
    assert q.pointers() == (q.home.data_ptr(), q.home.data_ptr() + 6 * 256)
    q.home.data = home
    with pytest.raises(ec.ECError):
        q.pointers()


@pytest.mark.parametrize("shape,cols", [((0,), 200), ((3, 0), 5), ((4,), 0), ((), 7)])
def test_empty_forms_have_addresses(stub, shape, cols):  # noqa: F811
    stub()
    p = -(-cols // 128) * 128
    q = ec.I8Tensor(gpu(torch.zeros(*shape, p, dtype=torch.int8)), gpu(torch.zeros(shape)), cols)
    assert len(q.pointers()) == 2
    if cols:
        assert len(ec.i8_quantize(gpu(torch.zeros(*shape, cols))).pointers()) == 2
