"""The C entry points of the norm, the routing and the 8-bit form on buffers with guards on both sides:
offsets, places and ids out of order or range write nothing outside, and forms that the Python binding
does not use."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import error_bounded_lossy_amd as ec  # noqa: E402
import layerref as R  # noqa: E402
from test_gpu_operators_abi import KINDS, TYPES, WILD, Buffers, call, i32, ids, values  # noqa: E402


def i8(rows, depth, seed=1):
    return ec.i8_quantize(values(seed, rows, depth))


# (rows, contraction and columns: tiles of 64, 128 and 256)
@pytest.mark.parametrize("rows,depth,cols", [(9, 256, 64), (90, 256, 65), (2000, 300, 2000), (4900, 2600, 2500)])
@pytest.mark.parametrize("offsets", WILD, ids=str)
def test_offsets_out_of_order_write_nothing_outside(offsets, rows, depth, cols):
    experts = len(offsets) - 1
    off = i32([v if abs(v) > 10 ** 6 else v * rows // 90 for v in offsets])
    x, p = values(1, rows, depth), R.pad(depth)
    w = ec.i8_quantize(values(2, experts, cols, depth))
    b = Buffers()
    codes, scales = b(torch.int8, rows, p), b(torch.float32, rows)
    call("ec_i8_quantize", x, 2, rows, depth, depth, codes, scales)
    for dtype, kind in KINDS.items():
        call("ec_i8_product_experts", codes, scales, rows, w.codes, w.scales, cols, p, off, experts, b(dtype, rows, cols), kind)
        b.done()
    need = ec.lib().ec_i8_linear_workspace_bytes(rows, depth, cols, experts)
    call("ec_i8_linear", x, 2, rows, depth, depth, w.codes, w.scales, cols, off, experts, b(torch.bfloat16, rows, cols), b(torch.uint8, need), need)
    b.done()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,depth,cols", [(1, 1, 1), (1, 4000, 33), (3, 200, 17), (16, 129, 100), (16, 20000, 16), (17, 64, 65), (130, 500, 131), (300, 128, 257)])
def test_products_write_nothing_outside(rows, depth, cols, dtype):
    a, w, kind = i8(rows, depth), i8(cols, depth, 2), KINDS[dtype]
    b = Buffers()
    y, z = b(dtype, rows, cols), b(dtype, rows, cols)
    call("ec_i8_product", a.codes, a.scales, rows, w.codes, w.scales, cols, a.padded, y, kind)
    x = values(1, rows, depth).to(dtype)
    need = ec.lib().ec_i8_linear_workspace_bytes(rows, depth, cols, 0)
    call("ec_i8_linear", x, kind, rows, depth, depth, w.codes, w.scales, cols, None, 0, z, b(torch.uint8, need) if need else None, need)
    b.done()
    assert torch.equal(y, R.i8_product(a.codes, a.scales, w.codes, w.scales, dtype))


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,depth,cols", [(17, 64, 65), (17, 5100, 65), (47, 20000, 3), (1, 12288, 130), (16, 12161, 129), (130, 8200, 131), (256, 5300, 257)])
def test_products_in_parts_write_nothing_outside(rows, depth, cols, dtype):
    a, w, kind = i8(rows, depth), i8(cols, depth, 2), KINDS[dtype]
    b = Buffers()
    y, z = b(dtype, rows, cols), b(dtype, rows, cols)
    need = ec.lib().ec_i8_product_parts_bytes(rows, cols, a.padded)
    assert (need > 0) == (depth > 64)
    call("ec_i8_product_parts", a.codes, a.scales, rows, w.codes, w.scales, cols, a.padded, y, kind, b(torch.uint8, need) if need else None, need)
    x = values(1, rows, depth).to(dtype)
    more = ec.lib().ec_i8_linear_workspace_bytes(rows, depth, cols, 0)
    # up to 16384 codes of up to 16 rows are quantized in the product's kernel, with no workspace
    assert more == 0 if rows <= 16 and rows * a.padded <= 16384 else more >= need + rows * (a.padded + 4)
    call("ec_i8_linear", x, kind, rows, depth, depth, w.codes, w.scales, cols, None, 0, z, b(torch.uint8, more) if more else None, more)
    b.done()
    q = ec.i8_quantize(x)
    assert torch.equal(y, R.i8_product(a.codes, a.scales, w.codes, w.scales, dtype))
    assert torch.equal(z, R.i8_product(q.codes, q.scales, w.codes, w.scales, dtype))


@pytest.mark.parametrize("tokens,k,cols", [(50, 2, 96), (33, 4, 33), (300, 3, 1111), (7, 1, 9000)])
def test_places_and_offsets_out_of_range_write_nothing_outside(tokens, k, cols):
    rows, experts = tokens * k, 4
    g = torch.Generator("cuda").manual_seed(tokens)
    r = ec.expert_sort(torch.randint(-1, experts, (tokens, k), generator=g, device="cuda", dtype=torch.int32), experts)
    place = r.place.reshape(-1).clone()
    wild = torch.tensor([rows, -7, 2 ** 31 - 1, -(2 ** 31), rows + 1], dtype=torch.int32, device="cuda")
    place[::3] = wild[torch.arange(len(place[::3]), device="cuda") % 5]
    place = place.reshape(tokens, k)
    q = i8(tokens, cols)
    here = (place >= 0) & (place < rows)
    at = place[here].long()
    token = torch.arange(tokens, device="cuda")[:, None].expand(-1, k)[here]
    b = Buffers()
    for off in (r.offsets, i32([0, 0, 0, 0, -1]), i32([0, 0, 0, 0, 2 ** 31 - 1]), i32([0, 0, 0, 0, -(2 ** 31)]), i32([0, 0, 0, 0, rows + 3])):
        codes, scales = b(torch.int8, rows, q.padded), b(torch.float32, rows)
        call("ec_expert_dispatch_i8", q.codes, q.scales, tokens, q.padded, place, k, off, experts, codes, scales)
        b.done()
        if off is r.offsets:
            kept = int(off[-1])
            assert torch.equal(codes[at], q.codes[token]) and torch.equal(scales[at], q.scales[token])
            assert not codes[kept:].any() and not scales[kept:].any()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,cols,stride", [(1, 5, 9), (40, 129, 131), (300, 1000, 1024), (2000, 2050, 2056), (3, 20000, 20001)])
def test_rows_write_nothing_outside(rows, cols, stride, dtype):
    kind, p = KINDS[dtype], R.pad(cols)
    x, r, w = (values(i, n, stride, dtype=dtype) for i, n in ((1, rows), (2, rows), (3, 1)))
    b = Buffers()
    codes, scales, y = b(torch.int8, rows, p), b(torch.float32, rows), b(dtype, rows, stride)
    call("ec_i8_quantize", x, kind, rows, cols, stride, codes, scales)
    mark = y.view(torch.uint8).clone().view(dtype)
    call("ec_i8_dequantize", codes, scales, rows, cols, y, kind, stride)
    b.done()
    q = ec.i8_quantize(x[:, :cols])
    assert torch.equal(codes, q.codes) and torch.equal(scales, q.scales) and torch.equal(y[:, :cols], ec.i8_dequantize(q, dtype))
    assert torch.equal(y[:, cols:].contiguous().view(torch.uint8), mark[:, cols:].contiguous().view(torch.uint8))
    h, n, rstd = b(dtype, rows, cols), b(dtype, rows, cols), b(torch.float32, rows)
    call("ec_rms_norm", x, stride, r, stride, kind, rows, cols, w, kind, 1e-5, h, n, rstd)
    codes, scales = b(torch.int8, rows, p), b(torch.float32, rows)
    call("ec_rms_norm_i8", x, stride, None, 0, kind, rows, cols, w, kind, 1e-5, None, codes, scales)
    need = ec.lib().ec_rms_norm_backward_workspace_bytes(rows, cols)
    dx, dw = b(dtype, rows, cols), b(dtype, cols)
    dy = values(4, rows, cols, dtype=dtype)
    call("ec_rms_norm_backward", dy, h, None, kind, rows, cols, rstd, w, kind, dx, dw, b(torch.uint8, need) if need else None, need)
    b.done()
    y2, saved = ec.rms_norm_forward(x[:, :cols], w[0, :cols], 1e-5, residual=r[:, :cols])
    assert torch.equal(n, y2) and torch.equal(h, saved.h) and torch.equal(rstd, saved.rstd)
    for got, want in zip((dx, dw), ec.rms_norm_backward(dy, saved)):
        assert torch.equal(got, want)
    q = ec.rms_norm_i8(x[:, :cols], w[0, :cols], 1e-5)
    assert torch.equal(codes, q.codes) and torch.equal(scales, q.scales)


def test_a_norm_of_no_rows_has_zeros_for_its_weights():
    b = Buffers()
    dw = b(torch.float32, 300)
    call("ec_rms_norm_backward", None, None, None, 0, 0, 300, None, None, 0, None, dw, None, 0)
    b.done()
    assert not dw.any()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("tokens,experts,groups,k", [(1, 1, 1, 1), (5, 6, 3, 2), (100, 60, 4, 5), (33, 257, 1, 8), (3, 1024, 64, 64), (9000, 64, 8, 4), (20000, 100, 1, 2)])
def test_routing_writes_nothing_outside(tokens, experts, groups, k, dtype):
    kind, stride = KINDS[dtype], experts + 3
    l = values(tokens, tokens, stride, dtype=dtype)
    g = torch.Generator("cuda").manual_seed(experts)
    bias, dw = torch.randn(experts, generator=g, device="cuda"), torch.randn(tokens, k, generator=g, device="cuda")
    wild = torch.randint(-(2 ** 31), 2 ** 31 - 1, (tokens, k), generator=g, device="cuda").int()
    wild[::2] %= experts
    b = Buffers()
    for score in (0, 1):
        for use, renormalize in ((None, 1), (bias, 0)):
            top = -(-k * groups // experts) if groups > 1 else 1
            i, w, d = b(torch.int32, tokens, k), b(torch.float32, tokens, k), b(dtype, tokens, experts)
            call("ec_expert_route", l, kind, tokens, stride, experts, use, k, score, groups, top, renormalize, 1.5, i, w)
            b.done()
            assert bool(((i >= 0) & (i < experts)).all())
            call("ec_expert_route_backward", dw, l, kind, tokens, stride, experts, wild, k, score, renormalize, 1.5, d)
            b.done()
            want = R.route_backward(dw[:50], l[:50, :experts], wild[:50], ("softmax", "sigmoid")[score], bool(renormalize), 1.5)
            off = want.abs() * torch.finfo(dtype).eps / 2 + 8 * 2.0 ** -24 * (want.abs() + 1.5 * dw.abs().amax().item()) + torch.finfo(dtype).tiny * torch.finfo(dtype).eps
            assert ((d[:50].cpu().double() - want).abs() <= off).all()
