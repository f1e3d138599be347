"""The C entry points of the 4-bit and exchange operators on buffers with guards on both sides:
offsets, places and ids out of order or range write nothing outside, and forms that the Python
binding does not use (one direction alone, rows of y with a stride)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import error_bounded_lossy_amd as ec  # noqa: E402
import mxref as R  # noqa: E402

KINDS = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
TYPES = list(KINDS)
ids = lambda v: str(v).replace("torch.", "") if isinstance(v, torch.dtype) else None  # noqa: E731
GUARD, MARK = 1 << 20, 0xA5


class Buffers:
    """Outputs, each between two guards; done() waits and looks at all guards."""

    def __init__(self):
        self.all = []

    def __call__(self, dtype, *shape):
        n = torch.Size(shape).numel() * dtype.itemsize
        raw = torch.full((2 * GUARD + (n + 255) // 256 * 256,), MARK, dtype=torch.uint8, device="cuda")
        self.all.append((raw, n))
        return raw[GUARD:GUARD + n].view(dtype).view(shape)

    def done(self):
        torch.cuda.synchronize()
        for raw, n in self.all:
            assert bool((raw[:GUARD] == MARK).all()) and bool((raw[GUARD + n:] == MARK).all())


def values(seed, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(dtype)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def call(name, *args):
    args = [a.data_ptr() if isinstance(a, torch.Tensor) else a for a in args]
    stream = torch.cuda.current_stream().cuda_stream
    assert getattr(ec.lib(), name)(*args, stream) == ec.EC_OK, name


def form(buffers, rows, padded):
    return buffers(torch.uint8, rows, padded // 2), buffers(torch.uint8, rows, padded // 32)


WILD = [[0, 50, 20, 90], [-5, 10, 400, 90], [70, 70, 10, 0], [0, 0, 0, 500], [90, 90, 90, 90],
        [-(2 ** 31), 2 ** 31 - 1, -(2 ** 31), 2 ** 31 - 1], [2 ** 31 - 1] * 4, [0, 90, 0, 90], [0, 1, 0, 2]]


# (rows, contraction and columns of the products: few rows, tiles of 64, 128 and 256)
@pytest.mark.parametrize("rows,depth,cols", [(9, 256, 64), (90, 256, 64), (2000, 300, 2000), (4900, 2600, 2500)])
@pytest.mark.parametrize("offsets", WILD, ids=str)
def test_offsets_out_of_order_write_nothing_outside(offsets, rows, depth, cols):
    experts = len(offsets) - 1
    off = i32([v if abs(v) > 10 ** 6 else v * rows // 90 for v in offsets])
    x, w = values(1, rows, depth), values(2, experts, cols, depth)
    dy = values(3, rows, cols)
    wr, wc = ec.mx_quantize_both(w)
    b = Buffers()
    L = ec.lib()
    pd, pc, pr = R.pad(depth), R.pad(cols), L.ec_mx_padded_groups(rows, experts)
    xr, xc, dr, dc = form(b, rows, pd), form(b, depth, pr), form(b, rows, pc), form(b, cols, pr)
    call("ec_mx_quantize_groups", x, 2, rows, depth, depth, off, experts, *xr, *xc)
    call("ec_mx_quantize_groups", dy, 2, rows, cols, cols, off, experts, *dr, *dc)
    for dtype, kind in KINDS.items():
        y, dx, dw = b(dtype, rows, cols), b(dtype, rows, depth), b(dtype, experts, cols, depth)
        call("ec_mx_product_experts", *xr, rows, wr.codes, wr.scales, cols, pd, off, experts, y, kind)
        call("ec_mx_product_experts", *dr, rows, wc.codes, wc.scales, depth, pc, off, experts, dx, kind)
        call("ec_mx_product_tokens", *dc, cols, *xc, depth, rows, off, experts, dw, kind)
        b.done()
    y = b(torch.bfloat16, rows, cols)
    need = L.ec_mx_linear_workspace_bytes(rows, depth, cols, experts)
    call("ec_mx_linear", x, 2, rows, depth, depth, wr.codes, wr.scales, cols, off, experts, y,
         b(torch.uint8, need) if need else None, need)
    b.done()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("tokens,k,cols", [(50, 2, 96), (33, 4, 33), (300, 3, 1111), (7, 1, 9000)])
def test_places_and_offsets_out_of_range_write_nothing_outside(tokens, k, cols, dtype):
    rows, kind, experts = tokens * k, KINDS[dtype], 4
    g = torch.Generator("cuda").manual_seed(tokens)
    r = ec.expert_sort(torch.randint(-1, experts, (tokens, k), generator=g, device="cuda", dtype=torch.int32), experts)
    place = r.place.reshape(-1).clone()
    wild = torch.tensor([rows, -7, 2 ** 31 - 1, -(2 ** 31), rows + 1], dtype=torch.int32, device="cuda")
    place[::3] = wild[torch.arange(len(place[::3]), device="cuda") % 5]
    place = place.reshape(tokens, k)
    x, ys = values(1, tokens, cols, dtype=dtype), values(2, rows, cols, dtype=dtype)
    w = torch.rand(tokens, k, generator=g, device="cuda")
    here = (place >= 0) & (place < rows)
    at = place[here].long()
    token = torch.arange(tokens, device="cuda")[:, None].expand(-1, k)[here]
    b = Buffers()
    for off in (r.offsets, i32([0, 0, 0, 0, -1]), i32([0, 0, 0, 0, 2 ** 31 - 1]), i32([0, 0, 0, 0, -(2 ** 31)]), i32([0, 0, 0, 0, rows + 3])):
        xs, dys, dw = b(dtype, rows, cols), b(dtype, rows, cols), b(torch.float32, tokens, k)
        q = form(b, rows, R.pad(cols))
        y, dx = b(dtype, tokens, cols), b(dtype, tokens, cols)
        call("ec_expert_dispatch", x, kind, tokens, cols, place, k, off, experts, xs)
        call("ec_expert_dispatch_mx", x, kind, tokens, cols, place, k, off, experts, *q)
        call("ec_expert_combine", ys, kind, tokens, cols, place, k, w, 0, y)
        call("ec_expert_combine_backward", x, ys, kind, tokens, cols, place, k, w, 0, off, experts, dys, dw)
        call("ec_expert_dispatch_backward", ys, kind, tokens, cols, place, k, dx)
        b.done()
        assert not dw[~here].any()
        if off is r.offsets:  # rows with a place hold their token, those of no expert zeros
            kept = int(off[-1])
            assert torch.equal(xs[at], x[token]) and not xs[kept:].any() and not dys[kept:].any()
            own = ec.mx_quantize(x)
            assert torch.equal(q[0][at], own.codes[token]) and torch.equal(q[1][at], own.scales[token])
            assert not q[0][kept:].any() and not q[1][kept:].any()


@pytest.mark.parametrize("tokens", [1, 700, 5000])
@pytest.mark.parametrize("wide", [4, 8])
def test_sorts_write_nothing_outside(tokens, wide):
    g = torch.Generator("cuda").manual_seed(tokens)
    i = torch.randint(-(2 ** 31), 2 ** 31 - 1, (tokens, 2), generator=g, device="cuda")
    i = torch.where(torch.rand(tokens, 2, generator=g, device="cuda") < 0.5, i % 1100, i).to(torch.int32 if wide == 4 else torch.int64)
    for experts in (1, 1000, 1024):
        b = Buffers()
        order, place, offsets = b(torch.int32, tokens * 2), b(torch.int32, tokens, 2), b(torch.int32, experts + 1)
        need = ec.lib().ec_expert_sort_workspace_bytes(tokens * 2, experts)
        call("ec_expert_sort", i, wide, tokens * 2, experts, order, place, offsets, b(torch.uint8, need) if need else None, need)
        b.done()
        for got, want in zip((order, place, offsets), R.sort(i.cpu(), experts)):
            assert torch.equal(got.cpu(), want)


# ---------------------------------------------------------------- forms of C alone


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("batch,rows,cols", [(1, 1, 1), (1, 33, 70), (3, 130, 260), (2, 257, 1000)])
def test_quantization_of_one_direction(batch, rows, cols, dtype):
    kind = KINDS[dtype]
    x = values(1, batch, rows, cols, dtype=dtype)
    want_rows, want_cols = ec.mx_quantize_both(x)
    b = Buffers()
    r, c = form(b, batch * rows, R.pad(cols)), form(b, batch * cols, R.pad(rows))
    call("ec_mx_quantize_both", x, kind, batch, rows, cols, rows * cols, cols, *r, None, None)
    call("ec_mx_quantize_both", x, kind, batch, rows, cols, rows * cols, cols, None, None, *c)
    b.done()
    for got, want in ((r, want_rows), (c, want_cols)):
        assert torch.equal(got[0], want.codes.flatten(0, 1)) and torch.equal(got[1], want.scales.flatten(0, 1))


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("counts", [[5], [1, 0, 40, 0, 130], [300, 0, 2, 128]], ids=str)
def test_quantization_of_groups_in_one_direction(counts, dtype):
    kind, cols, rows, groups = KINDS[dtype], 200, sum(counts), len(counts)
    x = values(1, rows, cols, dtype=dtype)
    off = i32([0] + counts).cumsum(0).int()
    b = Buffers()
    p = ec.lib().ec_mx_padded_groups(rows, groups)
    both, r, c = (*form(b, rows, 256), *form(b, cols, p)), form(b, rows, 256), form(b, cols, p)
    call("ec_mx_quantize_groups", x, kind, rows, cols, cols, off, groups, *both)
    call("ec_mx_quantize_groups", x, kind, rows, cols, cols, off, groups, *r, None, None)
    call("ec_mx_quantize_groups", x, kind, rows, cols, cols, off, groups, None, None, *c)
    b.done()
    for got, want in zip((*r, *c), both):
        assert torch.equal(got, want)
    code, s = R.quantize(x)
    assert torch.equal(R.unpack(r[0]), code.int()) and torch.equal(r[1].int(), s.int())
    at = 0
    for e, n in enumerate(counts):  # a group's part of a column starts at the padded rows before it
        if n:
            first = int(off[e])
            code, s = R.quantize(x[first:first + n].t())
            assert torch.equal(R.unpack(c[0][:, at // 2:(at + R.pad(n)) // 2]), code.int())
            assert torch.equal(c[1][:, at // 32:(at + R.pad(n)) // 32].int(), s.int())
            at += R.pad(n)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,cols,stride", [(1, 5, 9), (40, 129, 131), (300, 1000, 1024), (2000, 2050, 2056)])
def test_values_into_rows_with_a_stride(rows, cols, stride, dtype):
    q = ec.mx_quantize(values(1, rows, cols))
    b = Buffers()
    y = b(dtype, rows, stride)
    mark = y.view(torch.uint8).clone().view(dtype)
    call("ec_mx_dequantize", q.codes, q.scales, rows, cols, y, KINDS[dtype], stride)
    b.done()
    assert torch.equal(y[:, :cols], ec.mx_dequantize(q, dtype))
    assert torch.equal(y[:, cols:].contiguous().view(torch.uint8), mark[:, cols:].contiguous().view(torch.uint8))
