"""The token exchange on the GPU against its definition in 64 bits."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import error_bounded_lossy_amd as ec  # noqa: E402
import mxref as R  # noqa: E402

TYPES = [torch.bfloat16, torch.float16, torch.float32]
ids = lambda v: str(v).replace("torch.", "") if isinstance(v, torch.dtype) else None  # noqa: E731


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def choices(seed, tokens, k, experts, dropped=0.1):
    g = gen(seed)
    i = torch.randint(0, experts, (tokens, k), generator=g, device="cuda", dtype=torch.int32)
    i[torch.rand(tokens, k, generator=g, device="cuda") < dropped] = -1
    return i


def randn(seed, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen(seed), device="cuda").to(dtype)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("tokens,k,experts", [(0, 2, 5), (1, 1, 1), (1, 4, 8), (63, 1, 3), (64, 4, 64), (257, 3, 24),
                                              (1000, 2, 1), (1024, 4, 128), (1025, 4, 7), (5000, 4, 1024),
                                              (16384, 4, 128), (300001, 2, 129)])
def test_sort(tokens, k, experts, wide):
    i = choices(tokens + experts, tokens, k, experts)
    if wide:
        i = i.long()
    r = ec.expert_sort(i, experts)
    order, place, offsets = R.sort(i.cpu(), experts)
    assert torch.equal(r.offsets.cpu(), offsets)
    assert torch.equal(r.order.cpu(), order)
    assert torch.equal(r.place.cpu(), place)


@pytest.mark.parametrize("tokens", [200, 9000])
def test_sort_of_one_expert_all_dropped_and_wild_ids(tokens):
    for fill in (3, -1, 8, 2 ** 31 - 1, -(2 ** 31)):
        i = torch.full((tokens, 2), fill, dtype=torch.int32, device="cuda")
        r = ec.expert_sort(i, 8)
        order, place, offsets = R.sort(i.cpu(), 8)
        assert torch.equal(r.order.cpu(), order) and torch.equal(r.place.cpu(), place)
        assert torch.equal(r.offsets.cpu(), offsets)
    far = torch.full((tokens, 2), 2 ** 32 + 3, dtype=torch.int64, device="cuda")
    assert not ec.expert_sort(far, 8).offsets.any()


CASES = [(1, 1, 1, 1), (3, 2, 4, 33), (64, 4, 64, 4096), (70, 3, 5, 127), (33, 1, 8, 128), (129, 4, 24, 1111),
         (40, 6, 16, 9000), (500, 2, 128, 64), (17, 64, 3, 40), (300, 4, 8, 520)]


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("dropped", [0.0, 0.3, 1.0])
@pytest.mark.parametrize("tokens,k,experts,cols", CASES)
def test_exchange(tokens, k, experts, cols, dropped, dtype):
    wtype = TYPES[(tokens + k) % 3]
    i = choices(tokens, tokens, k, experts, dropped)
    r = ec.expert_sort(i, experts)
    place = r.place.long()
    rows, kept = tokens * k, int(r.offsets[-1])
    here = place >= 0
    x, ys = randn(1, tokens, cols, dtype=dtype), randn(2, rows, cols, dtype=dtype)
    dy, dxs = randn(3, tokens, cols, dtype=dtype), randn(4, rows, cols, dtype=dtype)
    w = torch.rand(tokens, k, generator=gen(5), device="cuda").to(wtype)
    # nothing of a dropped choice or of a row of no expert may reach a result
    ys[kept:] = float("nan")
    dxs[kept:] = float("inf")
    w[~here] = float("nan")
    token = torch.arange(tokens, device="cuda")[:, None].expand(-1, k)

    xs = torch.zeros(rows, cols, dtype=dtype, device="cuda")
    xs[place[here]] = x[token[here]]
    assert torch.equal(ec.expert_dispatch(x, r), xs)
    q = ec.expert_dispatch_mx(x, r)
    own = ec.mx_quantize(x)
    codes, scales = torch.zeros_like(q.codes), torch.zeros_like(q.scales)
    codes[place[here]], scales[place[here]] = own.codes[token[here]], own.scales[token[here]]
    assert torch.equal(q.codes, codes) and torch.equal(q.scales, scales) and q.cols == cols

    ysd = torch.where(here[..., None], ys.double()[place.clamp(min=0)], 0.0)
    wd = torch.where(here, w.double(), 0.0)[..., None]
    eps = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    # products and additions in fp32, then one rounding
    size = (ysd * wd).abs().sum(1)
    y = (ysd * wd).sum(1)
    R.check(ec.expert_combine(ys, r, w), y, (k + 1) * 2.0 ** -24 * size + eps * (y.abs() + size * 1e-5) + tiny, "y")
    dxd = torch.where(here[..., None], dxs.double()[place.clamp(min=0)], 0.0)
    dx, size = dxd.sum(1), dxd.abs().sum(1)
    R.check(ec.expert_dispatch_backward(dxs, r), dx, k * 2.0 ** -24 * size + eps * (dx.abs() + size * 1e-5) + tiny, "dx")

    dys, dw = ec.expert_combine_backward(dy, ys, r, w)
    want = torch.zeros(rows, cols, dtype=torch.float64, device="cuda")
    want[place[here]] = dy.double()[token[here]] * wd.expand(-1, -1, 1)[here]
    # one product in fp32 and one rounding
    R.check(dys, want, (2.0 ** -24 + eps) * want.abs() * (1 + 2.0 ** -8) + tiny, "dys")
    dot = (ysd * dy.double()[:, None]).sum(-1)
    size = (ysd * dy.double()[:, None]).abs().sum(-1)
    weps = torch.finfo(wtype).eps / 2
    R.check(dw, dot, (cols + 1) * 2.0 ** -24 * size + weps * (dot.abs() + size * 1e-3) + torch.finfo(wtype).smallest_normal * torch.finfo(wtype).eps, "dweights")
    assert dw.dtype == wtype and not dw[~here].any() and not dys[kept:].any()


def test_gradients_against_differences():
    # y is linear in ys and in the weights: differences give the gradients up to rounding
    tokens, k, experts, cols = 20, 3, 6, 50
    r = ec.expert_sort(choices(1, tokens, k, experts, 0.2), experts)
    ys, dy = randn(2, tokens * k, cols), randn(3, tokens, cols)
    w = torch.rand(tokens, k, generator=gen(4), device="cuda")
    dys, dw = ec.expert_combine_backward(dy, ys, r, w)
    loss = lambda a, b: (ec.expert_combine(a, r, b).double() * dy.double()).sum().item()  # noqa: E731
    # fp32 rounding of y (3 products each) against |dy|, over a difference of 2
    off = 2 * 4 * 2.0 ** -24 * (4 * ys.abs().max() * dy.abs().sum()).item()
    for t, j, c in ((0, 0, 0), (7, 2, 49), (19, 1, 20)):
        up, down = w.clone(), w.clone()
        up[t, j] += 1
        down[t, j] -= 1
        assert abs((loss(ys, up) - loss(ys, down)) / 2 - dw[t, j].item()) <= off
        row = int(r.place[t, j])
        if row >= 0:
            up, down = ys.clone(), ys.clone()
            up[row, c] += 1
            down[row, c] -= 1
            assert abs((loss(up, w) - loss(down, w)) / 2 - dys[row, c].item()) <= off
    x, dxs = randn(5, tokens, cols), randn(6, tokens * k, cols)
    dx = ec.expert_dispatch_backward(dxs, r)
    lin = lambda a: (ec.expert_dispatch(a, r).double() * torch.where(torch.arange(tokens * k, device="cuda")[:, None] < r.offsets[-1], dxs, 0.0).double()).sum().item()  # noqa: E731
    up, down = x.clone(), x.clone()
    up[3, 7] += 1
    down[3, 7] -= 1
    assert abs((lin(up) - lin(down)) / 2 - dx[3, 7].item()) <= 16 * 2.0 ** -24 * (x.abs().max() + 1).item() * dxs.abs().max().item()


def test_strides_streams_and_repeats():
    i = choices(1, 300, 4, 16)
    r = ec.expert_sort(i, 16)
    x = randn(2, 300, 700, dtype=torch.bfloat16)[:, 5:600]
    xs = ec.expert_dispatch(x, r)
    assert torch.equal(xs, ec.expert_dispatch(x.contiguous(), r))
    w = torch.rand(4, 300, generator=gen(3), device="cuda").t()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = ec.expert_combine(xs, r, w, stream=s)
    r2 = ec.expert_sort(i, 16, stream=s)
    dys, dw = ec.expert_combine_backward(x, xs, r, w, stream=s)
    s.synchronize()
    for _ in range(3):
        a, b = ec.expert_combine_backward(x, xs, r, w)
        assert torch.equal(a, dys) and torch.equal(b, dw)
    assert torch.equal(y, ec.expert_combine(xs, r, w)) and torch.equal(r2.place, r.place)


def test_graph_replays_equal_eager_calls():
    i = choices(1, 3000, 4, 32)
    x = randn(2, 3000, 264, dtype=torch.bfloat16)
    w = torch.rand(3000, 4, generator=gen(3), device="cuda")

    def step():
        r = ec.expert_sort(i, 32)
        xs = ec.expert_dispatch(x, r)
        q = ec.expert_dispatch_mx(x, r)
        y = ec.expert_combine(xs, r, w)
        return (r.order, r.place, r.offsets, xs, q.codes, q.scales, y,
                *ec.expert_combine_backward(y, xs, r, w), ec.expert_dispatch_backward(xs, r))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        i.copy_(choices(20 + k, 3000, 4, 32, 0.2 * k))
        x.copy_(randn(30 + k, 3000, 264, dtype=torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, step()):
            assert torch.equal(a, b), k


def test_places_out_of_range_count_as_dropped():
    i = choices(1, 50, 2, 4, 0.0)
    r = ec.expert_sort(i, 4)
    x = randn(2, 50, 96)
    ys = randn(3, 100, 96)
    w = torch.rand(50, 2, generator=gen(4), device="cuda")
    bad = r.place.clone()
    bad[::3] = 100
    bad[1::3] = -7
    wild = ec.Routing(r.order, bad, r.offsets, 50, 2, 4)
    gone = ec.Routing(r.order, torch.where((bad < 0) | (bad >= 100), -1, bad), r.offsets, 50, 2, 4)
    assert torch.equal(ec.expert_combine(ys, wild, w), ec.expert_combine(ys, gone, w))
    assert torch.equal(ec.expert_dispatch_backward(ys, wild), ec.expert_dispatch_backward(ys, gone))
    ec.expert_dispatch(x, wild)
    torch.cuda.synchronize()


def test_refusals_on_the_gpu():
    i = choices(1, 10, 2, 4)
    r = ec.expert_sort(i, 4)
    x, ys = randn(1, 10, 32), randn(2, 20, 32)
    w = torch.rand(10, 2, device="cuda")
    for call in (
        lambda: ec.expert_sort(i.float(), 4),
        lambda: ec.expert_sort(i[:, 0], 4),
        lambda: ec.expert_sort(i.cpu(), 4),
        lambda: ec.expert_sort(i, 0),
        lambda: ec.expert_dispatch(x[:9], r),
        lambda: ec.expert_dispatch(x.double(), r),
        lambda: ec.expert_dispatch_mx(ys, r),
        lambda: ec.expert_dispatch_backward(x, r),
        lambda: ec.expert_combine(x, r, w),
        lambda: ec.expert_combine(ys, r, w[:, :1]),
        lambda: ec.expert_combine(ys, r, w.double()),
        lambda: ec.expert_combine_backward(x, ys.half(), r, w),
        lambda: ec.expert_combine_backward(x[:, :8], ys, r, w),
    ):
        with pytest.raises(ec.ECError) as e:
            call()
        assert e.value.status == ec.EC_ERR_INVALID
    with pytest.raises(ec.ECError) as e:
        ec.expert_sort(i, 1025)
    assert e.value.status == ec.EC_ERR_UNSUPPORTED
    with pytest.raises(ec.ECError) as e:
        ec.expert_combine(randn(1, 130, 8), ec.expert_sort(choices(1, 2, 65, 4), 4), torch.rand(2, 65, device="cuda"))
    assert e.value.status == ec.EC_ERR_UNSUPPORTED
