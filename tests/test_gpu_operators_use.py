"""The operators as programs use them: the example's layer against its definition from end to end,
copies of weights, threads that share a stream."""
import copy
import io
import threading

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import error_bounded_lossy_amd as ec  # noqa: E402
import mxref as R  # noqa: E402
from test_gpu_expert_layer import CASES, layer, setup  # noqa: E402

TYPES = [torch.float32, torch.float16, torch.bfloat16]
ids = lambda v: str(v).replace("torch.", "") if isinstance(v, torch.dtype) else None  # noqa: E731


def groups(offsets):
    at = offsets.tolist()
    return list(enumerate(zip(at, at[1:])))


def gathered(rows, r, weights=None):
    """Each token's sum over its rows in 64 bits, and the sum of magnitudes."""
    parts = torch.where((r.place >= 0)[..., None], rows.double()[r.place.clamp(min=0).long()], 0.0)
    if weights is not None:
        parts = parts * weights.double()[..., None]
    return parts.sum(1), parts.abs().sum(1)


# Stage by stage from the library's own values, as a value near the border of two codes may take
# either of them.
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("tokens,width,hidden,experts,choices,dropped", CASES)
def test_decoding(tokens, width, hidden, experts, choices, dropped, dtype):
    x, up, down, ids, weights, _ = setup(tokens, width, hidden, experts, choices, dropped)
    x, up, down = x.to(dtype), ec.mx_quantize(up), ec.mx_quantize(down)
    y = layer().decode(x, up, down, ids, weights)
    r = ec.expert_sort(ids, experts)
    h = ec.mx_experts_product(ec.expert_dispatch_mx(x, r), up, r.offsets, dtype)
    act = torch.relu(h)
    ys = ec.mx_experts_linear(act, down, r.offsets)
    xs = torch.zeros(tokens * choices, width, dtype=dtype, device="cuda")
    here = r.place >= 0
    xs[r.place[here].long()] = x[torch.arange(tokens, device="cuda")[:, None].expand(-1, choices)[here]]
    form = lambda q, e, n: R.values(R.unpack(q.codes[e]), q.scales[e])[:, :n]  # noqa: E731
    for e, (a, b) in groups(r.offsets):
        if a < b:
            R.check(h[a:b], *R.mm_bound(R.near(xs[a:b]), form(up, e, width), dtype), "h")
            R.check(ys[a:b], *R.mm_bound(R.near(act[a:b]), form(down, e, hidden), dtype), "ys")
    want, size = gathered(ys, r, weights)
    eps, tiny = torch.finfo(dtype).eps / 2, torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    # choices products and additions in fp32, then one rounding
    off = (choices + 1) * 2.0 ** -24 * size
    R.check(y, want, off + eps * (want.abs() + off) + tiny, "y")


@pytest.mark.parametrize("tokens,width,hidden,experts,choices,dropped", CASES)
def test_the_gradient_of_the_input(tokens, width, hidden, experts, choices, dropped):
    x, up, down, ids, weights, dy = setup(tokens, width, hidden, experts, choices, dropped)
    _, grads = layer().train_step(x, up, down, ids, weights, lambda y: dy)
    r = ec.expert_sort(ids, experts)
    h, saved_up = ec.mx_experts_forward(ec.expert_dispatch(x, r), up, r.offsets)
    ys, saved_down = ec.mx_experts_forward(torch.relu(h), down, r.offsets)
    dys, _ = ec.expert_combine_backward(dy, ys, r, weights)
    passed = ec.mx_experts_backward(dys, saved_down)[0] * (h > 0)
    # row by row Q(passed) Q(up^T)^T and its bound, then each token's sum of both
    dxs = torch.zeros(tokens * choices, width, dtype=torch.float64, device="cuda")
    off = torch.zeros_like(dxs)
    for e, (a, b) in groups(r.offsets):
        if a < b:
            dxs[a:b], off[a:b] = R.mm_bound(R.near(passed[a:b]), R.near(up[e].t()), torch.float32)
    want, size = gathered(dxs, r)
    off, _ = gathered(off, r)
    # choices additions in fp32 of values that are off by so much
    R.check(grads["x"], want, off + choices * 2.0 ** -24 * (size + off) * 1.01 + 1e-44, "x")


# ---------------------------------------------------------------- copies


@pytest.mark.parametrize("rows", [1, 9, 300])
def test_products_of_copies_read_the_copies(rows):
    g = torch.Generator("cuda").manual_seed(rows)
    x, w = torch.randn(rows, 300, generator=g, device="cuda"), torch.randn(130, 300, generator=g, device="cuda")
    made = ec.mx_quantize(w)
    given = ec.MXTensor(made.codes.clone(), made.scales.clone(), 300)
    want = ec.mx_linear(x, made)
    for q in (made, given):
        f = io.BytesIO()
        torch.save(q, f)
        f.seek(0)
        copies = [copy.deepcopy(q), copy.deepcopy({"w": [q]})["w"][0], torch.load(f, weights_only=False)]
        q.codes.zero_()
        q.scales.fill_(127)
        for c in copies:
            assert torch.equal(ec.mx_linear(x, c), want)
        assert not ec.mx_linear(x, q).any()
        copies[0].codes.zero_()
        assert not ec.mx_linear(x, copies[0]).any() and torch.equal(ec.mx_linear(x, copies[1]), want)


def test_a_backward_from_a_copy_of_what_was_saved():
    g = torch.Generator("cuda").manual_seed(1)
    x, w = torch.randn(90, 64, generator=g, device="cuda"), torch.randn(3, 40, 64, generator=g, device="cuda")
    offsets = torch.tensor([0, 20, 20, 80], dtype=torch.int32, device="cuda")
    y, saved = ec.mx_experts_forward(x, w, offsets)
    want = ec.mx_experts_backward(y, saved)
    kept = copy.deepcopy(saved)
    offsets[1] = 10
    with pytest.raises(ec.ECError) as e:
        ec.mx_experts_backward(y, saved)
    assert e.value.status == ec.EC_ERR_INVALID
    for got, was in zip(ec.mx_experts_backward(y, kept), want):
        assert torch.equal(got, was)


def test_a_forward_and_its_backward_in_graphs_of_their_own():
    # the offsets' buffer is written to between the captures, and before each replay
    g = torch.Generator("cuda").manual_seed(1)
    x, w = torch.randn(90, 64, generator=g, device="cuda"), torch.randn(3, 40, 64, generator=g, device="cuda")
    dy = torch.randn(90, 40, generator=g, device="cuda")
    offsets = torch.tensor([0, 20, 20, 80], dtype=torch.int32, device="cuda")
    ec.mx_experts_backward(dy, ec.mx_experts_forward(x, w, offsets)[1])
    torch.cuda.synchronize()
    one, two = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(one):
        y, saved = ec.mx_experts_forward(x, w, offsets)
    offsets.copy_(torch.tensor([0, 5, 50, 90], dtype=torch.int32))
    with torch.cuda.graph(two, pool=one.pool()):
        dx, dw = ec.mx_experts_backward(dy, saved)
    for at in ([0, 5, 50, 90], [0, 0, 1, 64], [0, 30, 60, 61], [0, 0, 0, 0]):
        offsets.copy_(torch.tensor(at, dtype=torch.int32))
        one.replay()
        two.replay()
        torch.cuda.synchronize()
        y1, saved1 = ec.mx_experts_forward(x, w, offsets)
        for got, want in zip((y, dx, dw), (y1, *ec.mx_experts_backward(dy, saved1))):
            assert torch.equal(got, want), at


# ---------------------------------------------------------------- threads


def test_threads_that_share_a_stream():
    # calls with a workspace: each thread's results are its own
    g = torch.Generator("cuda").manual_seed(1)
    w = ec.mx_quantize(torch.randn(200, 512, generator=g, device="cuda"))
    xs = [torch.randn(300, 512, generator=g, device="cuda") for _ in range(4)]
    choice = [torch.randint(-1, 16, (3000, 2), generator=g, device="cuda", dtype=torch.int32) for _ in range(4)]
    want = [(ec.mx_linear(x, w), ec.expert_sort(c, 16)) for x, c in zip(xs, choice)]
    torch.cuda.synchronize()
    got, failed = [[] for _ in xs], []

    def work(i):
        try:
            for _ in range(100):
                got[i].append((ec.mx_linear(xs[i], w), ec.expert_sort(choice[i], 16)))
        except Exception as e:  # noqa: BLE001 (a thread's failure is the test's)
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for results, (y, r) in zip(got, want):
        assert len(results) == 100
        for y1, r1 in results:
            assert torch.equal(y1, y) and torch.equal(r1.place, r.place) and torch.equal(r1.order, r.order)
