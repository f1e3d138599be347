"""The norm, the routing and the 8-bit form as programs use them: the example's layer behind a norm and a
trained router, serving in 8 bits, graphs, streams, threads, copies."""
import copy
import math
import threading

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import error_bounded_lossy_amd as ec  # noqa: E402
import layerref as R  # noqa: E402
from test_gpu_expert_layer import layer  # noqa: E402

TYPES = [torch.float32, torch.float16, torch.bfloat16]
ids = lambda v: str(v).replace("torch.", "") if isinstance(v, torch.dtype) else None  # noqa: E731
U = 2.0 ** -24


def randn(seed, *shape, dtype=torch.float32, size=1.0):
    return (torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda") * size).to(dtype)


def groups(offsets):
    at = offsets.tolist()
    return list(enumerate(zip(at, at[1:])))


# ---------------------------------------------------------------- the layer


CASES = [(1, 128, 96, 4, 2), (37, 200, 130, 5, 3), (300, 256, 320, 8, 2), (1500, 320, 256, 16, 4)]


# Stage by stage from the library's own values: a value near the border of two codes may take either of
# them.  Codes and products are exact (the form is defined bit for bit), the rest as in the tests of each.
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("tokens,width,hidden,experts,choices", CASES)
def test_serving_in_8_bits(tokens, width, hidden, experts, choices, dtype):
    x, residual, norm = randn(1, tokens, width, dtype=dtype), randn(2, tokens, width, dtype=dtype), 1 + randn(3, width, dtype=dtype, size=0.1)
    router = ec.i8_quantize(randn(4, experts, width, size=width ** -0.5))
    up, down = (ec.i8_quantize(randn(s, experts, a, b, size=b ** -0.5)) for s, a, b in ((5, hidden, width), (6, width, hidden)))
    y = layer().serve(x, residual, norm, router, up, down, choices)

    q, h = ec.rms_norm_i8(x, norm, residual=residual)
    want = R.norm(h, norm, 1e-6)
    assert torch.equal(h, (x.float() + residual.float()).to(dtype))
    assert ((ec.i8_dequantize(q).double() - want).abs() <= q.scales.double()[:, None] * (0.5 + 127 * 110 * U)).all()
    logits = R.i8_product(q.codes, q.scales, router.codes, router.scales, torch.float32)
    want_ids, want_weights, _ = R.route(logits, choices, "softmax", None, 1, 1, True, 1.0)
    i, weights = ec.expert_route(logits, choices)
    assert torch.equal(i.cpu(), want_ids) and ((weights.cpu().double() - want_weights).abs() <= want_weights * U * 1.001).all()
    r = ec.expert_sort(i, experts)
    token = r.order.long() // choices
    ys = torch.zeros(tokens * choices, width, dtype=dtype, device="cuda")
    for e, (a, b) in groups(r.offsets):
        if a < b:
            t = token[a:b]
            act = torch.relu(R.i8_product(q.codes[t], q.scales[t], up.codes[e], up.scales[e], dtype))
            code, s = (v.cuda() for v in R.i8_quantize(act.cpu()))
            ys[a:b] = R.i8_product(code, s, down.codes[e], down.scales[e], dtype)
    parts = ys[r.place.long()].double() * weights.double()[..., None]
    out, size = parts.sum(1), parts.abs().sum(1)
    eps, tiny = torch.finfo(dtype).eps / 2, torch.finfo(dtype).tiny * torch.finfo(dtype).eps
    off = (choices + 1) * U * size + eps * out.abs() + tiny  # of the combined rows, then the addition of h
    assert ((y.double() - (h.double() + out)).abs() <= off * (1 + eps) + eps * (h.double() + out).abs() + tiny).all()


@pytest.mark.parametrize("tokens,width,hidden,experts,choices", CASES)
def test_gradients_of_norm_and_router(tokens, width, hidden, experts, choices):
    # the experts' own products are in 4 bits and tested elsewhere: here they are taken as they are (their
    # gradients with respect to their input and weights), and what is around them is differentiated in 64 bits
    x, residual, norm = randn(1, tokens, width), randn(2, tokens, width), 1 + randn(3, width, size=0.1)
    router = randn(4, width, experts, size=width ** -0.5)
    up, down = randn(5, experts, hidden, width, size=width ** -0.5), randn(6, experts, width, hidden, size=hidden ** -0.5)
    dy = randn(7, tokens, width)
    module = layer()
    seen = {}
    step = module.train_step

    def kept(n, up, down, i, weights, gradient):
        y, grads = step(n, up, down, i, weights, gradient)
        seen.update(n=n, ids=i, weights=weights, grads=grads, y=y)
        return y, grads

    module.train_step = kept
    y, grads = module.routed_step(x, residual, norm, router, up, down, choices, lambda y: dy)
    assert torch.equal(y, (x + residual) + seen["y"])
    h = (x + residual).double().requires_grad_()
    w, ro = norm.double().requires_grad_(), router.double().requires_grad_()
    n = R.norm(h, w, 1e-6)
    s = torch.softmax(n @ ro, 1)
    mine = s.gather(1, seen["ids"].long())
    mine = mine / mine.sum(1, keepdim=True)
    total = (n * seen["grads"]["x"].double()).sum() + (mine * seen["grads"]["weights"].double()).sum() + (h * dy.double()).sum()
    dh, dnorm, drouter = torch.autograd.grad(total, (h, w, ro))
    # a product in fp32 by the library that multiplies matrices, sums of `width` and `tokens` terms, and the
    # norm's own: relative to the largest of each, 2^-24 for each term in the worst order
    for got, want, terms in ((grads["x"], dh, width + experts), (grads["norm"], dnorm, tokens + width), (grads["router"], drouter, tokens + width)):
        assert ((got.double() - want).abs() <= 4 * terms * U * want.abs().amax() + 1e-12).all()


def test_the_example_runs(capsys, monkeypatch):
    monkeypatch.setattr("sys.argv", ["expert_layer.py", "--tokens", "60", "--width", "128", "--hidden", "160", "--experts", "4", "--steps", "2", "--routed"])
    layer().main()
    lines = capsys.readouterr().out.splitlines()
    assert len(lines) == 3 and all(math.isfinite(float(line.split()[-1])) for line in lines)


# ---------------------------------------------------------------- graphs


def test_a_serving_layer_in_a_graph():
    tokens, width, experts, choices = 50, 256, 8, 2
    x, residual, norm = randn(1, tokens, width, dtype=torch.bfloat16), randn(2, tokens, width, dtype=torch.bfloat16), randn(3, width)
    router = ec.i8_quantize(randn(4, experts, width))
    up, down = ec.i8_quantize(randn(5, experts, 96, width, size=0.1)), ec.i8_quantize(randn(6, experts, width, 96, size=0.1))
    serve = layer().serve
    serve(x, residual, norm, router, up, down, choices)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = serve(x, residual, norm, router, up, down, choices)
    for seed in range(4):
        x.copy_(randn(10 + seed, tokens, width, dtype=torch.bfloat16))
        if seed == 2:
            residual.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, serve(x, residual, norm, router, up, down, choices)), seed


def test_forward_and_backward_in_graphs_of_their_own():
    tokens, width, experts = 300, 192, 40
    x, w, dy, dh = randn(1, tokens, width), randn(2, width), randn(3, tokens, width), randn(4, tokens, width)
    logits, dw, bias = randn(5, tokens, experts), randn(6, tokens, 3), randn(7, experts, size=0.1)
    residual = randn(8, tokens, width)

    def forward():
        y, saved = ec.rms_norm_forward(x, w, residual=residual)
        return y, saved, *ec.expert_route(logits, 3, "sigmoid", bias, 4, 2)

    def backward(saved, i):
        return *ec.rms_norm_backward(dy, saved, dh), ec.expert_route_backward(dw, logits, i, "sigmoid")

    y, saved, i, weights = forward()
    backward(saved, i)
    torch.cuda.synchronize()
    one, two = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(one):
        y, saved, i, weights = forward()
    x.add_(1)
    with torch.cuda.graph(two, pool=one.pool()):
        back = backward(saved, i)
    for seed in range(4):
        for t in (x, residual, logits, dy, dw):
            t.copy_(randn(100 * seed + t.shape[1], *t.shape))
        w.mul_(1.1)
        one.replay()
        eager = forward()
        two.replay()
        torch.cuda.synchronize()
        for got, want in zip((y, saved.h, saved.rstd, i, weights, *back), (eager[0], eager[1].h, eager[1].rstd, *eager[2:], *backward(eager[1], eager[2]))):
            assert torch.equal(got, want), seed


def test_two_graphs_with_workspaces():
    # products that quantize on the way: each graph's workspace is its own, also where they share a pool
    a, b = randn(1, 100, 300), randn(2, 90, 300)
    w = ec.i8_quantize(randn(3, 200, 300))
    ec.i8_linear(a, w)
    torch.cuda.synchronize()
    one, two = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(one):
        y = ec.i8_linear(a, w)
    with torch.cuda.graph(two, pool=one.pool()):
        z = ec.i8_linear(b, w)
    for seed in range(3):
        a.copy_(randn(seed + 10, 100, 300))
        b.copy_(randn(seed + 20, 90, 300))
        one.replay()
        two.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ec.i8_linear(a, w)) and torch.equal(z, ec.i8_linear(b, w))


def test_two_graphs_and_two_streams_with_parts_of_a_contraction():
    a, b, w = randn(1, 100, 9000), randn(2, 60, 9000), ec.i8_quantize(randn(3, 200, 9000))
    q = ec.i8_quantize(a)
    assert ec.lib().ec_i8_product_parts_bytes(100, 200, q.padded) and ec.lib().ec_i8_product_parts_bytes(60, 200, q.padded)
    ec.i8_linear(a, w)
    torch.cuda.synchronize()
    one, two = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(one):
        y, p = ec.i8_linear(a, w), ec.i8_product(q, w)
    with torch.cuda.graph(two):
        z = ec.i8_linear(b, w)
    side = torch.cuda.Stream()
    for seed in range(4):
        a.copy_(randn(seed + 10, 100, 9000))
        b.copy_(randn(seed + 20, 60, 9000))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            two.replay()
        one.replay()
        eager = ec.i8_linear(b, w)
        other = ec.i8_linear(a, w, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(y, ec.i8_linear(a, w)) and torch.equal(z, ec.i8_linear(b, w))
        assert torch.equal(eager, z) and torch.equal(other, y) and torch.equal(p, ec.i8_product(q, w))
        s = ec.i8_quantize(b)
        assert torch.equal(z, R.i8_product(s.codes, s.scales, w.codes, w.scales, b.dtype))


# ---------------------------------------------------------------- streams, threads, copies


def everything(x, w, l, wq, stream=None):
    """Every operator once; the results as tensors."""
    out = []
    n, h = ec.rms_norm(x, w, residual=x, stream=stream)
    y, saved = ec.rms_norm_forward(x, w, stream=stream)
    q, h2 = ec.rms_norm_i8(x, w, residual=x, stream=stream)
    out += [n, h, y, h2, *ec.rms_norm_backward(x, saved, x, stream=stream), ec.i8_dequantize(q, stream=stream)]
    i, weights = ec.expert_route(l, 2, "sigmoid", stream=stream)
    out += [i, weights, ec.expert_route_backward(weights, l, i, "sigmoid", stream=stream)]
    r = ec.expert_sort(i, l.shape[1], stream=stream)
    xs = ec.expert_dispatch_i8(q, r, stream=stream)
    out += [ec.i8_dequantize(xs, torch.bfloat16, stream=stream), ec.i8_experts_product(xs, wq, r.offsets, stream=stream)]
    one = ec.I8Tensor(wq.codes[0], wq.scales[0], wq.cols)
    out += [ec.i8_linear(x, one, stream=stream), ec.i8_product(ec.i8_quantize(x, stream=stream), one, stream=stream)]
    return out + [ec.i8_experts_linear(n.repeat_interleave(2, 0), wq, r.offsets, stream=stream)]


def inputs(seed, tokens=120):
    return randn(seed, tokens, 320, dtype=torch.bfloat16), randn(seed + 1, 320), randn(seed + 2, tokens, 12), ec.i8_quantize(randn(seed + 3, 12, 70, 320))


def test_streams_of_their_own():
    args = inputs(1)
    want = everything(*args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        s.wait_stream(torch.cuda.current_stream())
        given = everything(*args, stream=s)
        with torch.cuda.stream(s):
            within = everything(*args)
        torch.cuda.current_stream().wait_stream(s)
        for a, b, c in zip(given, within, want):
            assert torch.equal(a, c) and torch.equal(b, c)


def test_threads():
    args = [inputs(10 * i, 60 + i) for i in range(4)]
    want = [everything(*a) for a in args]
    torch.cuda.synchronize()
    got, failed = [[] for _ in args], []

    def work(i):
        try:
            for _ in range(15):
                got[i].append(everything(*args[i]))
        except Exception as e:  # noqa: BLE001 (a thread's failure is the test's)
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for results, w in zip(got, want):
        assert len(results) == 15 and all(torch.equal(a, b) for r in results for a, b in zip(r, w))


def test_copies_are_read_where_they_are():
    x, w = randn(1, 20, 200), randn(2, 30, 200)
    for q in (ec.i8_quantize(w), ec.I8Tensor(*(lambda t: (t.codes.clone(), t.scales.clone()))(ec.i8_quantize(w)), 200)):
        other = copy.deepcopy(q)
        want = ec.i8_linear(x, q)
        q.codes.zero_()
        assert torch.equal(ec.i8_linear(x, other), want) and not ec.i8_linear(x, q).any()
    y, saved = ec.rms_norm_forward(x, w[0].clone())
    want = ec.rms_norm_backward(x, saved)
    assert all(torch.equal(a, b) for a, b in zip(ec.rms_norm_backward(x, copy.deepcopy(saved)), want))


def test_results_have_no_history():
    x, w = randn(1, 10, 64).requires_grad_(), randn(2, 64).requires_grad_()
    y, saved = ec.rms_norm_forward(x, w)
    i, weights = ec.expert_route(x, 2)
    for t in (y, weights, *ec.rms_norm_backward(x, saved), ec.i8_linear(x, ec.i8_quantize(x))):
        assert not t.requires_grad
