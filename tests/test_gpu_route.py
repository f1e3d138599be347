"""The routing of tokens to experts against 64 bits: the same experts, and weights and gradients that are
rounded once from 64 bits (a weight half a step of fp32, a gradient half a step of its type, and the rounding
to fp32 before it)."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import error_bounded_lossy_amd as ec  # noqa: E402
import layerref as R  # noqa: E402

TYPES = [torch.float32, torch.float16, torch.bfloat16]
ids = lambda v: str(v).replace("torch.", "") if isinstance(v, torch.dtype) else None  # noqa: E731
U = 2.0 ** -24


def logits_of(seed, tokens, experts, dtype, closed=0.05):
    g = torch.Generator("cuda").manual_seed(seed)
    l = 2 * torch.randn(tokens, experts, generator=g, device="cuda")
    l[torch.rand(tokens, experts, generator=g, device="cuda") < closed] = -math.inf
    if tokens > 2:
        l[1] = -math.inf  # a row with nothing open
        l[2, 1:] = -math.inf  # and with one expert
    return l.to(dtype)


def check(logits, choices, bias=None, score="softmax", groups=1, top_groups=1, renormalize=True, scale=1.0, seed=9):
    how = dict(score=score, renormalize=renormalize, scale=scale)
    got, weights = ec.expert_route(logits, choices, bias=bias, groups=groups, top_groups=top_groups, **how)
    want, exact, _ = R.route(logits, choices, score, bias, groups, top_groups, renormalize, scale)
    assert got.dtype == torch.int32 and weights.dtype == torch.float32
    assert torch.equal(got.cpu(), want)
    w = weights.cpu().double()
    assert torch.equal(torch.isnan(w), torch.isnan(exact))
    # 64 bits off by some units in the last place, then one rounding; the smallest numbers half a step of fp32's
    fine = ~torch.isnan(exact)
    assert ((w - exact).abs()[fine] <= (exact.abs() * U * (1 + 1e-6) + 2.0 ** -149)[fine]).all()
    g = torch.Generator("cuda").manual_seed(seed)
    dw = torch.randn(got.shape, generator=g, device="cuda")
    dl = ec.expert_route_backward(dw, logits, got, **how)
    assert dl.dtype == logits.dtype and dl.shape == logits.shape
    exact = R.route_backward(dw, logits, got, **how)
    d = dl.cpu().double()
    fine = ~torch.isnan(exact)
    assert torch.isnan(d)[~fine].all() and not torch.isnan(d)[fine].any()
    # differences of terms as large as scale times the gradient's; one or two roundings to fp32 before the last one
    step = torch.finfo(logits.dtype)
    terms = dw.cpu().double().abs().amax(1, keepdim=True) * scale
    off = exact.abs() * (step.eps / 2 + 3 * U) + terms.expand_as(exact) * 2 * U * 1e-3 + step.tiny * step.eps
    # the choice's own part and the mean part of a softmax over all are rounded to fp32 and then added
    off = off + terms.expand_as(exact) * 2 * U
    assert ((d - exact).abs()[fine] <= off[fine]).all()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("tokens,experts,choices", [(1, 1, 1), (3, 4, 2), (33, 8, 8), (20, 15, 3), (9, 60, 6), (8, 64, 64), (5, 65, 4),
                                                    (6, 130, 12), (5, 256, 8), (3, 500, 64), (3, 1024, 10)])
def test_routing(tokens, experts, choices, renormalize, score, dtype):
    l = logits_of(tokens + experts, tokens, experts, dtype)
    check(l, choices, None, score, renormalize=renormalize)
    bias = 0.2 * torch.randn(experts, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    check(l, choices, bias, score, renormalize=renormalize, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [True, False])
@pytest.mark.parametrize("experts,groups,top,choices", [(256, 8, 4, 8), (8, 4, 2, 3), (60, 4, 1, 4), (64, 64, 5, 5), (90, 3, 2, 6),
                                                        (1023, 33, 7, 9), (1000, 5, 2, 16), (160, 20, 3, 8), (32, 2, 1, 16), (12, 4, 4, 12)])
def test_groups(experts, groups, top, choices, biased, score):
    l = logits_of(experts + groups, 12, experts, torch.float32, closed=0.3)
    bias = 0.2 * torch.randn(experts, generator=torch.Generator("cuda").manual_seed(2), device="cuda") if biased else None
    check(l, choices, bias, score, groups, top)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_ties_go_to_the_lowest_index(dtype):
    l = torch.randint(-2, 3, (50, 96), generator=torch.Generator("cuda").manual_seed(3), device="cuda").to(dtype)
    l[0] = 0
    l[1, ::2] = -0.0
    l[1, 1::2] = 0.0
    check(l, 9)
    check(l, 9, torch.zeros(96, device="cuda"))
    check(l, 9, score="sigmoid", bias=torch.zeros(96, device="cuda"), groups=8, top_groups=3)
    got, _ = ec.expert_route(l, 9)
    assert got[0].tolist() == list(range(9)) and got[1].tolist() == list(range(9))


def test_what_is_not_finite():
    l = torch.randn(8, 40, generator=torch.Generator("cuda").manual_seed(4), device="cuda")
    l[1, 7] = math.nan
    l[2, 3] = math.inf
    l[3] = math.nan
    l[4, :] = torch.finfo(torch.float32).min  # masked by the type's lowest value: as any number
    l[5, 5] = 3e38
    l[6] = -1e30
    l[7] = -math.inf
    for score in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            check(l, 4, None, score, renormalize=renormalize)
    bias = torch.zeros(40, device="cuda")
    bias[0], bias[1] = -math.inf, math.inf  # never, and always
    check(l[:1], 40, bias, "sigmoid")
    assert ec.expert_route(l[:1], 39, bias=bias, score="sigmoid")[0][0, 0] == 1
    i, w = ec.expert_route(l[7:], 4)
    assert (i == -1).all() and not w.any()


def test_scores_too_small_for_a_sum():
    l = torch.tensor([[-800.0, -801.0, -1e4, -700.5], [-200.0, -201.0, -300.0, -100.0]], device="cuda")
    check(l, 3, score="sigmoid")
    check(l, 3, score="softmax", renormalize=False)


def test_ids_of_a_callers_own():
    # the same expert twice, dropped choices, ids out of range
    l = torch.randn(5, 20, generator=torch.Generator("cuda").manual_seed(5), device="cuda")
    i = torch.tensor([[3, 3, 1], [-1, 4, 4], [20, 2, -7], [0, 0, 0], [-1, -1, 99]], dtype=torch.int32, device="cuda")
    dw = torch.randn(5, 3, generator=torch.Generator("cuda").manual_seed(6), device="cuda")
    for score in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            d = ec.expert_route_backward(dw, l, i, score, renormalize, 1.5).cpu().double()
            want = R.route_backward(dw, l, i, score, renormalize, 1.5)
            assert ((d - want).abs() <= 8 * U * (want.abs() + 1.5 * dw.abs().amax().item())).all()


def test_gradient_against_differences():
    l = torch.randn(3, 16, generator=torch.Generator("cuda").manual_seed(7), device="cuda")
    dw = torch.randn(3, 4, generator=torch.Generator("cuda").manual_seed(8), device="cuda")
    for score in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            i, _ = ec.expert_route(l, 4, score, renormalize=renormalize)
            d = ec.expert_route_backward(dw, l, i, score, renormalize)

            def loss(v):
                s = torch.softmax(v, 1) if score == "softmax" else torch.sigmoid(v)
                m = s.gather(1, i.long())
                return ((m / m.sum(1, keepdim=True) if renormalize else m) * dw.double()).sum()

            for t, e in ((0, int(i[0, 0])), (1, int(i[1, 3])), (2, 5)):
                h = torch.zeros(3, 16, dtype=torch.float64, device="cuda")
                h[t, e] = 1e-5
                slope = (loss(l.double() + h) - loss(l.double() - h)) / 2e-5
                assert abs(slope - d[t, e].double()) <= 1e-6


def test_strides_and_no_tokens():
    base = torch.randn(30, 100, generator=torch.Generator("cuda").manual_seed(10), device="cuda")
    for l in (base[:, 3:40], base[::2, :50], base.t()[:60, :20], base[:0], base[:1]):
        got, want = ec.expert_route(l, 3), ec.expert_route(l.contiguous().clone(), 3)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        dw = torch.ones_like(got[1])
        assert torch.equal(ec.expert_route_backward(dw, l, got[0], renormalize=False),
                           ec.expert_route_backward(dw, l.contiguous().clone(), got[0], renormalize=False))


@pytest.mark.parametrize("choices", [1, 8])
def test_many_tokens(choices):
    l = logits_of(1, 40000, 32, torch.bfloat16)
    i, w = ec.expert_route(l, choices, "sigmoid")
    key = l.float()
    order = torch.sort(key, dim=1, descending=True, stable=True)
    want = torch.where(order.values[:, :choices] > -math.inf, order.indices[:, :choices], -1)
    assert torch.equal(i.long(), want)
    assert torch.allclose(w.sum(1), (i >= 0).any(1).float(), atol=1e-6)


@pytest.mark.parametrize("tokens", [40, 5000])
@pytest.mark.parametrize("experts,groups,top", [(64, 1, 1), (256, 8, 4), (40, 4, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scores_next_to_each_other_go_by_64_bits(score, experts, groups, top, tokens):
    # score + bias differ by parts of a unit of 32 bits, in clusters longer than the choices, or are equal
    g = torch.Generator("cuda").manual_seed(experts)
    l = torch.randn(tokens, experts, generator=g, device="cuda") * torch.rand(tokens, 1, generator=g, device="cuda") * 1e-6
    l[::3] = (l[::3] * 1e6).round() / 4
    l += torch.randn(tokens, 1, generator=g, device="cuda")
    bias = 1e-9 * torch.randint(-3, 4, (experts,), generator=g, device="cuda").float()
    s = torch.softmax(l.double(), 1) if score == "softmax" else 1 / (1 + torch.exp(-l.double()))
    by = s + bias.double()
    if groups > 1:
        best = by.unflatten(1, (groups, -1)).sort(-1, descending=True).values[..., :2].sum(-1)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :top]
        inside = torch.zeros_like(best, dtype=torch.bool).scatter_(1, kept, True)
        by = torch.where(inside[..., None], by.unflatten(1, (groups, -1)), -math.inf).flatten(1)
    got, _ = ec.expert_route(l, 7, score, bias, groups, top)
    # equal in one program's 64 bits may be a unit apart in another's: what is taken has to be as large
    mine = by.gather(1, got.long())
    want = torch.sort(by, dim=1, descending=True, stable=True)
    assert ((mine - want.values[:, :7]).abs() <= 4e-16 * (1 + mine.abs())).all()
    assert (got.sort(1).values.diff(dim=1) > 0).all()
    # without a bias the logits decide, exactly
    got, _ = ec.expert_route(l, 7, score)
    assert torch.equal(got.long(), torch.sort(l, dim=1, descending=True, stable=True).indices[:, :7])
