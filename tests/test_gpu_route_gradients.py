"""Gradients of the routing in rows that are nearly certain, relative to their own size."""
from decimal import Decimal, getcontext

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import error_bounded_lossy_amd as ec  # noqa: E402

U = 2.0 ** -24


def exact_gradient(logits, ids, dweights, score, renormalize, scale):
    """A row's dlogits by the definition in 60 digits, and how large the terms of the differences are that it
    is made of."""
    getcontext().prec = 60
    l, n = [Decimal(v) for v in logits], len(logits)
    d = [Decimal(v) * Decimal(scale) for v in dweights]
    if score == "softmax":
        e = [(v - max(l)).exp() for v in l]
        s = [v / sum(e) for v in e]
        slope = [1] * n
    else:
        s = [1 / (1 + (-v).exp()) for v in l]
        slope = [1 - v for v in s]
    if renormalize:  # between the chosen ones; a softmax's factors 1 - s go with the sum
        w = [s[i] / sum(s[j] for j in ids) for i in ids]
        mean, grad, size = sum(a * b for a, b in zip(w, d)), [Decimal(0)] * n, [Decimal(0)] * n
        for j, i in enumerate(ids):
            grad[i] += w[j] * (d[j] - mean) * slope[i]
            size[i] += w[j] * sum(a * abs(d[j] - b) for a, b in zip(w, d)) * slope[i]
        return grad, size
    ds = [Decimal(0)] * n
    for j, i in enumerate(ids):
        ds[i] += d[j]
    if score == "sigmoid":
        return [a * b * c for a, b, c in zip(s, slope, ds)], [a * b * abs(c) for a, b, c in zip(s, slope, ds)]
    mean = sum(a * b for a, b in zip(s, ds))
    return ([a * (b - mean) for a, b in zip(s, ds)],
            [a * sum(c * abs(b - x) for c, x in zip(s, ds)) for a, b in zip(s, ds)])


MODES = [("softmax", False), ("softmax", True), ("sigmoid", True), ("sigmoid", False)]  # and whether weights are renormalised
GAPS = [0.0, 4.0, 10.0, 14.0, 17.0, 20.0, 25.0, 30.0, 40.0, 60.0, 85.0]


def check_gradient(l, ids, dw, score, renormalize, scale=1.0):
    kind = torch.finfo(l.dtype)
    step, least = (0.0, 2.0 ** -150) if l.dtype == torch.float32 else (kind.eps / 2, kind.tiny * kind.eps)
    got = ec.expert_route_backward(dw.cuda(), l.cuda(), ids.cuda(), score, renormalize, scale).cpu()
    for t in range(len(l)):
        row = zip(got[t].tolist(), *exact_gradient(l[t].tolist(), ids[t].tolist(), dw[t].tolist(), score, renormalize, scale))
        for e, (d, want, size) in enumerate(row):
            # 64 bits whose exponentials and quotients are good to some 1e-14, one rounding to fp32, and of a
            # 16-bit type another
            off = float(abs(want)) * (U + step) * (1 + 1e-6) + float(size) * 1e-13 + least
            assert abs(d - float(want)) <= off, (t, e, d, float(want), off)


@pytest.mark.parametrize("score,renormalize", MODES)
@pytest.mark.parametrize("experts,choices", [(4, 1), (4, 2), (20, 3), (60, 8), (64, 1), (130, 4), (300, 2)])
def test_gradients_of_rows_that_are_nearly_certain(experts, choices, renormalize, score):
    g = torch.Generator().manual_seed(experts + choices)
    l = torch.randn(len(GAPS), experts, generator=g)
    top = torch.randint(0, experts, (len(GAPS), 1), generator=g)
    l.scatter_(1, top, l.amax(1, keepdim=True) + torch.tensor(GAPS)[:, None])
    if score == "sigmoid":  # all near one end, or some near either
        l = l - torch.tensor([0.0, 5.0, 20.0, 40.0])[torch.arange(len(GAPS)) % 4][:, None]
    ids = l.sort(dim=1, descending=True).indices[:, :choices].int()
    check_gradient(l, ids, torch.randn(len(GAPS), choices, generator=g), score, renormalize, 2.5)
    # without the likeliest, in another order, and equal gradients, which cancel
    if choices < experts:
        ids = l.sort(dim=1, descending=True).indices[:, 1:choices + 1].flip(1).int()
        check_gradient(l, ids, torch.randn(len(GAPS), choices, generator=g), score, renormalize)
    ids = l.sort(dim=1, descending=True).indices[:, :choices].int()
    check_gradient(l, ids, torch.full((len(GAPS), choices), 0.7), score, renormalize)


@pytest.mark.parametrize("score,renormalize", MODES)
@pytest.mark.parametrize("experts", [6, 200])
def test_gradients_of_an_expert_chosen_twice(experts, renormalize, score):
    g = torch.Generator().manual_seed(experts)
    l = torch.randn(4, experts, generator=g)
    l[:, 2] += torch.tensor([0.0, 9.0, 19.0, 30.0])
    ids = torch.tensor([[2, 2, 1], [2, 3, 2], [1, 2, 1], [2, 2, 2]], dtype=torch.int32)
    dw = torch.randn(4, 3, generator=g)
    check_gradient(l, ids, dw, score, renormalize)
    dw[:, 1] = -dw[:, 0] * (1 + 1e-6)  # the two parts nearly cancel
    check_gradient(l, ids, dw, score, renormalize)


@pytest.mark.parametrize("score,renormalize", MODES)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["float16", "bfloat16"])
def test_gradients_in_16_bits(dtype, renormalize, score):
    g = torch.Generator().manual_seed(7)
    l = torch.randn(6, 70, generator=g)
    l[:, 9] += torch.tensor([0.0, 3.0, 8.0, 12.0, 20.0, 60.0])
    ids = l.sort(dim=1, descending=True).indices[:, :5].int()
    check_gradient(l.to(dtype), ids, torch.randn(6, 5, generator=g), score, renormalize, 2.5)


@pytest.mark.parametrize("score,renormalize", MODES)
def test_gradients_of_scores_without_digits(renormalize, score):
    # sigmoids whose sum 64 bits do not hold, beside some that they do, and scores that 32 bits do not
    l = torch.tensor([[-800.0, -801.0, -820.0, -1e4], [-599.0, -601.0, -700.5, -605.25], [-90.0, -100.0, -104.5, -120.0],
                      [95.0, 100.0, 104.5, 300.0], [-700.0, 0.5, -1.0, 700.0]])
    ids = torch.tensor([[0, 1, 2], [0, 1, 3], [1, 0, 2], [3, 2, 1], [1, 2, 0]], dtype=torch.int32)
    check_gradient(l, ids, torch.randn(5, 3, generator=torch.Generator().manual_seed(8)), score, renormalize, 0.5)
