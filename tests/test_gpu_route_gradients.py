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
    got = ec.expert_route_backward(dw.cuda(), l.cuda(), ids.cuda(), score, renormalize, scale).cpu()
    for t in range(len(l)):
        row = zip(got[t].tolist(), *exact_gradient(l[t].tolist(), ids[t].tolist(), dw[t].tolist(), score, renormalize, scale))
        for e, (d, want, size) in enumerate(row):
            # 64 bits whose exponentials and quotients are good to some 1e-14, then one rounding to fp32
            off = float(abs(want)) * U * (1 + 1e-6) + float(size) * 1e-13 + 2.0 ** -150
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
