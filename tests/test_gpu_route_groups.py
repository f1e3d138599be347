"""Groups of experts whose best biases cancel in their sums, so that 32 bits do not tell which are taken."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import error_bounded_lossy_amd as ec  # noqa: E402
import layerref as R  # noqa: E402


@pytest.mark.parametrize("tokens", [3000, 40000])  # a wave for each, and several in a wave
@pytest.mark.parametrize("groups,top", [(32, 16), (8, 4)])
@pytest.mark.parametrize("score,size,spread", [("softmax", 0, 1e-3), ("softmax", 3, 1e-3), ("softmax", 10, 1e-3), ("softmax", 300, 1e-2), ("sigmoid", 30, 1e-4), ("sigmoid", 300, 1e-3)])
def test_groups_whose_best_biases_cancel(score, size, spread, groups, top, tokens):
    experts = 64
    n = experts // groups
    g = torch.Generator("cuda").manual_seed(groups + tokens)
    l = spread * torch.randn(tokens, experts, generator=g, device="cuda") + torch.randn(tokens, 1, generator=g, device="cuda")
    b = size * (0.5 + torch.rand(groups, generator=g, device="cuda"))
    bias = torch.full((groups, n), -4.0 * size, device="cuda")
    bias[:, 0], bias[:, n - 1] = b, -b
    s = torch.softmax(l.double(), 1) if score == "softmax" else 1 / (1 + torch.exp(-l.double()))
    by = s.unflatten(1, (groups, n)) + bias.double()
    best = by.sort(-1, descending=True).values[..., :2]
    sums = best.sum(-1)
    # every expert of the chosen groups is taken, so the ids tell the groups
    ids, _ = ec.expert_route(l, top * n, score, bias.flatten(), groups, top)
    got = (ids.long() // n).sort(1).values[:, ::n]
    assert torch.equal(got.repeat_interleave(n, 1), (ids.long() // n).sort(1).values)
    want = sums.sort(dim=1, descending=True).values[:, :top]
    # a score is off by some units of 64 bits in either program, a key and a sum by half a unit
    off = 2.0 ** -53 * (16 + 8 * best.abs().sum(-1).amax(1, keepdim=True))
    assert ((sums.gather(1, got).sort(dim=1, descending=True).values - want).abs() <= off).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups_whose_sums_have_no_number_in_32_bits(score):
    l = torch.randn(40, 64, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    bias = torch.zeros(64, device="cuda")
    bias[8:10], bias[17], bias[30:32], bias[40], bias[50], bias[56:] = 3e38, 3.4e38, 3.2e38, math.inf, -math.inf, -3.3e38
    for top in (1, 2, 4, 7):
        for b in (bias, bias.clamp(max=3.4e38), bias.clamp(max=0.0) - 3.0e38):
            ids, _ = ec.expert_route(l, 6, score, b, 8, top)
            assert torch.equal(ids.cpu(), R.route(l, 6, score, b, 8, top, True, 1.0)[0])
