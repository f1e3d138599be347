"""The norm, the routing and the 8-bit form in plain torch, in 64 bits, from their definitions."""
import math

import torch


def pad(cols):
    return -(-cols // 128) * 128


def i8_quantize(x):
    """Codes (int8, padded) and scales: the definition itself is in fp32 (a correctly rounded
    quotient twice), so this is exact."""
    x = x.float()
    m = x.abs().amax(-1)
    ok = torch.isfinite(m)
    s = torch.where(ok, m / 127.0, math.nan)
    by = torch.where(ok & (s > 0), s, math.inf)
    q = torch.round(x / by[..., None]).clamp(-127, 127)
    q = torch.where(ok[..., None], q, 0.0).nan_to_num(0.0)
    return torch.nn.functional.pad(q.to(torch.int8), (0, -x.shape[-1] % 128)), s


def i8_product(ac, a_scales, bc, b_scales, dtype):
    """Whole sums (below 2^53, so exact in float64), then fp32 as the form defines it."""
    acc = ac.double() @ bc.double().t()
    return (acc.float() * a_scales[:, None] * b_scales[None, :]).to(dtype)


def norm(h, weight, eps):
    h = h.double()
    return h * (h.square().mean(-1, keepdim=True) + eps).rsqrt() * weight.double()


def route(logits, choices, score, bias, groups, top_groups, renormalize, scale):
    """ids [tokens, choices], weights and scores in float64, one token at a time."""
    l = logits.double().cpu()
    tokens, experts = l.shape
    ids = torch.full((tokens, choices), -1, dtype=torch.int32)
    if score == "softmax":
        top = l.amax(1, keepdim=True)
        e = torch.exp(l - torch.where(top > -math.inf, top, 0.0))
        total = e.sum(1, keepdim=True)
        s = e / torch.where(total == 0, 1.0, total)
    else:
        s = 1 / (1 + torch.exp(-l))
    b = torch.zeros(experts, dtype=torch.float64) if bias is None else bias.double().cpu()
    by = s + b
    size = experts // groups
    big = lambda v: math.inf if v != v else v  # noqa: E731
    for t in range(tokens):
        open_ = [float(l[t, e]) != -math.inf and not float(by[t, e]) == -math.inf for e in range(experts)]
        if groups > 1 and top_groups < groups:
            sums = []
            for g in range(groups):
                v = sorted((big(float(by[t, e])) for e in range(g * size, (g + 1) * size) if open_[e]), reverse=True)[:2]
                sums.append(sum(v) if v else -math.inf)
            kept = sorted(range(groups), key=lambda g: (-sums[g], g))[:top_groups]
            open_ = [o and e // size in kept for e, o in enumerate(open_)]
        key = l[t] if bias is None else by[t]
        order = sorted((e for e in range(experts) if open_[e]),
                       key=lambda e: (0, 0.0, e) if float(key[e]) != float(key[e]) else (1, -float(key[e]), e))
        for j, e in enumerate(order[:choices]):
            ids[t, j] = e
    here = ids >= 0
    at = ids.clamp(min=0).long()
    if renormalize:
        # softmax of the chosen log scores: sums that have no digits do no harm
        logs = l if score == "softmax" else torch.where(l > -700, -torch.log1p(torch.exp(-l.clamp(min=-700))), l)
        mine = torch.where(here, logs.gather(1, at), -math.inf)
        top = mine.amax(1, keepdim=True)
        e = torch.exp(mine - torch.where(top > -math.inf, top, 0.0))
        total = e.sum(1, keepdim=True)
        w = e / torch.where(total == 0, 1.0, total)
    else:
        w = torch.where(here, s.gather(1, at), 0.0)
    return ids, torch.where(here, scale * w, 0.0), s


def route_backward(dweights, logits, ids, score, renormalize, scale):
    """dlogits in float64 by torch's differentiation of the weights' formula."""
    l = logits.double().cpu().clone().requires_grad_()
    ids = ids.cpu()
    here = (ids >= 0) & (ids < l.shape[1])
    at = torch.where(here, ids, 0).long()
    here = here & (l.detach().gather(1, at) != -math.inf)
    if score == "softmax":
        top = l.detach().amax(1, keepdim=True)
        e = torch.exp(l - torch.where(top > -math.inf, top, 0.0))
        total = e.sum(1, keepdim=True)
        s = e / torch.where(total == 0, 1.0, total)
    else:
        s = torch.sigmoid(l)
    mine = torch.where(here, s.gather(1, at), 0.0)
    if renormalize:
        # as in route(): the softmax of the chosen log scores, which has digits where the scores have none
        chosen = l.gather(1, at)
        logs = chosen if score == "softmax" else torch.where(chosen > -700, -torch.log1p(torch.exp(-chosen.clamp(min=-700))), chosen)
        logs = torch.where(here, logs, -math.inf)
        top = logs.detach().amax(1, keepdim=True)
        e = torch.exp(logs - torch.where(top > -math.inf, top, 0.0))
        total = e.sum(1, keepdim=True)
        mine = e / torch.where(total == 0, 1.0, total)
    w = scale * mine
    dl = torch.autograd.grad(w, l, torch.where(here, dweights.double().cpu(), 0.0))[0]
    if renormalize or score == "sigmoid":
        # The weights do not depend on the other logits (a softmax's sum cancels): their gradient is
        # zero, where differentiation through a row with a NaN has 0 times NaN.
        mine = torch.zeros(l.shape, dtype=torch.int32).scatter_add_(1, at, here.int()) > 0
        dl = torch.where(mine, dl, 0.0)
    return dl
