"""Measured cases of the operators around an expert layer: the root-mean-square norm with the residual's addition
(in its own type for training, in 8 bits for serving), the routing of tokens to experts, and products of 8-bit
integers with a scale for each token and channel, dense and by expert.

`listed()` gives the cases, `draw(rng)` further ones of the same ranges, `prepare` the inputs, `run` one
pass (`own` false: plain torch in 32 bits, `own` true: the library's kernels), `exact` the same results
in 64 bits from the definitions, `work` what one pass has to move and compute.

Norm: h = x + residual rounded to x's type, y = h / sqrt(mean(h^2) + eps) * weight.
8 bits: a row has the scale s = max|y| / 127 in float32, its codes are y / s rounded to whole numbers, ties to
even; a row of zeros has s = 0. Rows are padded with zeros to a multiple of 128 codes.
Routing: the score of an expert is softmax or sigmoid of the token's logits. Experts are chosen by score + bias
(without a bias: by logit), the largest first, ties to the lowest index; with groups (consecutive experts, as many
each) only those of the groups whose two best sum highest. An expert whose logit is -inf is never chosen: where no
other is left the choice is -1 with weight 0. A choice's weight is `scale` times its score, divided by the sum over
the token's choices where weights are renormalised.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
DEVICE = "cuda"
EPS = 1e-5


# ---------------------------------------------------------------- cases


def listed():
    return [
        # one decoded token between two layers, where latency is all: the norm's output goes into an 8-bit product
        {"name": "norm one token", "op": "norm", "rows": 1, "cols": 8192, "type": "bf16", "residual": True},
        # a prompt between two layers
        {"name": "norm prompt", "op": "norm", "rows": 8200, "cols": 5120, "type": "bf16", "residual": True},
        # a training batch: forward, then the gradients of the input and of the norm's weights
        {"name": "norm training", "op": "norm_train", "rows": 16384, "cols": 4096, "type": "bf16", "residual": True},
        # the first norm of a small model in full precision: no residual, sizes that divide nothing
        {"name": "norm training odd", "op": "norm_train", "rows": 1001, "cols": 1111, "type": "fp32", "residual": False},
        # a decoding batch routed with a balancing bias and groups
        {"name": "route decode", "op": "route", "tokens": 32, "experts": 256, "choices": 8, "type": "fp32", "score": "sigmoid", "bias": True, "groups": 8,
         "top_groups": 4, "renormalize": True, "scale": 2.5, "train": False},
        # a training batch of the same router, with the gradient of its logits
        {"name": "route training", "op": "route", "tokens": 16384, "experts": 256, "choices": 8, "type": "fp32", "score": "sigmoid", "bias": True, "groups": 8,
         "top_groups": 4, "renormalize": True, "scale": 2.5, "train": True},
        # a softmax router whose weights stay as they are: the gradient reaches every logit
        {"name": "route softmax", "op": "route", "tokens": 8190, "experts": 60, "choices": 4, "type": "bf16", "score": "softmax", "bias": False, "groups": 1,
         "top_groups": 1, "renormalize": False, "scale": 1.0, "train": True},
        # one decoded token through a square layer
        {"name": "int8 one token", "op": "product", "rows": 1, "depth": 8192, "cols": 8192, "type": "bf16"},
        # a ragged batch through a layer whose sizes divide nothing
        {"name": "int8 odd", "op": "product", "rows": 77, "depth": 2500, "cols": 1111, "type": "fp16"},
        # a long prompt through a large layer
        {"name": "int8 large", "op": "product", "rows": 8192, "depth": 8192, "cols": 8192, "type": "bf16"},
        # a decoding batch, normed into 8 bits before, sent to its experts and through their first product
        {"name": "int8 experts decode", "op": "experts", "tokens": 32, "choices": 4, "experts": 32, "depth": 2048, "cols": 1024, "type": "bf16"},
        # a prompt over experts: unequal groups of some hundred rows
        {"name": "int8 experts prompt", "op": "experts", "tokens": 8192, "choices": 4, "experts": 64, "depth": 4096, "cols": 2048, "type": "bf16"},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over the logarithm; half of them multiples of 8 where that fits."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if n >= 16 and rng.random() < 0.5:
        n -= n % 8
    return max(lo, min(hi, n))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_train", "norm_train", "route", "route", "route", "product", "product", "experts", "experts"])
    kind = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("norm", "norm_train"):
        cols = _spread(rng, 32, 8192)
        return {"op": op, "rows": _spread(rng, 1, min(16384, (1 << 25) // cols)), "cols": cols, "type": kind, "residual": rng.random() < 0.7}
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        experts = groups * rng.choice([2, 4, 8, 15, 32]) if groups > 1 else rng.choice([4, 8, 20, 60, 64, 128, 200, 256])
        top = rng.randint(1, groups)
        choices = min(rng.randint(1, 8), experts // groups * top)
        return {"op": op, "tokens": _spread(rng, 1, 16384), "experts": experts, "choices": choices, "type": kind,
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5, "groups": groups, "top_groups": top,
                "renormalize": choices > 1 and rng.random() < 0.6,  # one choice renormalised has a constant weight: nothing to train
                "scale": rng.choice([1.0, 2.5]), "train": rng.random() < 0.5}
    if op == "product":
        return {"op": op, "rows": _spread(rng, 1, 8192), "depth": _spread(rng, 64, 8192), "cols": _spread(rng, 64, 8192), "type": kind}
    return {"op": op, "tokens": _spread(rng, 1, 8192), "choices": rng.randint(1, 4), "experts": rng.choice([8, 20, 32, 64]), "depth": _spread(rng, 128, 4096),
            "cols": _spread(rng, 128, 2048), "type": kind}


def _padded(cols):
    return -(-cols // 128) * 128


def capacity(case):
    """The most rows one expert takes (a router's capacity, twice the even share): choices beyond it are dropped."""
    return max(8, -(-2 * case["tokens"] * case["choices"] // case["experts"]))


def work(case):
    b = BYTES[case["type"]]
    op = case["op"]
    if op == "norm":  # x, the residual and the weights in; the sum and 8-bit rows out
        n = case["rows"] * case["cols"]
        return {"bytes": n * (b + 1 + (2 * b if case["residual"] else 0)) + 4 * case["rows"] + b * case["cols"], "flops": 6 * n}
    if op == "norm_train":  # x and the residual in, y and the sum out; dy, the sum and its gradient in, dx out
        n = case["rows"] * case["cols"]
        return {"bytes": n * b * (8 if case["residual"] else 5) + 2 * b * case["cols"], "flops": 14 * n}
    if op == "route":
        n, k = case["tokens"] * case["experts"], case["tokens"] * case["choices"]
        return {"bytes": n * b + 8 * k + (n * b * (2 if not case["renormalize"] and case["score"] == "softmax" else 1) + 8 * k if case["train"] else 0), "flops": 8 * n}
    if op == "product":
        m, k, n = case["rows"], case["depth"], case["cols"]
        return {"bytes": m * k * b + n * k + 4 * n + m * n * b, "flops": 2 * m * n * k}
    r = case["tokens"] * case["choices"]
    k, n, e = case["depth"], case["cols"], min(case["experts"], r)
    return {"bytes": case["tokens"] * (k + 4) + 4 * r + e * n * (k + 4) + r * n * b, "flops": 2 * r * n * k}


# ---------------------------------------------------------------- inputs


def _generator(seed):
    return torch.Generator(device=DEVICE).manual_seed(int(seed))


def _activations(g, rows, cols, kind):
    """Normal values with a spread of row and column sizes, as activations have, and a few rows of zeros."""
    x = torch.randn(rows, cols, generator=g, device=DEVICE)
    x *= torch.exp(0.5 * torch.randn(cols, generator=g, device=DEVICE)) * torch.exp(0.5 * torch.randn(rows, 1, generator=g, device=DEVICE))
    x *= torch.rand(rows, 1, generator=g, device=DEVICE) >= 0.01
    if rows == 1:
        x += 0.01 * torch.randn(rows, cols, generator=g, device=DEVICE)
    return x.to(TYPES[kind])


def _gradients(g, rows, cols, kind):
    """Small heavy-tailed values."""
    x = torch.randn(rows, cols, generator=g, device=DEVICE)
    return (1e-3 * x * torch.exp(torch.randn(rows, cols, generator=g, device=DEVICE))).to(TYPES[kind])


def _weights(g, shape, kind):
    return (torch.randn(*shape, generator=g, device=DEVICE) / math.sqrt(shape[-1])).to(TYPES[kind])


def _routing(g, case):
    """Where a router sent the tokens: sorted by expert, what is over an expert's capacity dropped. order, place and
    offsets as the library's exchange has them."""
    t, k, e = case["tokens"], case["choices"], case["experts"]
    scores = torch.randn(t, e, generator=g, device=DEVICE) + 0.5 * torch.randn(e, generator=g, device=DEVICE)
    flat = torch.topk(scores, k, dim=1).indices.reshape(-1)
    by, order = torch.sort(flat, stable=True)
    counts = torch.bincount(flat, minlength=e)
    rank = torch.arange(t * k, device=DEVICE) - (torch.cumsum(counts, 0) - counts)[by]
    kept = order[rank < capacity(case)]
    offsets = torch.cat([counts.new_zeros(1), torch.cumsum(counts.clamp(max=capacity(case)), 0)])
    full = torch.full((t * k,), -1, dtype=torch.long, device=DEVICE)
    full[: kept.numel()] = kept
    place = torch.full((t * k,), -1, dtype=torch.long, device=DEVICE)
    place[kept] = torch.arange(kept.numel(), device=DEVICE)
    return full.int(), place.reshape(t, k).int(), offsets.int()


def prepare(case, seed):
    g = _generator(seed)
    op, kind = case["op"], case["type"]
    s = {"case": dict(case)}
    if op in ("norm", "norm_train"):
        rows, cols = case["rows"], case["cols"]
        s["x"] = _activations(g, rows, cols, kind)
        s["residual"] = _activations(g, rows, cols, kind) if case["residual"] else None
        s["weight"] = (1 + 0.2 * torch.randn(cols, generator=g, device=DEVICE)).to(TYPES[kind])
        if op == "norm_train":
            s["dy"] = _gradients(g, rows, cols, kind)
            s["dh"] = _gradients(g, rows, cols, kind) if case["residual"] else None  # from the layers behind
    elif op == "route":
        t, e = case["tokens"], case["experts"]
        logits = 1.5 * torch.randn(t, e, generator=g, device=DEVICE) + 0.5 * torch.randn(e, generator=g, device=DEVICE)
        hidden = torch.rand(t, e, generator=g, device=DEVICE) < 0.01  # experts a token may not use
        hidden |= torch.rand(t, 1, generator=g, device=DEVICE) < 0.004  # and the rows of a padded batch
        s["logits"] = logits.masked_fill_(hidden, -math.inf).to(TYPES[kind])
        s["bias"] = 0.1 * torch.randn(e, generator=g, device=DEVICE) if case["bias"] else None
        if case["train"]:
            s["dweights"] = 1e-2 * torch.randn(t, case["choices"], generator=g, device=DEVICE)
    elif op == "product":
        s["x"] = _activations(g, case["rows"], case["depth"], kind)
        s["codes"], s["scales"] = _quantised(_weights(g, (case["cols"], case["depth"]), kind))
    else:
        s["order"], s["place"], s["offsets"] = _routing(g, case)
        s["xcodes"], s["xscales"] = _quantised(_activations(g, case["tokens"], case["depth"], kind))
        parts = [_quantised(_weights(g, (case["cols"], case["depth"]), kind)) for _ in range(case["experts"])]
        s["codes"], s["scales"] = (torch.stack(p) for p in zip(*parts))
    return s


# ---------------------------------------------------------------- plain forms, in 32 bits


def _quantised(x):
    """int8 codes [rows, padded] and float32 scales [rows] of x's rows."""
    x = x.float()
    scales = x.abs().amax(-1) / 127
    codes = torch.round(x / torch.where(scales > 0, scales, 1.0)[:, None]).to(torch.int8)
    return torch.nn.functional.pad(codes, (0, -x.shape[-1] % 128)), scales


def _values(codes, scales, cols):
    return codes[..., :cols].float() * scales[..., None]


def _plain_norm(s):
    kind = s["x"].dtype
    h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(kind)
    f, w = h.float(), s["weight"].float()
    r = torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS)
    if s["case"]["op"] == "norm":
        codes, scales = _quantised(f * r * w)
        out = {"values": _values(codes, scales, f.shape[1]).to(torch.bfloat16)}
        return out if s["residual"] is None else {**out, "h": h}
    dy, n = s["dy"].float(), f * r
    part = dy * w
    dx = r * (part - n * (part * n).mean(-1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"y": (n * w).to(kind), "h": h, "dx": dx.to(kind), "dweight": (dy * n).sum(0).to(kind)}


def _plain_route(s):
    c = s["case"]
    logits = s["logits"].double()  # which experts: in 64 bits, values next to each other decide
    open_ = logits > -math.inf
    if c["score"] == "softmax":
        top = logits.amax(1, keepdim=True)
        raw = torch.exp(logits - torch.where(top > -math.inf, top, 0.0))
        total = raw.sum(1, keepdim=True)
        scores = raw / torch.where(total > 0, total, 1.0)
    else:
        scores = 1 / (1 + torch.exp(-logits))
    biased = scores if s["bias"] is None else scores + s["bias"].double()
    key = torch.where(open_, logits if s["bias"] is None else biased, -math.inf)
    if c["groups"] > 1:
        best = torch.where(open_, biased, -math.inf).unflatten(1, (c["groups"], -1)).sort(-1, descending=True).values[..., :2]
        score = torch.where(best > -math.inf, best, 0.0).sum(-1)
        score = torch.where(best[..., 0] > -math.inf, score, -math.inf)
        group = torch.sort(score, dim=1, descending=True, stable=True).indices[:, : c["top_groups"]]
        kept = torch.zeros_like(score, dtype=torch.bool).scatter_(1, group, True)
        key = torch.where(kept[..., None], key.unflatten(1, (c["groups"], -1)), -math.inf).flatten(1)
    best, ids = torch.sort(key, dim=1, descending=True, stable=True)
    best, ids = best[:, : c["choices"]], ids[:, : c["choices"]]
    here = best > -math.inf
    f = scores.float()
    mine = torch.where(here, f.gather(1, ids), 0.0)
    total = mine.sum(1, keepdim=True)
    total = torch.where(total > 0, total, 1.0) if c["renormalize"] else torch.ones_like(total)
    weights = c["scale"] * mine / total
    out = {"ids": torch.where(here, ids, -1).int(), "weights": weights}
    if c["train"]:
        d = torch.where(here, s["dweights"], 0.0) * c["scale"]
        if c["renormalize"]:
            d = (d - (d * mine / total).sum(1, keepdim=True)) / total
        ds = torch.zeros_like(f).scatter_add_(1, ids, torch.where(here, d, 0.0))
        dl = f * (1 - f) * ds if c["score"] == "sigmoid" else f * (ds - (ds * f).sum(1, keepdim=True))
        out["dlogits"] = dl.to(TYPES[c["type"]])
    return out


def _plain_experts(s):
    """By expert with as many rows for each as its capacity; the rows of no expert are zeros."""
    c = s["case"]
    e, cap, depth = c["experts"], capacity(c), c["depth"]
    order, offsets = s["order"].long(), s["offsets"].long()
    row = torch.arange(order.numel(), device=order.device)
    expert = torch.searchsorted(offsets[1:], row, right=True)
    valid = order >= 0
    at = torch.where(valid, expert * cap + (row - offsets[expert.clamp(max=e - 1)]), e * cap)
    x = _values(s["xcodes"], s["xscales"], depth)
    padded = x.new_zeros(e * cap + 1, depth)
    padded[at] = torch.where(valid[:, None], x[order.clamp(min=0) // c["choices"]], 0.0)
    w = _values(s["codes"], s["scales"], depth)
    y = torch.bmm(padded[:-1].reshape(e, cap, depth), w.transpose(1, 2).contiguous()).flatten(0, 1)
    return {"y": torch.cat([y, y.new_zeros(1, c["cols"])])[at].to(TYPES[c["type"]])}


def _plain(s):
    op = s["case"]["op"]
    if op in ("norm", "norm_train"):
        return _plain_norm(s)
    if op == "route":
        return _plain_route(s)
    if op == "product":
        x = _values(*_quantised(s["x"]), s["case"]["depth"])
        return {"y": torch.mm(x, _values(s["codes"], s["scales"], s["case"]["depth"]).t()).to(s["x"].dtype)}
    return _plain_experts(s)


# ---------------------------------------------------------------- the library


def _library(s):
    import error_bounded_lossy_amd as ec

    c = s["case"]
    op = c["op"]
    if op == "norm":
        q = ec.rms_norm_i8(s["x"], s["weight"], EPS, residual=s["residual"])
        if s["residual"] is None:
            return {"values": ec.i8_dequantize(q, torch.bfloat16)}
        return {"values": ec.i8_dequantize(q[0], torch.bfloat16), "h": q[1]}
    if op == "norm_train":
        y, saved = ec.rms_norm_forward(s["x"], s["weight"], EPS, residual=s["residual"])
        dx, dweight = ec.rms_norm_backward(s["dy"], saved, dh=s["dh"])
        return {"y": y, "h": saved.h, "dx": dx, "dweight": dweight}
    if op == "route":
        how = {"score": c["score"], "renormalize": c["renormalize"], "scale": c["scale"]}
        ids, weights = ec.expert_route(s["logits"], c["choices"], bias=s["bias"], groups=c["groups"], top_groups=c["top_groups"], **how)
        out = {"ids": ids, "weights": weights}
        if c["train"]:
            out["dlogits"] = ec.expert_route_backward(s["dweights"], s["logits"], ids, **how)
        return out
    w = ec.I8Tensor(s["codes"], s["scales"], c["depth"])
    if op == "product":
        return {"y": ec.i8_linear(s["x"], w)}
    r = ec.Routing(s["order"], s["place"], s["offsets"], c["tokens"], c["choices"], c["experts"])
    xs = ec.expert_dispatch_i8(ec.I8Tensor(s["xcodes"], s["xscales"], c["depth"]), r)
    return {"y": ec.i8_experts_product(xs, w, r.offsets, TYPES[c["type"]])}


def run(state):
    return _library(state) if own else _plain(state)


# ---------------------------------------------------------------- the definitions, in 64 bits


def _whole(y, s):
    """y / s to whole numbers, ties to even, as the values they stand for."""
    q = y / torch.where(s > 0, s, 1.0)
    low = torch.floor(q)
    up = (q - low > 0.5) | ((q - low == 0.5) & (low % 2 == 1))
    return (low + up) * s


def _exact_norm(s):
    train = s["case"]["op"] == "norm_train"
    x = s["x"]
    h = x if s["residual"] is None else (x.double() + s["residual"].double()).to(x.dtype)  # the sum is kept in x's type
    f = h.double().requires_grad_(train)
    w = s["weight"].double().requires_grad_(train)
    y = f * (f.square().mean(1, keepdim=True) + EPS).pow(-0.5) * w
    if not train:
        out = {"values": _whole(y, y.abs().amax(1, keepdim=True) / 127)}
        return out if s["residual"] is None else {**out, "h": h.double()}
    dx, dw = torch.autograd.grad(y, (f, w), s["dy"].double())
    if s["dh"] is not None:
        dx = dx + s["dh"].double()
    return {"y": y.detach(), "h": h.double(), "dx": dx, "dweight": dw}


def _exact_route(s):
    c = s["case"]
    logits = s["logits"].double().requires_grad_(c["train"])
    closed = logits.detach() == -math.inf
    if c["score"] == "softmax":
        e = torch.exp(logits - logits.detach().amax(1, keepdim=True).clamp(min=-1e30))
        total = e.sum(1, keepdim=True)
        scores = e / torch.where(total > 0, total, 1.0)
    else:
        scores = torch.sigmoid(logits)
    flat = scores.detach()
    by = flat if s["bias"] is None else flat + s["bias"].double()
    by = by.masked_fill(closed, -math.inf)
    key = logits.detach().clone() if s["bias"] is None else by.clone()

    def first_largest(v):
        """The largest of each row and the first place that has it."""
        top = v.amax(1, keepdim=True)
        at = torch.arange(v.shape[1], device=v.device).expand_as(v)
        return top, torch.where(v == top, at, v.shape[1]).amin(1, keepdim=True)

    if c["groups"] > 1:
        n = c["experts"] // c["groups"]
        cols = []
        for g in range(c["groups"]):
            part = by[:, g * n:(g + 1) * n].clone()
            one, at = first_largest(part)
            part.scatter_(1, at, -math.inf)
            two = part.amax(1, keepdim=True)
            cols.append(one + torch.where(two > -math.inf, two, 0.0))
        sums = torch.cat(cols, 1)
        closed_group = torch.ones_like(sums, dtype=torch.bool)
        for _ in range(c["top_groups"]):
            _, at = first_largest(sums)
            closed_group.scatter_(1, at, False)
            sums.scatter_(1, at, -math.inf)
        key.masked_fill_(closed_group.repeat_interleave(n, 1), -math.inf)
    picked, ok = [], []
    for _ in range(c["choices"]):
        top, at = first_largest(key)
        picked.append(at)
        ok.append(top > -math.inf)
        key.scatter_(1, at, -math.inf)
    ids, ok = torch.cat(picked, 1), torch.cat(ok, 1)
    mine = scores.gather(1, ids) * ok
    if c["renormalize"]:
        total = mine.sum(1, keepdim=True)
        mine = mine / torch.where(total > 0, total, 1.0)
    weights = c["scale"] * mine
    out = {"ids": None, "weights": weights.detach()}
    if c["train"]:
        out["dlogits"], = torch.autograd.grad(weights, logits, s["dweights"].double())
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm_train"):
        return _exact_norm(s)
    if op == "route":
        return _exact_route(s)
    depth = case["depth"]
    w = s["codes"][..., :depth].double() * s["scales"].double()[..., None]
    if op == "product":
        x = s["x"].double()
        x = _whole(x, (x.abs().amax(1, keepdim=True) / 127).float().double())  # a scale is held in float32
        return {"y": torch.mm(x, w.t())}
    x = s["xcodes"][:, :depth].double() * s["xscales"].double()[:, None]
    at, order = s["offsets"].tolist(), s["order"].long()
    y = torch.zeros(order.numel(), case["cols"], dtype=torch.float64, device=DEVICE)
    for e, (a, b) in enumerate(zip(at, at[1:])):
        if b > a:
            y[a:b] = torch.mm(x[order[a:b] // case["choices"]], w[e].t())
    return {"y": y}
