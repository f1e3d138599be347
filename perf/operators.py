"""Measured cases of the 4-bit and expert operators: the microscaled 4-bit format (quantisation and
product), the product of rows grouped by expert, and the exchange of tokens sorted by expert.

`listed()` gives the cases, `draw(rng)` further ones of the same ranges, `prepare` the inputs, `run` one
pass (`own` false: plain torch in 32 bits, `own` true: the library's kernels), `exact` the same results
in 64 bits from the definitions, `work` what one pass has to move and compute.

The format: 32 consecutive elements share a scale 2^(s - 127) held as the byte s; an element is a sign
and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6, held in 4 bits (sign in the top bit), the even element of a pair
in the low half of its byte. With m the largest magnitude of the block, the scale's exponent is
floor(log2 m) - 2 and at least -127; elements are rounded to the nearest value, ties to the even code,
and saturate at 6. Rows are padded with zeros to a multiple of 128 elements.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DEVICE = "cuda"
VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- cases


def listed():
    return [
        # one token's activations before a product, where latency is all
        {"name": "quantise one token", "op": "quantise", "rows": 1, "cols": 8192, "type": "bf16", "both": False},
        # a batch of embedding lookups, 26 tables of 8192 rows: the batch this repository's benchmark compresses
        {"name": "quantise lookups", "op": "quantise", "rows": 212992, "cols": 128, "type": "fp32", "both": False},
        # activations kept for a backward pass: blocks along the features and along the tokens
        {"name": "quantise both ways", "op": "quantise", "rows": 8200, "cols": 5120, "type": "bf16", "both": True},
        # one decoded token through a square layer
        {"name": "product one token", "op": "product", "rows": 1, "depth": 8192, "cols": 8192, "type": "bf16"},
        # a ragged batch through a layer whose sizes divide nothing
        {"name": "product odd", "op": "product", "rows": 77, "depth": 2500, "cols": 1111, "type": "fp16"},
        # a long prompt through a large layer
        {"name": "product large", "op": "product", "rows": 8192, "depth": 8192, "cols": 8192, "type": "bf16"},
        # a training step of one layer: output and both gradients
        {"name": "product training", "op": "train", "rows": 4100, "depth": 4096, "cols": 4096, "type": "bf16"},
        # a decoding batch over experts: a few rows for each
        {"name": "experts decode", "op": "experts", "tokens": 32, "choices": 4, "experts": 32, "depth": 2048, "cols": 1024, "type": "bf16"},
        # a prompt over experts: unequal groups of some hundred rows
        {"name": "experts prompt", "op": "experts", "tokens": 8192, "choices": 4, "experts": 64, "depth": 4096, "cols": 2048, "type": "bf16"},
        # a training step of an expert layer's product: output and both gradients
        {"name": "experts training", "op": "experts_train", "tokens": 8192, "choices": 2, "experts": 16, "depth": 2048, "cols": 2048, "type": "bf16"},
        # a decoding batch sent to its experts in 4 bits and brought back
        {"name": "exchange decode", "op": "exchange", "tokens": 64, "choices": 4, "experts": 64, "cols": 4096, "type": "bf16", "payload": "mx4", "train": False},
        # a training batch sent to its experts and brought back, with the gradients of both ways
        {"name": "exchange training", "op": "exchange", "tokens": 16384, "choices": 4, "experts": 128, "cols": 4096, "type": "bf16", "payload": "same", "train": True},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over the logarithm; half of them multiples of 8 where that fits."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if n >= 16 and rng.random() < 0.5:
        n -= n % 8
    return max(lo, min(hi, n))


def draw(rng):
    op = rng.choice(["quantise", "product", "product", "train", "experts", "experts", "experts_train", "exchange", "exchange"])
    kind = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "quantise":
        cols = _spread(rng, 32, 8192)
        return {"op": op, "rows": _spread(rng, 1, min(65536, (1 << 25) // cols)), "cols": cols, "type": kind, "both": rng.random() < 0.5}
    if op == "product":
        return {"op": op, "rows": _spread(rng, 1, 8192), "depth": _spread(rng, 64, 8192), "cols": _spread(rng, 64, 8192), "type": kind}
    if op == "train":
        return {"op": op, "rows": _spread(rng, 32, 4100), "depth": _spread(rng, 64, 4096), "cols": _spread(rng, 64, 4096), "type": kind}
    if op in ("experts", "experts_train"):
        small = op == "experts_train"
        return {"op": op, "tokens": _spread(rng, 1, 8192), "choices": rng.randint(1, 2 if small else 4), "experts": rng.choice([8, 12, 16] if small else [8, 20, 32, 64]),
                "depth": _spread(rng, 128, 2048 if small else 4096), "cols": _spread(rng, 128, 2048), "type": kind}
    return {"op": op, "tokens": _spread(rng, 1, 16384 if kind != "fp32" else 8192), "choices": rng.randint(1, 4), "experts": rng.choice([8, 24, 64, 128]), "cols": _spread(rng, 64, 4096),
            "type": kind, "payload": rng.choice(["same", "mx4"]), "train": rng.random() < 0.5}


def capacity(case):
    """The most rows one expert takes (a router's capacity, twice the even share): choices beyond it are dropped."""
    return max(8, -(-2 * case["tokens"] * case["choices"] // case["experts"]))


def work(case):
    b = {"bf16": 2, "fp16": 2, "fp32": 4}[case["type"]]
    q = 0.5 + 1 / 32  # bytes of an element in the 4-bit form
    op = case["op"]
    if op == "quantise":  # read once; the values come back as the same type
        n = case["rows"] * case["cols"]
        return {"bytes": n * b * (3 if case["both"] else 2), "flops": 4 * n}
    if op == "product":
        m, k, n = case["rows"], case["depth"], case["cols"]
        return {"bytes": m * k * b + n * k * q + m * n * b, "flops": 2 * m * n * k}
    if op == "train":
        m, k, n = case["rows"], case["depth"], case["cols"]
        return {"bytes": 2 * b * (m * k + n * k + m * n), "flops": 6 * m * n * k}
    r = case["tokens"] * case["choices"]
    if op == "experts":
        k, n, e = case["depth"], case["cols"], min(case["experts"], r)
        return {"bytes": r * k * b + e * n * k * q + r * n * b, "flops": 2 * r * n * k}
    if op == "experts_train":
        k, n, e = case["depth"], case["cols"], case["experts"]
        return {"bytes": 2 * b * (r * k + e * n * k + r * n), "flops": 6 * r * n * k}
    t, d = case["tokens"], case["cols"]
    ids = r * (4 + 4 + 4) + 4 * case["experts"]
    forward = ids + t * d * b + r * d * b + r * d * b + t * d * b + 4 * r  # x in, sorted rows out; rows in, y out
    backward = t * d * b + r * d * b + r * d * b + 4 * r + r * d * b + t * d * b if case["train"] else 0  # dy, ys in, dys, dw out; dxs in, dx out
    return {"bytes": forward + backward, "flops": 2 * r * d * (4 if case["train"] else 1)}


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
    """Choices of every token (distinct, some experts liked better than others) and their weights. What is over an
    expert's capacity is -1: dropped."""
    t, k, e = case["tokens"], case["choices"], case["experts"]
    scores = torch.randn(t, e, generator=g, device=DEVICE) + 0.5 * torch.randn(e, generator=g, device=DEVICE)
    top, ids = torch.topk(scores, k, dim=1)
    weights = torch.softmax(top, dim=1)
    flat = ids.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    counts = torch.bincount(flat, minlength=e)
    first = torch.cumsum(counts, 0) - counts
    rank = torch.empty_like(flat)
    rank[order] = torch.arange(t * k, device=DEVICE) - first[flat[order]]
    flat = torch.where(rank < capacity(case), flat, torch.full_like(flat, -1))
    return flat.reshape(t, k).to(torch.int32), weights


def _offsets(ids, experts):
    flat = ids.reshape(-1).long()
    counts = torch.bincount(flat[flat >= 0], minlength=experts)
    return torch.cat([counts.new_zeros(1), torch.cumsum(counts, 0)]).to(torch.int32)


def prepare(case, seed):
    g = _generator(seed)
    op, kind = case["op"], case["type"]
    s = {"case": dict(case)}
    if op == "quantise":
        s["x"] = _activations(g, case["rows"], case["cols"], kind)
    elif op == "product":
        s["x"] = _activations(g, case["rows"], case["depth"], kind)
        s["codes"], s["scales"] = _pack(*_quantised(_weights(g, (case["cols"], case["depth"]), kind)))
    elif op == "train":
        s["x"] = _activations(g, case["rows"], case["depth"], kind)
        s["w"] = _weights(g, (case["cols"], case["depth"]), kind)
        s["dy"] = _gradients(g, case["rows"], case["cols"], kind)
    elif op in ("experts", "experts_train"):
        ids, _ = _routing(g, case)
        s["offsets"] = _offsets(ids, case["experts"])
        s["x"] = _activations(g, ids.numel(), case["depth"], kind)
        shape = (case["experts"], case["cols"], case["depth"])
        if op == "experts":
            parts = [_pack(*_quantised(_weights(g, shape[1:], kind))) for _ in range(case["experts"])]
            s["codes"], s["scales"] = (torch.stack(p) for p in zip(*parts))
        else:
            s["w"] = _weights(g, shape, kind)
            s["dy"] = _gradients(g, ids.numel(), case["cols"], kind)
    else:
        s["ids"], s["weights"] = _routing(g, case)
        s["x"] = _activations(g, case["tokens"], case["cols"], kind)
        s["ys"] = _activations(g, s["ids"].numel(), case["cols"], kind)  # the experts' answers
        if case["train"]:
            s["dy"] = _gradients(g, case["tokens"], case["cols"], kind)
            s["dxs"] = _gradients(g, s["ids"].numel(), case["cols"], kind)
    return s


# ---------------------------------------------------------------- plain forms, in 32 bits


def _quantised(x):
    """Codes [.., blocks, 32] and scale bytes [.., blocks] of x along its last dimension, padded to 128 elements."""
    x = x.float()
    x = torch.nn.functional.pad(x, (0, -x.shape[-1] % 128))
    x = x.unflatten(-1, (-1, 32))
    exponent = (x.abs().amax(-1).view(torch.int32) >> 23) - 2  # of the scale, biased
    scale = exponent.clamp(min=0)
    inverse = ((254 - scale) << 23).view(torch.float32)  # 2^(127 - scale): always a normal number
    a = (x * inverse[..., None]).abs()
    code = torch.zeros_like(x, dtype=torch.uint8)
    code += a > 0.25
    code += a >= 0.75
    code += a > 1.25
    code += a >= 1.75
    code += a > 2.5
    code += a >= 3.5
    code += a > 5.0
    code += torch.signbit(x).to(torch.uint8) * 8
    return code, scale.to(torch.uint8)


def _pack(code, scale):
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale


def _values(code, scale):
    """What codes [.., blocks, 32] and scale bytes stand for, as one row."""
    table = torch.tensor(VALUES + tuple(-v for v in VALUES), device=code.device)
    size = torch.where(scale > 0, scale.int() << 23, torch.full_like(scale, 1, dtype=torch.int32) << 22).view(torch.float32)
    return (table[code.int()] * size[..., None]).flatten(-2)


def _unpack(codes, scales):
    code = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    return _values(code.unflatten(-1, (-1, 32)), scales)


def _near(x):
    """x rounded to the 4-bit form along its last dimension, in float32."""
    return _values(*_quantised(x))[..., : x.shape[-1]]


def _grouped(x, offsets, case):
    """Sorted rows as [experts, capacity, cols], and where each row of x is in it (past the end: nowhere)."""
    e, cap = case["experts"], capacity(case)
    row = torch.arange(x.shape[0], device=x.device, dtype=torch.int32)
    expert = torch.searchsorted(offsets[1:], row, right=True)
    valid = expert < e
    at = torch.where(valid, expert * cap + (row - offsets[expert.clamp(max=e - 1)]), e * cap)
    padded = x.new_zeros(e * cap + 1, x.shape[1])
    padded[at] = torch.where(valid[:, None], x, torch.zeros_like(x))
    return padded[:-1].reshape(e, cap, -1), at


def _ungrouped(y, at):
    return torch.cat([y.flatten(0, 1), y.new_zeros(1, y.shape[2])])[at]


def _plain(s):
    case = s["case"]
    op, kind = case["op"], TYPES[case["type"]]
    if op == "quantise":
        x = s["x"]
        y = _near(x).to(kind)
        return {"rows": y, "columns": _near(x.t().contiguous()).to(kind)} if case["both"] else {"rows": y}
    if op == "product":
        w = _unpack(s["codes"], s["scales"])[:, : case["depth"]]
        return {"y": torch.mm(_near(s["x"]), w.t()).to(kind)}
    if op == "train":
        x, w, dy = s["x"].float(), s["w"].float(), s["dy"].float()
        y = torch.mm(_near(x), _near(w).t())
        dx = torch.mm(_near(dy), _near(w.t().contiguous()).t())
        dw = torch.mm(_near(dy.t().contiguous()), _near(x.t().contiguous()).t())
        return {"y": y.to(kind), "dx": dx.to(kind), "dw": dw.to(kind)}
    if op == "experts":
        x, at = _grouped(_near(s["x"]), s["offsets"], case)
        w = _unpack(s["codes"], s["scales"])[..., : case["depth"]]
        return {"y": _ungrouped(torch.bmm(x, w.transpose(1, 2).contiguous()), at).to(kind)}
    if op == "experts_train":
        w = s["w"].float()
        x, at = _grouped(s["x"].float(), s["offsets"], case)
        dy, _ = _grouped(s["dy"].float(), s["offsets"], case)
        wt, xt, dyt = (v.transpose(1, 2).contiguous() for v in (w, x, dy))
        y = torch.bmm(_near(x), _near(w).transpose(1, 2).contiguous())
        dx = torch.bmm(_near(dy), _near(wt).transpose(1, 2).contiguous())
        dw = torch.bmm(_near(dyt), _near(xt).transpose(1, 2).contiguous())
        return {"y": _ungrouped(y, at).to(kind), "dx": _ungrouped(dx, at).to(kind), "dw": dw.to(kind)}
    ids, choices, experts = s["ids"], case["choices"], case["experts"]
    flat = torch.where(ids >= 0, ids, experts).reshape(-1)
    by, order = torch.sort(flat, stable=True)
    offsets = torch.searchsorted(by, torch.arange(experts + 1, device=ids.device, dtype=torch.int32))
    row = torch.arange(flat.numel(), device=ids.device)
    valid = row < offsets[-1]
    place = torch.empty_like(order)
    place[order] = torch.where(valid, row, -1)
    place = place.reshape(ids.shape)
    here = (place >= 0)[..., None]
    x = s["x"].float() if case["payload"] == "same" else _near(s["x"])
    xs = torch.where(valid[:, None], x[order // choices], 0.0)
    weights = s["weights"][..., None]
    answers = torch.where(here, s["ys"].float()[place.clamp(min=0)], 0.0)
    out = {"order": torch.where(valid, order, -1).int(), "place": place.int(), "offsets": offsets.int(), "xs": xs.to(kind), "y": (answers * weights).sum(1).to(kind)}
    if case["train"]:
        dy = s["dy"].float()
        part = torch.where(valid[:, None], dy[order // choices] * weights.reshape(-1)[order, None], 0.0)
        out["dys"] = part.to(kind)
        out["dweights"] = torch.where(here[..., 0], (answers * dy[:, None]).sum(-1), 0.0)
        out["dx"] = torch.where(here, s["dxs"].float()[place.clamp(min=0)], 0.0).sum(1).to(kind)
    return out


# ---------------------------------------------------------------- the library


def _library(s):
    import error_bounded_lossy_amd as ec

    case = s["case"]
    op = case["op"]
    if op == "quantise":
        x = s["x"]
        if case["both"]:
            rows, columns = ec.mx_quantize_both(x)
            return {"rows": ec.mx_dequantize(rows, x.dtype), "columns": ec.mx_dequantize(columns, x.dtype)}
        return {"rows": ec.mx_dequantize(ec.mx_quantize(x), x.dtype)}
    if op == "product":
        return {"y": ec.mx_linear(s["x"], ec.MXTensor(s["codes"], s["scales"], case["depth"]))}
    if op == "train":
        y, saved = ec.mx_linear_forward(s["x"], s["w"])
        dx, dw = ec.mx_linear_backward(s["dy"], saved)
        return {"y": y, "dx": dx, "dw": dw}
    if op == "experts":
        return {"y": ec.mx_experts_linear(s["x"], ec.MXTensor(s["codes"], s["scales"], case["depth"]), s["offsets"])}
    if op == "experts_train":
        y, saved = ec.mx_experts_forward(s["x"], s["w"], s["offsets"])
        dx, dw = ec.mx_experts_backward(s["dy"], saved)
        return {"y": y, "dx": dx, "dw": dw}
    routing = ec.expert_sort(s["ids"], case["experts"])
    if case["payload"] == "same":
        xs = ec.expert_dispatch(s["x"], routing)
    else:
        xs = ec.mx_dequantize(ec.expert_dispatch_mx(s["x"], routing), s["x"].dtype)
    out = {"order": routing.order, "place": routing.place, "offsets": routing.offsets, "xs": xs, "y": ec.expert_combine(s["ys"], routing, s["weights"])}
    if case["train"]:
        out["dys"], out["dweights"] = ec.expert_combine_backward(s["dy"], s["ys"], routing, s["weights"])
        out["dx"] = ec.expert_dispatch_backward(s["dxs"], routing)
    return out


def run(state):
    return _library(state) if own else _plain(state)


# ---------------------------------------------------------------- the definitions, in 64 bits


def _two_to(e):
    """2^e for whole e of a normal number, in 64 bits (a library's power need not be exact, and ties are)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_near(x):
    """The last dimension in blocks of 32: the scale from the exponent of the largest magnitude, then the nearest
    element by the spacing of its binade."""
    x = x.double()
    n = x.shape[-1]
    x = torch.nn.functional.pad(x, (0, -n % 32)).unflatten(-1, (-1, 32))
    _, e = torch.frexp(x.abs().amax(-1, keepdim=True))  # m = f 2^e with f in [0.5, 1)
    e = torch.where(x.abs().amax(-1, keepdim=True) == 0, torch.full_like(e, -127), e - 3).clamp(min=-127)
    v = x * _two_to(-e)
    step = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0)).to(v.dtype)
    v = (torch.round(v / step) * step).clamp(-6, 6)
    return (v * _two_to(e)).flatten(-2)[..., :n]


def _exact_weights(s):
    """The stored 4-bit weights: (2 + f) halves of a power of two, or f halves in the lowest binade."""
    def part(c):
        c = c.long()
        f, b = (c & 1).double(), (c >> 1) & 3
        v = torch.where(b == 0, f / 2, (1 + f / 2) * _two_to(b - 1))
        return torch.where(c >= 8, -v, v)

    codes = torch.stack([part(s["codes"] & 15), part(s["codes"] >> 4)], -1).flatten(-2)
    size = _two_to(s["scales"].long() - 127)
    return (codes.unflatten(-1, (-1, 32)) * size[..., None]).flatten(-2)[..., : s["case"]["depth"]]


def _mm(a, b):
    """a bᵀ."""
    return torch.matmul(a, b.transpose(-1, -2).contiguous())


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantise":
        y = _exact_near(s["x"])
        return {"rows": y, "columns": _exact_near(s["x"].t().contiguous())} if case["both"] else {"rows": y}
    if op == "product":
        return {"y": _mm(_exact_near(s["x"]), _exact_weights(s))}
    if op == "train":
        x, w, dy = s["x"], s["w"], s["dy"]
        xt, wt, dyt = (v.t().contiguous() for v in (x, w, dy))
        return {"y": _mm(_exact_near(x), _exact_near(w)), "dx": _mm(_exact_near(dy), _exact_near(wt)), "dw": _mm(_exact_near(dyt), _exact_near(xt))}
    if op in ("experts", "experts_train"):
        at = s["offsets"].tolist()
        y = torch.zeros(s["x"].shape[0], case["cols"], dtype=torch.float64, device=DEVICE)
        if op == "experts":
            w = _exact_weights(s)
            for e, (a, b) in enumerate(zip(at, at[1:])):
                y[a:b] = _mm(_exact_near(s["x"][a:b]), w[e])
            return {"y": y}
        dx = torch.zeros(s["x"].shape, dtype=torch.float64, device=DEVICE)
        dw = torch.zeros(s["w"].shape, dtype=torch.float64, device=DEVICE)
        for e, (a, b) in enumerate(zip(at, at[1:])):
            x, w, dy = s["x"][a:b], s["w"][e], s["dy"][a:b]
            y[a:b] = _mm(_exact_near(x), _exact_near(w))
            dx[a:b] = _mm(_exact_near(dy), _exact_near(w.t().contiguous()))
            if b > a:
                dw[e] = _mm(_exact_near(dy.t().contiguous()), _exact_near(x.t().contiguous()))
        return {"y": y, "dx": dx, "dw": dw}
    ids = s["ids"].reshape(-1).long().cpu()
    order = torch.tensor(sorted((i for i in range(len(ids)) if ids[i] >= 0), key=lambda i: (int(ids[i]), i)), dtype=torch.long)
    counts = torch.bincount(ids[ids >= 0], minlength=case["experts"])
    total, rows = len(order), len(ids)
    full = torch.full((rows,), -1, dtype=torch.long)
    full[:total] = order
    place = torch.full((rows,), -1, dtype=torch.long)
    place[order] = torch.arange(total)
    order = order.to(DEVICE)
    token, w = order // case["choices"], s["weights"].double().reshape(-1)[order, None]
    x = s["x"].double() if case["payload"] == "same" else _exact_near(s["x"])
    shape = (rows, case["cols"])
    xs = torch.zeros(shape, dtype=torch.float64, device=DEVICE)
    xs[:total] = x[token]
    ys = s["ys"][:total].double()
    y = torch.zeros_like(x).index_add_(0, token, ys * w)
    out = {"order": full.int(), "place": place.reshape(s["ids"].shape).int(), "offsets": torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int(), "xs": xs, "y": y}
    if case["train"]:
        dys = torch.zeros(shape, dtype=torch.float64, device=DEVICE)
        dys[:total] = s["dy"].double()[token] * w
        dweights = torch.zeros(rows, dtype=torch.float64, device=DEVICE)
        dweights[order] = (s["dy"].double()[token] * ys).sum(-1)
        dx = torch.zeros_like(x).index_add_(0, token, s["dxs"][:total].double())
        out |= {"dys": dys, "dweights": dweights.reshape(s["ids"].shape), "dx": dx}
    return out
