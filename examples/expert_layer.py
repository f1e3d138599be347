"""An expert layer on the 4-bit operators: a decoding step and training steps.

    python examples/expert_layer.py [--tokens 512] [--width 512] [--hidden 768] [--experts 8] [--steps 10] [--routed]

Each token goes to `choices` experts, each a 4-bit linear layer up, a ReLU and a
4-bit linear layer down, and comes back as their weighted sum.  The router is
fixed; the experts' weights learn to match a teacher of the same form.  With
--routed, the layer begins with the residual's addition and a norm, the norm's
weights and the router learn too, and it is served in 8 bits in the end.
With several GPUs, the all-to-all goes between the exchange and the experts.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import error_bounded_lossy_amd as ec  # noqa: E402


def route(x, router, choices):
    """The best experts of each token and their weights."""
    top, ids = torch.topk(x.float() @ router, choices, dim=1)
    return ids.to(torch.int32), torch.softmax(top, dim=1)


def decode(x, up, down, ids, weights):
    """One step of serving with weights in the 4-bit form: tokens are quantized once, sent in
    4 bits, and multiplied as they arrive."""
    r = ec.expert_sort(ids, up.shape[0])
    h = ec.mx_experts_product(ec.expert_dispatch_mx(x, r), up, r.offsets, x.dtype)
    return ec.expert_combine(ec.mx_experts_linear(torch.relu(h), down, r.offsets), r, weights)


def train_step(x, up, down, ids, weights, gradient):
    """The layer's output and, with gradient(y) the loss's gradient there, those of x, both weights
    and the router's weights."""
    r = ec.expert_sort(ids, up.shape[0])
    h, saved_up = ec.mx_experts_forward(ec.expert_dispatch(x, r), up, r.offsets)
    ys, saved_down = ec.mx_experts_forward(torch.relu(h), down, r.offsets)
    y = ec.expert_combine(ys, r, weights)

    dys, dweights = ec.expert_combine_backward(gradient(y), ys, r, weights)
    dh, ddown = ec.mx_experts_backward(dys, saved_down)
    dxs, dup = ec.mx_experts_backward(dh * (h > 0), saved_up)
    return y, {"x": ec.expert_dispatch_backward(dxs, r), "up": dup, "down": ddown, "weights": dweights}


def routed_step(x, residual, norm, router, up, down, choices, gradient):
    """train_step behind the residual's addition, the norm and a router that is trained: the layer's
    output h + experts(norm(h)), and the gradients of x (and the residual alike) and all weights.
    gradient(y) is the loss's gradient at the output."""
    n, saved = ec.rms_norm_forward(x, norm, residual=residual)
    logits = n.float() @ router
    ids, weights = ec.expert_route(logits, choices)
    dy = []

    def at_experts(y):
        dy.append(gradient(saved.h + y))
        return dy[0]

    y, grads = train_step(n, up, down, ids, weights, at_experts)
    dlogits = ec.expert_route_backward(grads["weights"], logits, ids)
    dn = grads["x"].float() + dlogits @ router.t()
    dx, dnorm = ec.rms_norm_backward(dn.to(n.dtype), saved, dh=dy[0])
    return saved.h + y, {"x": dx, "norm": dnorm, "router": n.float().t() @ dlogits, "up": grads["up"], "down": grads["down"]}


def serve(x, residual, norm, router, up, down, choices):
    """The same layer served in 8 bits: router [experts, width], up [experts, hidden, width] and down
    [experts, width, hidden] in the 8-bit form.  What the norm writes is what the router and the
    experts read."""
    q, h = ec.rms_norm_i8(x, norm, residual=residual)
    ids, weights = ec.expert_route(ec.i8_product(q, router, torch.float32), choices)
    r = ec.expert_sort(ids, up.lead[0])
    a = ec.i8_experts_product(ec.expert_dispatch_i8(q, r), up, r.offsets, x.dtype)
    return h + ec.expert_combine(ec.i8_experts_linear(torch.relu(a), down, r.offsets), r, weights)


def main():
    p = argparse.ArgumentParser()
    for name, default in (("tokens", 512), ("width", 512), ("hidden", 768), ("experts", 8), ("choices", 2), ("steps", 10)):
        p.add_argument(f"--{name}", type=int, default=default)
    p.add_argument("--routed", action="store_true")
    a = p.parse_args()
    g = torch.Generator(device="cuda").manual_seed(0)

    def weights_of(rows, cols):
        return torch.randn(a.experts, rows, cols, generator=g, device="cuda") / cols ** 0.5

    x = torch.randn(a.tokens, a.width, generator=g, device="cuda").bfloat16()
    router = torch.randn(a.width, a.experts, generator=g, device="cuda") / a.width ** 0.5
    ids, weights = route(x, router, a.choices)
    teacher = [ec.mx_quantize(weights_of(a.hidden, a.width).bfloat16()), ec.mx_quantize(weights_of(a.width, a.hidden).bfloat16())]
    target = decode(x, *teacher, ids, weights).float()

    up, down = weights_of(a.hidden, a.width), weights_of(a.width, a.hidden)
    if a.routed:
        routed(a, g, x, router, up, down, target)
        return
    for step in range(a.steps):
        y, grads = train_step(x, up.bfloat16(), down.bfloat16(), ids, weights,
                              lambda y: (y.float() - target).bfloat16())
        for w, d in ((up, grads["up"]), (down, grads["down"])):
            w -= 0.03 / (a.tokens * a.choices / a.experts) * d.float()
        print(f"step {step}: mean squared error {(y.float() - target).square().mean().item():.4f}")
    y = decode(x[:1], ec.mx_quantize(up.bfloat16()), ec.mx_quantize(down.bfloat16()), ids[:1], weights[:1])
    print(f"one token decoded: {(y.float() - target[:1]).square().mean().item():.4f}")


def routed(a, g, x, router, up, down, target):
    residual = torch.randn(a.tokens, a.width, generator=g, device="cuda").bfloat16()
    norm, target = torch.ones(a.width, device="cuda"), target + (x + residual).float()
    error = lambda y: (y.float() - target).square().mean().item()  # noqa: E731
    for step in range(a.steps):
        y, grads = routed_step(x, residual, norm.bfloat16(), router, up.bfloat16(), down.bfloat16(), a.choices,
                               lambda y: (y.float() - target).bfloat16())
        rate = 0.03 / (a.tokens * a.choices / a.experts)
        for w, name in ((up, "up"), (down, "down"), (router, "router"), (norm, "norm")):
            w -= rate * grads[name].float()
        print(f"step {step}: mean squared error {error(y):.4f}")
    served = [ec.i8_quantize(w.bfloat16()) for w in (router.t().contiguous(), up, down)]
    print(f"served in 8 bits: {error(serve(x, residual, norm.bfloat16(), *served, a.choices)):.4f}")


if __name__ == "__main__":
    main()
