"""The routing and the token exchange of an expert layer on gfx950
(include/ec_experts.h): experts chosen by their scores, tokens sorted by expert
and brought back with weights applied, with the gradients of all of it, and
dispatches that send the 4-bit form of mx.py or the 8-bit form of i8.py.

Calls run on torch's current stream of the tensors' device, or on `stream`, on
which the results are then allocated.  Results carry no autograd history: the
gradients are functions of their own.
"""
from __future__ import annotations

import math

import torch

from . import _binding as _b
from .i8 import I8Tensor, _empty_i8
from .mx import TYPES, MXTensor, _empty, _refuse, _rows, _type

SCORES = {"softmax": 0, "sigmoid": 1}


def _ints(t, shape) -> bool:
    return (isinstance(t, torch.Tensor) and t.dtype == torch.int32 and t.shape == shape
            and t.is_contiguous())


class Routing:
    """Where the choices ids [tokens, choices] go: order, int32 [tokens * choices], the flat choice
    of each sorted row (-1 past the last); place, int32 [tokens, choices], the row of each choice
    (-1: dropped); offsets, int32 [experts + 1], the rows of each expert."""

    __slots__ = ("order", "place", "offsets", "tokens", "choices", "experts")

    def __init__(self, order, place, offsets, tokens, choices, experts):
        if not (_ints(order, (tokens * choices,)) and _ints(place, (tokens, choices))
                and _ints(offsets, (experts + 1,)) and choices > 0 and experts > 0
                and order.device == place.device == offsets.device):
            _refuse("Routing: int32 order [tokens * choices], place [tokens, choices] and "
                    "offsets [experts + 1], contiguous and on one device, are wanted")
        self._set(order, place, offsets, tokens, choices, experts)

    def _set(self, order, place, offsets, tokens, choices, experts):
        self.order, self.place, self.offsets = order, place, offsets
        self.tokens, self.choices, self.experts = tokens, choices, experts


def _logits(x, score, scale, what):
    kind = _type(x, what)
    if x.dim() != 2 or x.shape[1] == 0 or score not in SCORES:
        _refuse(f"{what}: logits [tokens, experts] and a score of {sorted(SCORES)} are wanted")
    if not math.isfinite(scale):
        _refuse(f"{what}: a finite scale is wanted")
    return *_rows(x), kind


def expert_route(logits: torch.Tensor, choices: int, score: str = "softmax",
                 bias: torch.Tensor | None = None, groups: int = 1, top_groups: int = 1,
                 renormalize: bool = True, scale: float = 1.0, stream=None):
    """(ids, int32 [tokens, choices], weights, float32 [tokens, choices]) of logits [tokens,
    experts]: the experts with the largest score + bias (float32 [experts]; without a bias the
    largest logits), the largest first and of equal ones the lowest index, and their scores times
    scale, divided by the sum of the chosen scores with renormalize.

    score: "softmax" or "sigmoid".  With groups, experts are taken from the top_groups of as many
    runs of consecutive experts whose two best score + bias sum highest.  An expert whose logit is
    -inf is not taken: where none is left, the id is -1 (which expert_sort drops) and the weight 0."""
    if stream is not None or _b.elsewhere(logits):
        return _b.on_stream(expert_route, (logits, choices, score, bias, groups, top_groups,
                                           renormalize, scale), stream)
    r, stride, kind = _logits(logits, score, scale, "expert_route")
    tokens, experts = r.shape
    if (groups < 1 or experts % groups or not 0 < top_groups <= groups
            or not 0 < choices <= experts // groups * top_groups):
        _refuse("expert_route: groups of as many experts each, and no more choices than experts "
                "in top_groups of them are wanted")
    if bias is not None:
        if bias.dtype != torch.float32 or bias.shape != (experts,) or bias.device != r.device:
            _refuse("expert_route: a float32 bias [experts] on the logits' device is wanted")
        if not bias.is_contiguous():
            bias = bias.contiguous()
    ids = r.new_empty((tokens, choices), dtype=torch.int32)
    weights = r.new_empty((tokens, choices), dtype=torch.float32)
    _b.check(_b.lib().ec_expert_route(
        r.data_ptr(), kind, tokens, stride, experts, None if bias is None else bias.data_ptr(),
        choices, SCORES[score], groups, top_groups, bool(renormalize), scale, ids.data_ptr(),
        weights.data_ptr(), _b.current_stream(r)), "ec_expert_route")
    return ids, weights


def expert_route_backward(dweights: torch.Tensor, logits: torch.Tensor, ids: torch.Tensor,
                          score: str = "softmax", renormalize: bool = True, scale: float = 1.0,
                          stream=None) -> torch.Tensor:
    """dlogits [tokens, experts] of expert_route's weights, from dweights, float32 [tokens,
    choices], and the ids of the forward pass with its score, renormalize and scale.  Which experts
    are taken has no gradient, and so neither has the bias."""
    if stream is not None or _b.elsewhere(logits):
        return _b.on_stream(expert_route_backward,
                            (dweights, logits, ids, score, renormalize, scale), stream)
    r, stride, kind = _logits(logits, score, scale, "expert_route_backward")
    tokens, experts = r.shape
    if (ids.dim() != 2 or ids.dtype != torch.int32 or ids.shape[0] != tokens or ids.shape[1] == 0
            or dweights.dtype != torch.float32 or dweights.shape != ids.shape
            or ids.device != r.device or dweights.device != r.device):
        _refuse("expert_route_backward: int32 ids and float32 dweights [tokens, choices] on the "
                "logits' device are wanted")
    if not ids.is_contiguous():
        ids = ids.contiguous()
    if not dweights.is_contiguous():
        dweights = dweights.contiguous()
    dlogits = r.new_empty((tokens, experts))
    _b.check(_b.lib().ec_expert_route_backward(
        dweights.data_ptr(), r.data_ptr(), kind, tokens, stride, experts, ids.data_ptr(),
        ids.shape[1], SCORES[score], bool(renormalize), scale, dlogits.data_ptr(),
        _b.current_stream(r)), "ec_expert_route_backward")
    return dlogits


def expert_sort(ids: torch.Tensor, experts: int, stream=None) -> Routing:
    """Sort the choices ids [tokens, choices] (int32 or int64) stably by expert; ids outside
    [0, experts), as a router's -1, are dropped."""
    if stream is not None or _b.elsewhere(ids):
        return _b.on_stream(expert_sort, (ids, experts), stream)
    if ids.dim() != 2 or ids.dtype not in (torch.int32, torch.int64) or not ids.is_cuda or ids.shape[1] == 0:
        _refuse("expert_sort: int32 or int64 ids [tokens, choices] on the GPU are wanted")
    if not 0 < experts <= 0x7fffffff:
        _refuse("expert_sort: a positive number of experts is wanted")
    if not ids.is_contiguous():
        ids = ids.contiguous()
    n = ids.numel()
    place = torch.empty_like(ids, dtype=torch.int32)
    order, offsets = place.new_empty(n), place.new_empty(experts + 1)
    L = _b.lib()
    need = L.ec_expert_sort_workspace_bytes(n, experts)
    # held until the call is back: before, its kernels are not all enqueued
    ws = place.new_empty(need, dtype=torch.uint8) if need else None
    _b.check(L.ec_expert_sort(ids.data_ptr(), ids.element_size(), n, experts, order.data_ptr(),
                              place.data_ptr(), offsets.data_ptr(),
                              ws.data_ptr() if need else None, need,
                              _b.current_stream(ids)), "ec_expert_sort")
    r = object.__new__(Routing)  # of these arrays there is nothing to check
    r._set(order, place, offsets, ids.shape[0], ids.shape[1], experts)
    return r


def _tokens(x, r, what):
    kind = _type(x, what)
    if x.dim() != 2 or x.shape[0] != r.tokens or x.shape[1] == 0 or x.device != r.place.device:
        _refuse(f"{what}: [tokens, cols] on the routing's device is wanted")
    return (x if x.is_contiguous() else x.contiguous()), kind


def _sorted(x, r, what):
    kind = _type(x, what)
    if (x.dim() != 2 or x.shape[0] != r.tokens * r.choices or x.shape[1] == 0
            or x.device != r.place.device):
        _refuse(f"{what}: [tokens * choices, cols] on the routing's device is wanted")
    return (x if x.is_contiguous() else x.contiguous()), kind


def _weights(w, r, what):
    kind = _type(w, what)
    if w.shape != r.place.shape or w.device != r.place.device:
        _refuse(f"{what}: weights [tokens, choices] on the routing's device are wanted")
    return (w if w.is_contiguous() else w.contiguous()), kind


def expert_dispatch(x: torch.Tensor, routing: Routing, stream=None) -> torch.Tensor:
    """The tokens x [tokens, cols] in sorted order, [tokens * choices, cols]; zeros in rows of no
    expert."""
    if stream is not None or _b.elsewhere(x):
        return _b.on_stream(expert_dispatch, (x, routing), stream)
    r = routing
    x, kind = _tokens(x, r, "expert_dispatch")
    cols = x.shape[1]
    xs = x.new_empty((r.tokens * r.choices, cols))
    _b.check(_b.lib().ec_expert_dispatch(x.data_ptr(), kind, r.tokens, cols, r.place.data_ptr(),
                                         r.choices, r.offsets.data_ptr(), r.experts,
                                         xs.data_ptr(), _b.current_stream(x)),
             "ec_expert_dispatch")
    return xs


def expert_dispatch_mx(x: torch.Tensor, routing: Routing, stream=None) -> MXTensor:
    """The same in the 4-bit form: what an all-to-all then moves is 17/32 of a byte an element."""
    if stream is not None or _b.elsewhere(x):
        return _b.on_stream(expert_dispatch_mx, (x, routing), stream)
    r = routing
    x, kind = _tokens(x, r, "expert_dispatch_mx")
    cols = x.shape[1]
    q = _empty((r.tokens * r.choices,), cols, x)
    at = q.home.data_ptr()
    _b.check(_b.lib().ec_expert_dispatch_mx(x.data_ptr(), kind, r.tokens, cols,
                                            r.place.data_ptr(), r.choices, r.offsets.data_ptr(),
                                            r.experts, at, at + q._split,
                                            _b.current_stream(x)), "ec_expert_dispatch_mx")
    return q


def expert_dispatch_i8(x: I8Tensor, routing: Routing, stream=None) -> I8Tensor:
    """The same of tokens that are in the 8-bit form, as rms_norm_i8 makes them: x [tokens, cols]."""
    if stream is not None or _b.elsewhere(x.home):
        return _b.on_stream(expert_dispatch_i8, (x, routing), stream)
    r = routing
    if (len(x.lead) != 1 or x.lead[0] != r.tokens or x.cols == 0 or not x.home.is_cuda
            or x.home.device != r.place.device):
        _refuse("expert_dispatch_i8: rows [tokens, cols] on the routing's device are wanted")
    q = _empty_i8((r.tokens * r.choices,), x.cols, x.home)
    _b.check(_b.lib().ec_expert_dispatch_i8(
        *x.pointers(), r.tokens, x.padded, r.place.data_ptr(), r.choices, r.offsets.data_ptr(),
        r.experts, *q.pointers(), _b.current_stream(x.home)), "ec_expert_dispatch_i8")
    return q


def expert_dispatch_backward(dxs: torch.Tensor, routing: Routing, stream=None) -> torch.Tensor:
    """dx [tokens, cols]: each token's sum over its rows of dxs."""
    if stream is not None or _b.elsewhere(dxs):
        return _b.on_stream(expert_dispatch_backward, (dxs, routing), stream)
    r = routing
    dxs, kind = _sorted(dxs, r, "expert_dispatch_backward")
    dx = dxs.new_empty((r.tokens, dxs.shape[1]))
    _b.check(_b.lib().ec_expert_dispatch_backward(dxs.data_ptr(), kind, r.tokens, dxs.shape[1],
                                                  r.place.data_ptr(), r.choices, dx.data_ptr(),
                                                  _b.current_stream(dxs)),
             "ec_expert_dispatch_backward")
    return dx


def expert_combine(ys: torch.Tensor, routing: Routing, weights: torch.Tensor,
                   stream=None) -> torch.Tensor:
    """y [tokens, cols]: each token's weighted sum over its rows of ys [tokens * choices, cols]."""
    if stream is not None or _b.elsewhere(ys):
        return _b.on_stream(expert_combine, (ys, routing, weights), stream)
    r = routing
    ys, kind = _sorted(ys, r, "expert_combine")
    w, wkind = _weights(weights, r, "expert_combine")
    y = ys.new_empty((r.tokens, ys.shape[1]))
    _b.check(_b.lib().ec_expert_combine(ys.data_ptr(), kind, r.tokens, ys.shape[1],
                                        r.place.data_ptr(), r.choices, w.data_ptr(), wkind,
                                        y.data_ptr(), _b.current_stream(ys)), "ec_expert_combine")
    return y


def expert_combine_backward(dy: torch.Tensor, ys: torch.Tensor, routing: Routing,
                            weights: torch.Tensor, stream=None):
    """(dys [tokens * choices, cols], dweights [tokens, choices]) of expert_combine."""
    if stream is not None or _b.elsewhere(dy):
        return _b.on_stream(expert_combine_backward, (dy, ys, routing, weights), stream)
    r = routing
    dy, kind = _tokens(dy, r, "expert_combine_backward")
    ys, kind2 = _sorted(ys, r, "expert_combine_backward")
    w, wkind = _weights(weights, r, "expert_combine_backward")
    if kind != kind2 or dy.shape[1] != ys.shape[1]:
        _refuse("expert_combine_backward: dy and ys of one type and width are wanted")
    dys, dw = torch.empty_like(ys), torch.empty_like(w)
    _b.check(_b.lib().ec_expert_combine_backward(
        dy.data_ptr(), ys.data_ptr(), kind, r.tokens, ys.shape[1], r.place.data_ptr(), r.choices,
        w.data_ptr(), wkind, r.offsets.data_ptr(), r.experts, dys.data_ptr(), dw.data_ptr(),
        _b.current_stream(dy)), "ec_expert_combine_backward")
    return dys, dw
