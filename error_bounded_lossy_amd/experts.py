"""The token exchange of an expert layer on gfx950 (include/ec_experts.h):
tokens sorted by expert and brought back with weights applied, with the
gradients of both ways, and a dispatch that sends the 4-bit form of mx.py.

Calls run on torch's current stream of the tensors' device, or on `stream`, on
which the results are then allocated.  Results carry no autograd history: the
gradients are functions of their own.
"""
from __future__ import annotations

import torch

from . import _binding as _b
from .mx import TYPES, MXTensor, _empty, _refuse, _type


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
