"""The root-mean-square norm in front of a layer on gfx950 (include/ec_norm.h):
with the residual's addition, its output in x's type or in the 8-bit form of
i8.py, and its gradients.

Calls run on torch's current stream of the tensors' device, or on `stream`, on
which the results are then allocated.  Results carry no autograd history: the
gradients are a function of their own.
"""
from __future__ import annotations

import torch

from . import _binding as _b
from .i8 import I8Tensor, _empty_i8
from .mx import TYPES, _refuse, _rows, _type


def _inputs(x, weight, residual, what):
    """x and the residual as rows with their strides, the contiguous weight, and the types."""
    kind, wkind = _type(x, what), _type(weight, what)
    cols = x.shape[-1] if x.dim() else 0
    if cols == 0 or weight.shape != (cols,) or weight.device != x.device:
        _refuse(f"{what}: x [.., cols] and weight [cols] on one device are wanted")
    if not weight.is_contiguous():
        weight = weight.contiguous()
    r, stride = _rows(x)
    if residual is None:
        return r, stride, None, 0, kind, weight, wkind
    if (residual.shape != x.shape or residual.dtype != x.dtype
            or residual.device != x.device):
        _refuse(f"{what}: a residual of x's shape, type and device is wanted")
    return r, stride, *_rows(residual), kind, weight, wkind


def _like(x):
    """A contiguous tensor of x's form (torch's own empty_like takes less time, but keeps strides)."""
    return torch.empty_like(x) if x.is_contiguous() else x.new_empty(x.shape)


def _norm(x, weight, eps, residual, saved, what):
    r, stride, s, s_stride, kind, weight, wkind = _inputs(x, weight, residual, what)
    rows, cols = r.shape
    y, h = _like(x), None if s is None else _like(x)
    rstd = x.new_empty(rows, dtype=torch.float32) if saved else None
    _b.check(_b.lib().ec_rms_norm(
        r.data_ptr(), stride, None if s is None else s.data_ptr(), s_stride, kind, rows, cols,
        weight.data_ptr(), wkind, eps, None if h is None else h.data_ptr(), y.data_ptr(),
        rstd.data_ptr() if saved else None, _b.current_stream(x)), "ec_rms_norm")
    return y, h, rstd, weight


def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
             residual: torch.Tensor | None = None, stream=None):
    """y = h / sqrt(mean(h^2) + eps) weight of x [.., cols] and weight [cols], with h = x; with a
    residual (y, h), h = x + residual in x's type."""
    if stream is not None or _b.elsewhere(x):
        return _b.on_stream(rms_norm, (x, weight, eps, residual), stream)
    y, h, _, _ = _norm(x, weight, eps, residual, False, "rms_norm")
    return y if h is None else (y, h)


def rms_norm_i8(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                residual: torch.Tensor | None = None, stream=None):
    """The same with y in the 8-bit form, an I8Tensor: what i8_product and expert_dispatch_i8
    read."""
    if stream is not None or _b.elsewhere(x):
        return _b.on_stream(rms_norm_i8, (x, weight, eps, residual), stream)
    r, stride, s, s_stride, kind, weight, wkind = _inputs(x, weight, residual, "rms_norm_i8")
    rows, cols = r.shape
    q: I8Tensor = _empty_i8(x.shape[:-1], cols, x)
    h = None if s is None else _like(x)
    at = q.home.data_ptr()
    _b.check(_b.lib().ec_rms_norm_i8(
        r.data_ptr(), stride, None if s is None else s.data_ptr(), s_stride, kind, rows, cols,
        weight.data_ptr(), wkind, eps, None if h is None else h.data_ptr(), at, at + q._split,
        _b.current_stream(x)), "ec_rms_norm_i8")
    return q if h is None else (q, h)


class RMSNormSaved:
    """What the backward pass of the norm needs: h (the sum, or x itself), 1 / sqrt(mean(h^2) +
    eps) of each row, and the weight.  They have to keep their values until then: writes that torch
    counts are found."""

    __slots__ = ("h", "rstd", "weight", "versions")

    def __init__(self, h, rstd, weight):
        self.h, self.rstd, self.weight = h, rstd, weight
        # How often torch counts that they were written to (None: it does not count, for an
        # inference tensor and in a graph, whose replays the count knows nothing of).
        self.versions = None, None
        if not _b.capturing(h):
            self.versions = tuple(None if t.is_inference() else t._version for t in (h, weight))

    def same_values(self) -> bool:
        h, weight = self.versions
        return ((h is None or h == self.h._version)
                and (weight is None or weight == self.weight._version))

    def __reduce__(self):
        if not self.same_values():
            _refuse("RMSNormSaved: its tensors were written to since the forward pass")
        return RMSNormSaved, (self.h, self.rstd, self.weight)


def rms_norm_forward(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                     residual: torch.Tensor | None = None, stream=None):
    """y of rms_norm and what the backward pass needs, which holds the sum as `h`."""
    if stream is not None or _b.elsewhere(x):
        return _b.on_stream(rms_norm_forward, (x, weight, eps, residual), stream)
    y, h, rstd, weight = _norm(x, weight, eps, residual, True, "rms_norm_forward")
    return y, RMSNormSaved(x if h is None else h, rstd, weight)


def rms_norm_backward(dy: torch.Tensor, saved: RMSNormSaved, dh: torch.Tensor | None = None,
                      stream=None):
    """(dx, dweight) from dy and dh, the gradient that reaches h by other ways: dx, of h's shape,
    is the gradient of x and of the residual alike."""
    if stream is not None or _b.elsewhere(dy):
        return _b.on_stream(rms_norm_backward, (dy, saved, dh), stream)
    h, rstd, weight = saved.h, saved.rstd, saved.weight
    kind = _type(dy, "rms_norm_backward")
    shape, device = h.shape, h.device
    if (dy.shape != shape or dy.dtype != h.dtype or dy.device != device or dh is not None
            and (dh.shape != shape or dh.dtype != h.dtype or dh.device != device)):
        _refuse("rms_norm_backward: gradients of the forward's shape, type and device are wanted")
    if not saved.same_values():
        _refuse("rms_norm_backward: what was saved was written to since the forward pass")
    if not h.is_contiguous():
        h = h.contiguous()
    if not dy.is_contiguous():
        dy = dy.contiguous()
    if dh is not None and not dh.is_contiguous():
        dh = dh.contiguous()
    dx, dweight = torch.empty_like(h), torch.empty_like(weight)
    rows, cols = rstd.shape[0], shape[-1]
    L = _b.lib()
    need = L.ec_rms_norm_backward_workspace_bytes(rows, cols)
    # held until the call is back: before, its kernels are not all enqueued
    ws = h.new_empty(need, dtype=torch.uint8) if need else None
    _b.check(L.ec_rms_norm_backward(
        dy.data_ptr(), h.data_ptr(), None if dh is None else dh.data_ptr(), kind, rows, cols,
        rstd.data_ptr(), weight.data_ptr(), TYPES[weight.dtype], dx.data_ptr(),
        dweight.data_ptr(), ws.data_ptr() if need else None, need, _b.current_stream(dy)),
        "ec_rms_norm_backward")
    return dx, dweight
