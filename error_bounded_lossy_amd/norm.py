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
    """x and the residual as rows with their strides, and the types."""
    kind = _type(x, what)
    wkind = _type(weight, what)
    if (x.dim() == 0 or x.shape[-1] == 0 or weight.shape != x.shape[-1:]
            or weight.device != x.device):
        _refuse(f"{what}: x [.., cols] and weight [cols] on one device are wanted")
    if residual is not None and (residual.shape != x.shape or residual.dtype != x.dtype
                                 or residual.device != x.device):
        _refuse(f"{what}: a residual of x's shape, type and device is wanted")
    r, stride = _rows(x)
    s, s_stride = (None, 0) if residual is None else _rows(residual)
    return r, stride, s, s_stride, kind, weight.contiguous(), wkind


def _norm(x, weight, eps, residual, saved, what):
    r, stride, s, s_stride, kind, weight, wkind = _inputs(x, weight, residual, what)
    y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    h = None if s is None else torch.empty_like(y)
    rstd = torch.empty(r.shape[0], dtype=torch.float32, device=x.device) if saved else None
    _b.check(_b.lib().ec_rms_norm(
        r.data_ptr(), stride, None if s is None else s.data_ptr(), s_stride, kind, r.shape[0],
        r.shape[1], weight.data_ptr(), wkind, eps, None if h is None else h.data_ptr(),
        y.data_ptr(), rstd.data_ptr() if saved else None, _b.current_stream(x)), "ec_rms_norm")
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
    q: I8Tensor = _empty_i8(x.shape[:-1], x.shape[-1], x)
    h = None if s is None else torch.empty(x.shape, dtype=x.dtype, device=x.device)
    _b.check(_b.lib().ec_rms_norm_i8(
        r.data_ptr(), stride, None if s is None else s.data_ptr(), s_stride, kind, r.shape[0],
        r.shape[1], weight.data_ptr(), wkind, eps, None if h is None else h.data_ptr(),
        *q.pointers(), _b.current_stream(x)), "ec_rms_norm_i8")
    return q if h is None else (q, h)


class RMSNormSaved:
    """What the backward pass of the norm needs: h (the sum, or x itself), 1 / sqrt(mean(h^2) +
    eps) of each row, and the weight.  None of them may be written to until then."""

    __slots__ = ("h", "rstd", "weight")

    def __init__(self, h, rstd, weight):
        self.h, self.rstd, self.weight = h, rstd, weight


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
    _type(dy, "rms_norm_backward")
    for t in (dy,) if dh is None else (dy, dh):
        if t.shape != h.shape or t.dtype != h.dtype or t.device != h.device:
            _refuse("rms_norm_backward: gradients of the forward's shape, type and device are wanted")
    dy, h = dy.contiguous(), h.contiguous()
    dh = None if dh is None else dh.contiguous()
    dx, dweight = torch.empty_like(h), torch.empty_like(weight)
    rows, cols = rstd.shape[0], h.shape[-1]
    L = _b.lib()
    need = L.ec_rms_norm_backward_workspace_bytes(rows, cols)
    # held until the call is back: before, its kernels are not all enqueued
    ws = h.new_empty(need, dtype=torch.uint8) if need else None
    _b.check(L.ec_rms_norm_backward(
        dy.data_ptr(), h.data_ptr(), None if dh is None else dh.data_ptr(), TYPES[h.dtype], rows,
        cols, rstd.data_ptr(), weight.data_ptr(), TYPES[weight.dtype], dx.data_ptr(),
        dweight.data_ptr(), ws.data_ptr() if need else None, need, _b.current_stream(dy)),
        "ec_rms_norm_backward")
    return dx, dweight
