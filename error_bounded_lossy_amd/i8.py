"""The 8-bit integer form on gfx950 (include/ec_i8.h): rows of whole numbers
with one scale each, and products of them on the matrix cores.

Calls run on torch's current stream of the tensors' device, or on `stream`, on
which the results are then allocated.  Results carry no autograd history: the
form is for serving (training has the block scales of mx.py).
"""
from __future__ import annotations

import math

import torch

from . import _binding as _b
from .mx import TYPES, _offsets, _refuse, _rows, _type

# of a product that may be taken in parts of its contraction (include/ec_i8.h)
MOST_PARTS_ROWS = 256


class I8Tensor:
    """A tensor in the 8-bit form along its last dimension, of `cols` elements: codes, int8
    [..., padded] with zeros from cols on, and scales, float32 [...]."""

    # What the library makes holds both in one allocation, `home`, codes first (`_scales` is None,
    # and `_split` the bytes of codes), and has them as tensors only when asked, as an MXTensor
    # does.  Addresses are taken from the tensors at each call: a caller may replace their memory, as
    # a module does that moves or converts what it holds, but not their form.
    __slots__ = ("cols", "padded", "lead", "home", "_scales", "_split", "_checked")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, cols: int):
        p = (cols + 127) // 128 * 128
        *lead, width = form = codes.shape
        if (codes.dtype != torch.int8 or scales.dtype != torch.float32 or cols < 0
                or width != p or list(scales.shape) != lead
                or not codes.is_contiguous() or not scales.is_contiguous()
                or codes.device != scales.device):
            _refuse("I8Tensor: int8 codes [..., padded] and float32 scales [...], contiguous and "
                    "on one device, are wanted")
        self.cols, self.padded, self.lead = cols, p, form[:-1]
        self.home, self._scales, self._split = codes, scales, codes.numel()
        self._checked = codes.data_ptr(), scales.data_ptr()

    def __reduce__(self):
        return _restored, (self.home, self._scales, tuple(self.lead), self.cols)

    def _moved(self) -> tuple[int, int]:
        """The addresses of memory that is not where or what it was: of the same form, or refused."""
        codes, scales = self.home, self._scales
        if scales is None:
            ok = codes.shape == (math.prod(self.lead) * (self.padded + 4),)
        else:
            ok = (codes.shape == (*self.lead, self.padded) and scales.shape == self.lead
                  and scales.dtype == torch.float32 and scales.is_contiguous()
                  and scales.device == codes.device)
        if not ok or codes.dtype != torch.int8 or not codes.is_contiguous():
            _refuse("I8Tensor: its memory was replaced by some of another form")
        start = codes.data_ptr()
        self._checked = start, start + self._split if scales is None else scales.data_ptr()
        return self._checked

    def pointers(self) -> tuple[int, int]:
        """Where codes and scales are now."""
        home, scales, split = self.home, self._scales, self._split
        start = home.data_ptr()
        if scales is None:
            at = start, start + split
            return at if at == self._checked else self._moved()
        at = start, scales.data_ptr()
        # (the type is looked at each time: a module that is converted twice may have scales of
        # another one where the first ones were)
        if (at != self._checked or home.numel() != split or scales.dtype != torch.float32
                or scales.numel() * self.padded != split or not home.is_contiguous()
                or not scales.is_contiguous()):
            return self._moved()
        return at

    @property
    def codes(self) -> torch.Tensor:
        if self._scales is not None:
            return self.home
        return self.home[:self._split].view(*self.lead, self.padded)

    @property
    def scales(self) -> torch.Tensor:
        if self._scales is not None:
            return self._scales
        return self.home[self._split:].view(torch.float32).view(self.lead)

    @property
    def shape(self) -> torch.Size:
        return torch.Size((*self.lead, self.cols))

    @property
    def device(self) -> torch.device:
        return self.home.device

    def numel_bytes(self) -> int:
        return math.prod(self.lead) * (self.padded + 4)


def _empty_i8(lead, cols, like) -> I8Tensor:
    """`like`: any tensor on the device.  Of these forms there is nothing to check."""
    q = object.__new__(I8Tensor)
    q.cols, q.padded, q.lead, q._scales = cols, (cols + 127) // 128 * 128, lead, None
    rows = math.prod(lead)
    q._split = rows * q.padded  # a multiple of 128: the scales behind are aligned
    q.home = like.new_empty(q._split + rows * 4, dtype=torch.int8)
    start = q.home.data_ptr()
    q._checked = start, start + q._split
    return q


def _restored(home, scales, lead, cols) -> I8Tensor:
    """An I8Tensor of the parts that a copy or a file holds."""
    if scales is not None:
        return I8Tensor(home, scales, cols)
    rows, padded = math.prod(lead), (cols + 127) // 128 * 128
    if (home.dtype != torch.int8 or home.shape != (rows * (padded + 4),) or cols < 0
            or not home.is_contiguous()):
        _refuse("I8Tensor: int8 memory of codes and scales in one piece is wanted")
    q = object.__new__(I8Tensor)
    q.cols, q.padded, q.lead, q.home = cols, padded, torch.Size(lead), home
    q._scales, q._split, q._checked = None, rows * padded, None
    return q


def i8_quantize(x: torch.Tensor, stream=None) -> I8Tensor:
    """x [..., cols] in the 8-bit form along its last dimension, one scale a row."""
    if stream is not None or _b.elsewhere(x):
        return _b.on_stream(i8_quantize, (x,), stream)
    kind = _type(x, "i8_quantize")
    if x.dim() == 0 or x.shape[-1] == 0:
        _refuse("i8_quantize: at least one element a row is wanted")
    r, stride = _rows(x)
    q = _empty_i8(x.shape[:-1], x.shape[-1], x)
    _b.check(_b.lib().ec_i8_quantize(r.data_ptr(), kind, r.shape[0], r.shape[1], stride,
                                     *q.pointers(), _b.current_stream(x)), "ec_i8_quantize")
    return q


def i8_dequantize(q: I8Tensor, dtype: torch.dtype = torch.float32, stream=None) -> torch.Tensor:
    """The values that q holds, rounded once to dtype."""
    if stream is not None or _b.elsewhere(q.home):
        return _b.on_stream(i8_dequantize, (q, dtype), stream)
    kind = TYPES.get(dtype)
    if kind is None or not q.home.is_cuda or q.cols == 0:
        _refuse("i8_dequantize: a nonempty row on the GPU and float32, float16 or bfloat16 are wanted")
    y = q.home.new_empty((*q.lead, q.cols), dtype=dtype)
    _b.check(_b.lib().ec_i8_dequantize(*q.pointers(), y.numel() // q.cols, q.cols, y.data_ptr(), kind,
                                       q.cols, _b.current_stream(y)), "ec_i8_dequantize")
    return y


def i8_product(a: I8Tensor, b: I8Tensor, dtype: torch.dtype = torch.bfloat16,
               stream=None) -> torch.Tensor:
    """a b^T [rows, cols] of a [rows, depth] and b [cols, depth], summed in whole numbers."""
    if stream is not None or _b.elsewhere(a.home):
        return _b.on_stream(i8_product, (a, b, dtype), stream)
    kind = TYPES.get(dtype)
    if (kind is None or len(a.lead) != 1 or len(b.lead) != 1 or a.cols != b.cols or a.cols == 0
            or b.lead[0] == 0 or not a.home.is_cuda or a.home.device != b.home.device):
        _refuse("i8_product: [rows, depth] and [cols, depth] on one GPU are wanted")
    rows, cols = a.lead[0], b.lead[0]
    y = a.home.new_empty((rows, cols), dtype=dtype)
    need = _b.lib().ec_i8_product_parts_bytes(rows, cols, a.padded) if rows <= MOST_PARTS_ROWS else 0
    if need:
        # held until the call is back: before, its kernels are not all enqueued
        ws = a.home.new_empty(need, dtype=torch.int8)
        _b.check(_b.lib().ec_i8_product_parts(*a.pointers(), rows, *b.pointers(), cols, a.padded,
                                              y.data_ptr(), kind, ws.data_ptr(), need,
                                              _b.current_stream(y)), "ec_i8_product_parts")
        return y
    _b.check(_b.lib().ec_i8_product(*a.pointers(), rows, *b.pointers(), cols, a.padded,
                                    y.data_ptr(), kind, _b.current_stream(y)), "ec_i8_product")
    return y


def i8_experts_product(a: I8Tensor, b: I8Tensor, offsets: torch.Tensor,
                       dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """Rows a [rows, depth] sorted by expert, rows [offsets[e], offsets[e + 1]) times the weights of
    expert e, b [experts, cols, depth]; zeros in rows of no expert."""
    if stream is not None or _b.elsewhere(a.home):
        return _b.on_stream(i8_experts_product, (a, b, offsets, dtype), stream)
    kind = TYPES.get(dtype)
    if (kind is None or len(a.lead) != 1 or len(b.lead) != 2 or a.cols != b.cols or a.cols == 0
            or 0 in b.lead or not a.home.is_cuda or a.home.device != b.home.device):
        _refuse("i8_experts_product: [rows, depth] and [experts, cols, depth] on one GPU are wanted")
    experts, cols = b.lead
    _offsets(offsets, experts, a.home.device, "i8_experts_product")
    rows = a.lead[0]
    y = a.home.new_empty((rows, cols), dtype=dtype)
    _b.check(_b.lib().ec_i8_product_experts(*a.pointers(), rows, *b.pointers(), cols, a.padded,
                                            offsets.data_ptr(), experts, y.data_ptr(), kind,
                                            _b.current_stream(y)), "ec_i8_product_experts")
    return y


def _linear(x, w, offsets, experts, what):
    kind = _type(x, what)
    cols, depth = w.lead[-1], x.shape[-1]
    if w.cols != depth or depth == 0 or 0 in w.lead or w.home.device != x.device:
        _refuse(f"{what}: weights [.., cols, depth] on the device of x [.., depth] are wanted")
    r, stride = _rows(x)
    rows = r.shape[0]
    L = _b.lib()
    y = x.new_empty((*x.shape[:-1], cols))
    need = L.ec_i8_linear_workspace_bytes(rows, depth, cols, experts)
    # held until the call is back: before, its kernels are not all enqueued
    ws = w.home.new_empty(need, dtype=torch.int8) if need else None
    _b.check(L.ec_i8_linear(r.data_ptr(), kind, rows, depth, stride, *w.pointers(), cols,
                            offsets.data_ptr() if experts else None, experts, y.data_ptr(),
                            ws.data_ptr() if need else None, need,
                            _b.current_stream(x)), "ec_i8_linear")
    return y


def i8_linear(x: torch.Tensor, w: I8Tensor, stream=None) -> torch.Tensor:
    """x w^T with x [..., depth] quantized on the way, one scale a row, and weights w [cols, depth]
    with one scale an output channel."""
    if stream is not None or _b.elsewhere(x):
        return _b.on_stream(i8_linear, (x, w), stream)
    if len(w.lead) != 1 or x.dim() == 0:
        _refuse("i8_linear: x [.., depth] and weights [cols, depth] are wanted")
    return _linear(x, w, None, 0, "i8_linear")


def i8_experts_linear(x: torch.Tensor, w: I8Tensor, offsets: torch.Tensor,
                      stream=None) -> torch.Tensor:
    """i8_experts_product of rows x [rows, depth] that are quantized on the way."""
    if stream is not None or _b.elsewhere(x):
        return _b.on_stream(i8_experts_linear, (x, w, offsets), stream)
    if len(w.lead) != 2 or x.dim() != 2:
        _refuse("i8_experts_linear: x [rows, depth] and weights [experts, cols, depth] are wanted")
    _offsets(offsets, w.lead[0], x.device, "i8_experts_linear")
    return _linear(x, w, offsets, w.lead[0], "i8_experts_linear")
