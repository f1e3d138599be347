"""The microscaled 4-bit floating-point format on gfx950 (include/ec_mx.h):
quantization, its inverse, products of 4-bit operands, and the training steps
of a layer and of an expert layer built from them.

Like the rest of the binding this module only checks and marshals arguments;
every step runs in the library's kernels on torch's current stream of the
tensors' device, or on `stream`, on which the results are then allocated (the
caller orders that stream after what produced the inputs).  Results carry no
autograd history, whatever their inputs have: gradients come from the backward
functions, which a torch.autograd.Function may call.
"""
from __future__ import annotations

import math

import torch

from . import _binding as _b
from ._binding import EC_ERR_INVALID, ECError

TYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}


def _refuse(what: str):
    raise ECError(EC_ERR_INVALID, what)


def _type(t: torch.Tensor, what: str) -> int:
    code = TYPES.get(t.dtype)
    if code is None or not t.is_cuda:
        _refuse(f"{what}: a float32, float16 or bfloat16 tensor on the GPU is wanted")
    return code


def _rows(x: torch.Tensor) -> tuple[torch.Tensor, int]:
    """x as [rows, cols] with unit column stride, and its row stride (a copy only where its strides
    allow no view).  Strides of sizes of one hold anything: those of contiguous rows are not read."""
    if x.dim() != 2:
        x = x.reshape(-1, x.shape[-1])
    if not x.is_contiguous():
        if x.stride(1) == 1 and x.stride(0) >= x.shape[1]:
            return x, x.stride(0)
        x = x.contiguous()
    return x, x.shape[1]


class MXTensor:
    """A tensor in the 4-bit form along its last dimension, of `cols` elements:
    codes, uint8 [..., padded / 2], and scales, uint8 [..., padded / 32]."""

    # What the library makes holds both in one allocation, `home`, codes first (`_scales` is None,
    # and `_split` the bytes of codes), and has them as tensors only when asked: an allocation or a
    # view costs the host as much as a small kernel.  Addresses are taken from the tensors at each
    # call: copies, and tensors whose memory the caller replaces, are read where they are.
    __slots__ = ("cols", "padded", "lead", "home", "_scales", "_split", "_checked")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, cols: int):
        p = (cols + 127) // 128 * 128
        *lead, half = form = codes.shape
        if (codes.dtype != torch.uint8 or scales.dtype != torch.uint8 or cols < 0
                or half * 2 != p or scales.shape != (*lead, p // 32)
                or not codes.is_contiguous() or not scales.is_contiguous()
                or codes.device != scales.device):
            _refuse("MXTensor: uint8 codes [..., padded / 2] and scales [..., padded / 32], "
                    "contiguous and on one device, are wanted")
        self.cols, self.padded, self.lead = cols, p, form[:-1]
        self.home, self._scales, self._split = codes, scales, codes.numel()
        self._checked = codes.data_ptr(), scales.data_ptr()

    def __reduce__(self):
        return _restored, (self.home, self._scales, tuple(self.lead), self.cols, self.padded)

    def _moved(self) -> tuple[int, int]:
        """The addresses of a caller's tensors that are not where or what they were."""
        for t, per in ((self.home, 2), (self._scales, 32)):
            if (t.shape != (*self.lead, self.padded // per) or t.dtype != torch.uint8
                    or not t.is_contiguous() or t.device != self.home.device):
                _refuse("MXTensor: its memory was replaced by some of another form")
        self._checked = self.home.data_ptr(), self._scales.data_ptr()
        return self._checked

    def pointers(self) -> tuple[int, int]:
        """Where codes and scales are now."""
        scales = self._scales
        if scales is None:
            start = self.home.data_ptr()
            return start, start + self._split
        codes = self.home
        at = codes.data_ptr(), scales.data_ptr()
        if (at != self._checked or codes.numel() != self._split
                or scales.numel() * 16 != self._split or not codes.is_contiguous()
                or not scales.is_contiguous()):
            return self._moved()
        return at

    @property
    def codes(self) -> torch.Tensor:
        if self._scales is not None:
            return self.home
        return self.home[:self._split].view(*self.lead, self.padded // 2)

    @property
    def scales(self) -> torch.Tensor:
        if self._scales is not None:
            return self._scales
        return self.home[self._split:].view(*self.lead, self.padded // 32)

    @property
    def codes_ptr(self) -> int:
        return self.pointers()[0]

    @property
    def scales_ptr(self) -> int:
        return self.pointers()[1]

    @property
    def shape(self) -> torch.Size:
        return torch.Size((*self.lead, self.cols))

    @property
    def device(self) -> torch.device:
        return self.home.device

    def numel_bytes(self) -> int:
        return math.prod(self.lead) * (self.padded // 32) * 17


def _empty(lead, cols, like, p=None) -> MXTensor:
    m = object.__new__(MXTensor)
    m.cols, m.padded, m.lead = cols, (cols + 127) // 128 * 128 if p is None else p, lead
    # bytes of codes, the scales behind: a multiple of 64, so both are aligned
    m._split = math.prod(lead) * (m.padded // 2)
    m.home = like.new_empty(m._split // 16 * 17, dtype=torch.uint8)
    m._scales = m._checked = None
    return m


def _restored(home, scales, lead, cols, p) -> MXTensor:
    """An MXTensor of the parts that a copy or a file holds."""
    if scales is not None:
        return MXTensor(home, scales, cols)
    m = object.__new__(MXTensor)
    m.cols, m.padded, m.lead, m.home = cols, p, torch.Size(lead), home
    m._split = math.prod(lead) * (p // 2)
    m._scales = m._checked = None
    if (home.dtype != torch.uint8 or home.shape != (m._split // 16 * 17,)
            or not home.is_contiguous() or cols < 0 or p % 128 or p < cols):
        _refuse("MXTensor: uint8 memory in one piece is wanted, and rows padded to 128 elements")
    return m


def mx_quantize(x: torch.Tensor, stream=None) -> MXTensor:
    """x [..., cols] in the 4-bit form along its last dimension."""
    if stream is not None or _b.elsewhere(x):
        return _b.on_stream(mx_quantize, (x,), stream)
    kind = _type(x, "mx_quantize")
    if x.dim() == 0 or x.shape[-1] == 0:
        _refuse("mx_quantize: at least one element a row is wanted")
    r, stride = _rows(x)
    q = _empty(x.shape[:-1], x.shape[-1], x)
    at = q.home.data_ptr()
    _b.check(_b.lib().ec_mx_quantize(r.data_ptr(), kind, r.shape[0], r.shape[1], stride, at,
                                     at + q._split, _b.current_stream(x)), "ec_mx_quantize")
    return q


def mx_quantize_both(x: torch.Tensor, stream=None) -> tuple[MXTensor, MXTensor]:
    """x [rows, cols] or [batch, rows, cols] along its rows, and transposed along its columns
    ([..., cols, rows]), in one pass over x."""
    if stream is not None or _b.elsewhere(x):
        return _b.on_stream(mx_quantize_both, (x,), stream)
    kind = _type(x, "mx_quantize_both")
    if x.dim() not in (2, 3) or x.shape[-1] == 0:
        _refuse("mx_quantize_both: [rows, cols] or [batch, rows, cols] is wanted")
    rows, cols = x.shape[-2:]
    if not x.is_contiguous() and (x.stride(-1) != 1 or x.stride(-2) < cols):
        x = x.contiguous()
    stride, batch_stride = cols, rows * cols
    if not x.is_contiguous():
        stride, batch_stride = x.stride(-2), x.stride(0)
    lead = x.shape[:-2]
    batch = x.shape[0] if x.dim() == 3 else 1
    a, b = _empty((*lead, rows), cols, x), _empty((*lead, cols), rows, x)
    if rows and batch:
        at, bt = a.home.data_ptr(), b.home.data_ptr()
        _b.check(_b.lib().ec_mx_quantize_both(
            x.data_ptr(), kind, batch, rows, cols, batch_stride, stride, at, at + a._split, bt,
            bt + b._split, _b.current_stream(x)), "ec_mx_quantize_both")
    return a, b


def mx_dequantize(q: MXTensor, dtype: torch.dtype = torch.float32, stream=None) -> torch.Tensor:
    """The values that q holds, rounded once to dtype."""
    if stream is not None or _b.elsewhere(q.home):
        return _b.on_stream(mx_dequantize, (q, dtype), stream)
    kind = TYPES.get(dtype)
    if kind is None or not q.home.is_cuda or q.cols == 0 or q.padded - q.cols > 127:
        _refuse("mx_dequantize: a nonempty row on the GPU and float32, float16 or bfloat16 are wanted")
    lead = q.lead
    y = q.home.new_empty((*lead, q.cols), dtype=dtype)
    rows = y.numel() // q.cols
    _b.check(_b.lib().ec_mx_dequantize(*q.pointers(), rows, q.cols,
                                       y.data_ptr(), kind, q.cols, _b.current_stream(y)),
             "ec_mx_dequantize")
    return y


def _offsets(offsets: torch.Tensor, groups: int, device, what: str) -> torch.Tensor:
    if (offsets.dtype != torch.int32 or offsets.dim() != 1 or not offsets.is_contiguous()
            or offsets.shape[0] != groups + 1 or offsets.device != device):
        _refuse(f"{what}: int32 offsets [experts + 1] on the tensors' device are wanted")
    return offsets


def mx_product(a: MXTensor, b: MXTensor, dtype: torch.dtype = torch.bfloat16,
               stream=None) -> torch.Tensor:
    """a b^T [rows, cols] of a [rows, depth] and b [cols, depth], summed in fp32, rounded once."""
    if stream is not None or _b.elsewhere(a.home):
        return _b.on_stream(mx_product, (a, b, dtype), stream)
    kind = TYPES.get(dtype)
    if (kind is None or len(a.lead) != 1 or len(b.lead) != 1 or a.cols != b.cols or a.cols == 0
            or a.padded != b.padded or a.padded - a.cols > 127
            or not a.home.is_cuda or a.home.device != b.home.device):
        _refuse("mx_product: [rows, depth] and [cols, depth] on one GPU are wanted")
    rows, cols = a.lead[0], b.lead[0]
    y = a.home.new_empty((rows, cols), dtype=dtype)
    _b.check(_b.lib().ec_mx_product(*a.pointers(), rows, *b.pointers(), cols, a.padded,
                                    y.data_ptr(), kind, _b.current_stream(y)), "ec_mx_product")
    return y


def _linear(x, w, offsets, experts, what):
    kind = _type(x, what)
    cols, depth = w.lead[-1], x.shape[-1]
    if (w.cols != depth or depth == 0 or w.padded - depth > 127
            or w.home.device != x.device):
        _refuse(f"{what}: weights [.., cols, depth] on the device of x [.., depth] are wanted")
    r, stride = _rows(x)
    rows = r.shape[0]
    L = _b.lib()
    y = x.new_empty((*x.shape[:-1], cols))
    need = L.ec_mx_linear_workspace_bytes(rows, depth, cols, experts)
    # held until the call is back: before, its kernels are not all enqueued
    ws = w.home.new_empty(need) if need else None
    _b.check(L.ec_mx_linear(r.data_ptr(), kind, rows, depth, stride, *w.pointers(), cols,
                            offsets.data_ptr() if experts else None, experts, y.data_ptr(),
                            ws.data_ptr() if need else None, need,
                            _b.current_stream(x)), "ec_mx_linear")
    return y


def mx_linear(x: torch.Tensor, w: MXTensor, stream=None) -> torch.Tensor:
    """x w^T with x [..., depth] quantized on the way and weights w [cols, depth]."""
    if stream is not None or _b.elsewhere(x):
        return _b.on_stream(mx_linear, (x, w), stream)
    if len(w.lead) != 1:
        _refuse("mx_linear: weights [cols, depth] are wanted")
    return _linear(x, w, None, 0, "mx_linear")


def mx_experts_linear(x: torch.Tensor, w: MXTensor, offsets: torch.Tensor,
                      stream=None) -> torch.Tensor:
    """Rows x [rows, depth] sorted by expert, rows [offsets[e], offsets[e + 1]) times the weights
    of expert e, w [experts, cols, depth]; zeros in rows of no expert."""
    if stream is not None or _b.elsewhere(x):
        return _b.on_stream(mx_experts_linear, (x, w, offsets), stream)
    if len(w.lead) != 2 or x.dim() != 2:
        _refuse("mx_experts_linear: x [rows, depth] and weights [experts, cols, depth] are wanted")
    experts = w.lead[0]
    _offsets(offsets, experts, x.device, "mx_experts_linear")
    return _linear(x, w, offsets, experts, "mx_experts_linear")


def mx_experts_product(a: MXTensor, b: MXTensor, offsets: torch.Tensor,
                       dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """mx_experts_linear of rows that are in the 4-bit form already, as expert_dispatch_mx makes
    them: a [rows, depth], b [experts, cols, depth]."""
    if stream is not None or _b.elsewhere(a.home):
        return _b.on_stream(mx_experts_product, (a, b, offsets, dtype), stream)
    if (dtype not in TYPES or len(a.lead) != 1 or len(b.lead) != 2 or a.cols != b.cols
            or a.cols == 0 or 0 in b.lead or a.padded != b.padded or a.padded - a.cols > 127
            or not a.home.is_cuda
            or a.home.device != b.home.device):
        _refuse("mx_experts_product: [rows, depth] and [experts, cols, depth] on one GPU are wanted")
    _offsets(offsets, b.lead[0], a.home.device, "mx_experts_product")
    return _experts_product(a, b, offsets, dtype)


class MXLinearSaved:
    """What the backward pass of a 4-bit layer needs: its input and weights along their columns
    (17/32 of a byte an element), and for experts the offsets.  An input's columns in groups are
    padded by group: only the backward pass reads them."""

    __slots__ = ("x", "w", "offsets", "rows", "dtype", "version")

    def __init__(self, x, w, offsets, rows, dtype):
        self.x, self.w, self.offsets, self.rows, self.dtype = x, w, offsets, rows, dtype
        # The offsets are the caller's; writes to them that torch counts are found.  In a captured
        # graph they are read at each replay, which the count knows nothing of, and torch counts
        # none for inference tensors, which are copied.
        self.version = None
        if offsets is not None:
            if offsets.is_inference():
                self.offsets = offsets.clone()
            elif not _b.capturing(offsets):
                self.version = offsets._version

    def same_offsets(self) -> bool:
        return self.version is None or self.version == self.offsets._version

    def __reduce__(self):
        if not self.same_offsets():
            _refuse("MXLinearSaved: its offsets were written to since the forward pass")
        return MXLinearSaved, (self.x, self.w, self.offsets, self.rows, self.dtype)


def mx_linear_forward(x: torch.Tensor, w: torch.Tensor, stream=None):
    """y = Q(x) Q(w)^T of x [rows, depth] and w [cols, depth], and what the backward needs."""
    if stream is not None or _b.elsewhere(x):
        return _b.on_stream(mx_linear_forward, (x, w), stream)
    if (x.dim() != 2 or w.dim() != 2 or x.shape[1] != w.shape[1] or x.dtype != w.dtype
            or x.device != w.device or w.shape[0] == 0):
        _refuse("mx_linear_forward: x [rows, depth] and w [cols, depth] of one type are wanted")
    xr, xc = mx_quantize_both(x)
    wr, wc = mx_quantize_both(w)
    return mx_product(xr, wr, x.dtype), MXLinearSaved(xc, wc, None, x.shape[0], x.dtype)


def mx_linear_backward(dy: torch.Tensor, saved: MXLinearSaved, stream=None):
    """dx = Q(dy) Q(w^T)^T and dw = Q(dy^T) Q(x^T)^T, blocks along the summed dimension."""
    if stream is not None or _b.elsewhere(dy):
        return _b.on_stream(mx_linear_backward, (dy, saved), stream)
    if (saved.offsets is not None or dy.dim() != 2 or dy.dtype != saved.dtype
            or dy.shape != (saved.rows, saved.w.cols) or dy.device != saved.x.device):
        _refuse("mx_linear_backward: dy [rows, cols] of the forward's type is wanted")
    if saved.rows == 0:
        return (dy.new_zeros(0, saved.x.lead[0]),
                dy.new_zeros(dy.shape[1], saved.x.lead[0]))
    dr, dc = mx_quantize_both(dy)
    return mx_product(dr, saved.w, dy.dtype), mx_product(dc, saved.x, dy.dtype)


def _quantize_groups(x, offsets, experts):
    r, stride = _rows(x)
    rows, cols = x.shape
    L = _b.lib()
    a = _empty((rows,), cols, x)
    b = _empty((cols,), rows, x, int(L.ec_mx_padded_groups(rows, experts)))
    if rows:
        at, bt = a.home.data_ptr(), b.home.data_ptr()
        _b.check(L.ec_mx_quantize_groups(r.data_ptr(), TYPES[x.dtype], rows, cols, stride,
                                         offsets.data_ptr(), experts, at, at + a._split, bt,
                                         bt + b._split, _b.current_stream(x)),
                 "ec_mx_quantize_groups")
    return a, b


def _experts_product(a, b, offsets, dtype):
    experts, cols = b.lead
    rows = a.lead[0]
    y = a.home.new_empty((rows, cols), dtype=dtype)
    _b.check(_b.lib().ec_mx_product_experts(
        *a.pointers(), rows, *b.pointers(), cols,
        a.padded, offsets.data_ptr(), experts, y.data_ptr(), TYPES[dtype],
        _b.current_stream(y)), "ec_mx_product_experts")
    return y


def mx_experts_forward(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, stream=None):
    """The training forward of mx_experts_linear from weights w [experts, cols, depth] of x's type;
    the blocks of the saved columns begin anew at every expert's first row.  The backward pass reads
    the same offsets: they have to keep their values until then."""
    if stream is not None or _b.elsewhere(x):
        return _b.on_stream(mx_experts_forward, (x, w, offsets), stream)
    _type(x, "mx_experts_forward")
    if (x.dim() != 2 or w.dim() != 3 or x.shape[1] != w.shape[2] or x.dtype != w.dtype
            or x.device != w.device or 0 in w.shape):
        _refuse("mx_experts_forward: x [rows, depth] and w [experts, cols, depth] of one type are wanted")
    _offsets(offsets, w.shape[0], x.device, "mx_experts_forward")
    xr, xc = _quantize_groups(x, offsets, w.shape[0])
    wr, wc = mx_quantize_both(w)
    return (_experts_product(xr, wr, offsets, x.dtype),
            MXLinearSaved(xc, wc, offsets, x.shape[0], x.dtype))


def mx_experts_backward(dy: torch.Tensor, saved: MXLinearSaved, stream=None):
    """dx [rows, depth] and dw [experts, cols, depth]; rows of no expert give zeros and take no
    part, an expert without rows gets zeros."""
    if stream is not None or _b.elsewhere(dy):
        return _b.on_stream(mx_experts_backward, (dy, saved), stream)
    if (saved.offsets is None or dy.dim() != 2 or dy.dtype != saved.dtype
            or dy.shape != (saved.rows, saved.w.cols) or dy.device != saved.x.device):
        _refuse("mx_experts_backward: dy [rows, cols] of the forward's type is wanted")
    if not saved.same_offsets():
        _refuse("mx_experts_backward: the offsets were written to since the forward pass")
    experts, depth = saved.w.lead
    cols = saved.w.cols
    dr, dc = _quantize_groups(dy, saved.offsets, experts)
    dx = _experts_product(dr, saved.w, saved.offsets, dy.dtype)
    dw = torch.empty((experts, cols, depth), dtype=dy.dtype, device=dy.device)
    _b.check(_b.lib().ec_mx_product_tokens(
        *dc.pointers(), cols, *saved.x.pointers(), depth, saved.rows,
        saved.offsets.data_ptr(), experts,
        dw.data_ptr(), TYPES[dy.dtype], _b.current_stream(dy)), "ec_mx_product_tokens")
    return dx, dw
