"""What mx.py and experts.py share: the library, and the stream a call runs on."""
from __future__ import annotations

import torch

import error_bounded_lossy_amd as _ec
from error_bounded_lossy_amd import EC_ERR_INVALID, ECError  # noqa: F401


def lib():
    return _ec._lib or _ec.lib()


def check(status: int, what: str):
    if status:
        raise ECError(status, what)


def current_stream(t: torch.Tensor) -> int:
    """The handle of torch's current stream on t's device (the raw getter: a Stream object costs
    more than a small call's launch)."""
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def elsewhere(t: torch.Tensor) -> bool:
    """Whether t lies on a GPU that is not the current one."""
    device = t.get_device()  # -1: not on a GPU
    return device >= 0 and device != torch._C._cuda_getDevice()


def capturing(t: torch.Tensor) -> bool:
    """Whether calls on t, on the current stream, are being recorded into a graph."""
    return t.get_device() >= 0 and torch._C._cuda_isCurrentStreamCapturing()


def _tensors(v):
    if isinstance(v, torch.Tensor):
        yield v
    elif hasattr(v, "__slots__"):
        for name in v.__slots__:
            yield from _tensors(getattr(v, name))


def on_stream(call, args, stream):
    """call(*args) on `stream` (None: the current one) of the first tensor's device.  Tensors from
    other streams stay allocated until the work on this one is done."""
    first = next((t for a in args for t in _tensors(a)), None)
    if first is None or not first.is_cuda:
        raise ECError(EC_ERR_INVALID, f"{call.__name__}: tensors on the GPU are wanted")
    if stream is not None and (not hasattr(stream, "stream_id")
                               or getattr(stream, "device", None) != first.device):
        raise ECError(EC_ERR_INVALID, f"{call.__name__}: a stream of the tensors' device is wanted")
    with torch.cuda.device(first.device), torch.cuda.stream(stream):
        try:
            return call(*args)
        finally:  # a call that failed may have enqueued a part of its work
            if stream is not None:
                for a in args:
                    for t in _tensors(a):
                        t.record_stream(stream)
