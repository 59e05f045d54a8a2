"""What the bindings share: errors, the current stream and device, argument
checks and type codes."""
from __future__ import annotations

import contextlib

import torch

from . import _lib
from ._lib import LMHEAD_BF16, LMHEAD_F16, LMHEAD_F32, NOT_HANDLED, OK


class LmHeadError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


class NotHandled(LmHeadError):
    """The shape lies outside the kernels' contract; nothing was launched."""


def status_string(status: int) -> str:
    return _lib.load().lmhead_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status == OK:
        return
    if status == NOT_HANDLED:
        raise NotHandled(status, where)
    raise LmHeadError(status, where)


# torch's current raw HIP stream of a device index, without building a Stream
# object per call (the public route below when this build lacks it)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_handle(device, stream):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(device.index if device.index is not None else torch.cuda.current_device())
    return torch.cuda.current_stream(device).cuda_stream


_NO_SWITCH = contextlib.nullcontext()

# torch's current device index without its lazy-initialisation check (a device
# tensor is in hand wherever this is called)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _device_ctx(device):
    """The library launches on the current device: make it `device`, switching
    (and switching back) only when it is another one."""
    idx = device.index
    return _NO_SWITCH if idx is None or _current_device() == idx else torch.cuda.device(idx)


def _alloc_on(stream):
    """Where a call's outputs and workspace are allocated: the stream it runs
    on, so that the allocator's reuse of their memory is ordered with it."""
    return _NO_SWITCH if stream is None else torch.cuda.stream(stream)


def _need(cond: bool, msg: str):
    if not cond:
        raise ValueError(msg)


def _same_device(first, *tensors):
    dev = first.device
    for t in tensors:
        if t is not None and t.device != dev:  # the message only on failure: this runs on every call
            devs = {str(t.device) for t in (first, *tensors) if t is not None}
            raise ValueError(f"all tensors must be on one device, got {sorted(devs)}")


_DTYPES = {torch.float32: LMHEAD_F32, torch.bfloat16: LMHEAD_BF16, torch.float16: LMHEAD_F16}
