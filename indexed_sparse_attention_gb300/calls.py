"""A library call on a tensor's device and stream."""
from __future__ import annotations

import torch

from . import _check, lib

#: The handle of a device's current stream; torch.cuda.current_stream builds a Stream object around it (2 us a call).
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
#: The current device's number, without torch.cuda.current_device's look at whether CUDA is up (a tensor is there).
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _call(name: str, device, stream, *args):
    """One library call with the tensors' device as the current one (the library
    launches there), on `stream` or that device's current stream."""
    if device.type != "cuda":
        raise ValueError(f"{name}: the tensors are on {device}, not on a GPU")
    _call_at(name, device.index, stream, *args)


def _call_at(name: str, index: int, stream, *args):
    """_call for the device that Tensor.get_device gives (-1: not a GPU), which costs half of Tensor.device."""
    if index < 0:
        raise ValueError(f"{name}: the tensors are not on a GPU")
    fn = getattr(lib(), name)
    if stream is None:
        stream = _current_stream(index)
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    if index == _current_device():
        status = fn(*args, int(stream))
    else:
        with torch.cuda.device(index):
            status = fn(*args, int(stream))
    if status:
        _check(name, status)
