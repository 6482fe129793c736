"""Argument checks shared by the rope and cache bindings.

A decoding step is a handful of microseconds on the GPU, so the checks take
the shortest way through a good call (about 0.3 us a tensor) and only a bad one
goes through the full checks of ``attention``, which name what is wrong.
"""
from __future__ import annotations

import torch

from .attention import _check, _same_device


def raw_stream(index: int) -> int:
    """The current stream of a device as an integer (torch.cuda.current_stream(...).cuda_stream
    without the object).  The name is looked up at the call: a torch without CUDA has none."""
    return torch._C._cuda_getCurrentRawStream(index)


def want(t, name: str, shape: tuple, dtype, first: torch.Tensor) -> None:
    """Raise unless t is a contiguous tensor of this shape and dtype on the
    (CUDA) device of `first`."""
    try:
        if (t.dtype == dtype and t.shape == shape and t.is_cuda and t.get_device() == first.get_device()
                and t.is_contiguous()):
            return
    except AttributeError:
        pass
    _check(t, name, shape, dtype)
    _same_device(first, t)


def on_device(index: int):
    """None when `index` is the current CUDA device, else a guard that makes it so."""
    return None if torch._C._cuda_getDevice() == index else torch.cuda.device(index)
