"""Calls into libnvfp4.so on a tensor's device and current stream, with little Python between.

A decoding step makes many calls of a few microseconds each; the stream lookup through ``torch.cuda.current_stream``
alone takes 2.0 us on a Grace core, the raw lookup below 0.1 us.
"""
from __future__ import annotations

import torch

from . import _lib

_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_functions: dict = {}


def call(name: str, device: torch.device, *args) -> None:
    """Runs the C function `name` with args and `device`'s current stream, on that device; raises NVFP4Error."""
    fn = _functions.get(name)
    if fn is None:
        fn = _functions[name] = getattr(_lib.load(), name)
    index = device.index
    if index == _current_device():
        rc = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, _raw_stream(index))
    if rc:
        _lib.check(rc, name)
