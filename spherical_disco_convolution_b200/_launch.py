"""What every call of a training operator does before it enters libdisco, kept short: these calls
take a few microseconds of GPU time on small layers, so the host's share counts."""

from __future__ import annotations

import torch

from . import disco as D

DTYPES = {torch.float32: D.DISCO_F32, torch.bfloat16: D.DISCO_BF16}


def dense(t: torch.Tensor, what: str) -> int:
    """The type code of a dense CUDA tensor; raises for any other."""
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"libdisco takes contiguous CUDA tensors: {what} is not one")
    code = DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype} of {what}; use float32 or bfloat16")
    return code


def like(t, x: torch.Tensor, shape, what: str):
    """The pointer of t, which is None or dense, of x's type and device, and of the given shape."""
    if t is None:
        return None
    if t.dtype != x.dtype:
        raise TypeError(f"libdisco takes tensors of one dtype; {what} is {t.dtype}, not {x.dtype}")
    if t.device != x.device:
        raise ValueError(f"{what} is on {t.device}, not {x.device}")
    if not t.is_contiguous():
        raise ValueError(f"libdisco takes contiguous CUDA tensors: {what} is not one")
    if t.shape != shape:
        raise ValueError(f"{what} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t.data_ptr()


def launch(x: torch.Tensor, fn, *args) -> None:
    """fn(*args, stream) with x's device current, on that device's current stream."""
    # looked up here, since a torch without CUDA has neither (and then no x comes this far)
    device, stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
    index = x.get_device()
    if index == device():
        fn(*args, stream(index))
    else:
        with torch.cuda.device(index):
            fn(*args, stream(index))
