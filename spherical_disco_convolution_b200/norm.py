"""Layer norm of a field over its channels, on the libdisco C ABI.

The norm between two DISCO layers: the field is (B, C, nlat, nlon), as the convolution takes and
gives it, and every grid point is normalised over its C channels.  Everything runs in libdisco's
CUDA kernels (there is no CPU path); PyTorch supplies memory, streams and autograd bookkeeping.
fp32 or bf16, all tensors of a call in one type; statistics and sums over channels are fp32, sums over
points go on in fp64 after some tiles.
"""

from __future__ import annotations

import functools
import math

import torch

from . import disco as D
from ._launch import dense, launch, like

_workspace_size = functools.lru_cache(maxsize=1024)(D.disco_norm_workspace_size)


def _sizes(x):
    shape = x.shape
    if len(shape) < 2 or x.numel() == 0:
        raise ValueError(f"x has shape {tuple(shape)}, expected (B, C, *points) without an empty axis")
    return shape[0], shape[1], math.prod(shape[2:])


def layer_norm(x: torch.Tensor, gain=None, bias=None, eps: float = 1e-5):
    """(out, stats) of x (B, C, *points): out = gain * (x - mean) * r + bias with mean and r =
    1 / sqrt(var + eps) over the channels of each point; stats (2, B, *points) holds mean and r in
    fp32, which layer_norm_backward takes.  gain and bias are (C,), in x's type, or None.  out has
    gradients where autograd records and x, gain or bias asks for them; stats has none."""
    if torch.is_grad_enabled() and (x.requires_grad or (gain is not None and gain.requires_grad)
                                    or (bias is not None and bias.requires_grad)):
        return _LayerNormFn.apply(x, gain, bias, eps)
    return _forward(x, gain, bias, eps)


def _forward(x, gain, bias, eps):
    code = dense(x, "x")
    B, C, n = _sizes(x)
    gain = like(gain, x, (C,), "gain")
    bias = like(bias, x, (C,), "bias")
    out = torch.empty_like(x)
    stats = x.new_empty((2, B, *x.shape[2:]), dtype=torch.float32)
    launch(x, D.disco_norm, B, C, n, code, x.data_ptr(), gain, bias, eps, out.data_ptr(), stats.data_ptr())
    return out, stats


def layer_norm_backward(dout: torch.Tensor, x: torch.Tensor, stats: torch.Tensor, gain=None, need_input: bool = True,
                        need_gain: bool = True, need_bias: bool = True):
    """(dx, dgain, dbias) of layer_norm from the field it took and the stats it returned; None for
    each one not needed."""
    code = dense(x, "x")
    B, C, n = _sizes(x)
    dout = like(dout, x, x.shape, "dout")
    gain = like(gain, x, (C,), "gain")
    if stats.dtype != torch.float32 or not stats.is_contiguous() or stats.device != x.device or \
            stats.shape != (2, B, *x.shape[2:]):
        raise ValueError("stats is the contiguous fp32 tensor (2, B, *points) that layer_norm returned")
    if not (need_input or need_gain or need_bias):
        return None, None, None
    dx = torch.empty_like(x) if need_input else None
    dgain = x.new_empty(C) if need_gain else None
    dbias = x.new_empty(C) if need_bias else None
    ws, nb = None, 0
    if need_gain or need_bias:
        nb = _workspace_size(B, C, n, code)
        ws = x.new_empty(nb, dtype=torch.uint8)
    launch(x, D.disco_norm_backward, B, C, n, code, dout, x.data_ptr(), stats.data_ptr(), gain,
           None if dx is None else dx.data_ptr(), None if dgain is None else dgain.data_ptr(),
           None if dbias is None else dbias.data_ptr(), None if ws is None else ws.data_ptr(), nb)
    return dx, dgain, dbias


class _LayerNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gain, bias, eps):
        out, stats = _forward(x, gain, bias, eps)
        ctx.save_for_backward(x, stats, gain)
        ctx.mark_non_differentiable(stats)
        return out, stats

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout, _):
        x, stats, gain = ctx.saved_tensors
        need = ctx.needs_input_grad
        return (*layer_norm_backward(dout.contiguous(), x, stats, gain, need[0], need[1], need[2]), None)


class LayerNormS2(torch.nn.Module):
    """Layer norm over the channels of every grid point of a (B, C, nlat, nlon) field.

    On a grid split over ranks each rank norms the points it holds; the gradients of weight and
    bias are then that rank's share of the sum over points, to be added over the ranks."""

    def __init__(self, channels, eps=1e-5, affine=True, bias=True, device=None, dtype=torch.float32):
        super().__init__()
        if channels < 1:
            raise ValueError(f"channels={channels} must be positive")
        if dtype not in (torch.float32, torch.bfloat16):
            raise TypeError(f"unsupported dtype {dtype}; use float32 or bfloat16")
        self.channels, self.eps = channels, float(eps)
        self.weight = torch.nn.Parameter(torch.ones(channels, device=device, dtype=dtype)) if affine else None
        self.bias = torch.nn.Parameter(torch.zeros(channels, device=device, dtype=dtype)) if affine and bias else None

    def forward(self, x):
        if x.dim() < 2 or x.shape[1] != self.channels:
            raise ValueError(f"x has shape {tuple(x.shape)}, expected (B, {self.channels}, *points)")
        gain, bias = (None if p is None else p.contiguous() for p in (self.weight, self.bias))
        return _LayerNormFn.apply(x.contiguous(), gain, bias, self.eps)[0]
