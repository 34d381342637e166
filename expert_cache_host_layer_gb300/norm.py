"""The residual's addition and the root-mean-square norm of the sum, as torch calls.

    norm = RMSNorm(hidden, weight, eps=1e-6)              # once
    norm.apply(x, out)                                    # out = x w / sqrt(mean x^2 + eps)
    norm.apply(x, out, delta=y, total=x)                  # x += y; out = the norm of the sum

x, delta, total and out are [rows, hidden] tensors (rows may lie apart: views of
a wider tensor are fine), bf16 or float32, each its own; total has x's type.
With a float8_e4m3fn out the norm is given as codes and float32 scales
[rows, RMSNorm.num_scales], one to each ``group`` channels (0: to each row).
The caller owns every tensor; work is enqueued on ``stream`` (default: torch's
current stream of the tensors' device), and tensors of a call with ``stream``
are recorded on it.  include/ft.h (ft_add_norm) has the formulas and what may
overlap.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import FT_BF16, FT_F32, FT_FP8E4M3, _check, ft_norm, library

_add_norm = library().ft_add_norm
_pack = struct.Struct("@qPqPqPqPqPiii0q").pack  # ft_norm_args (a fourth of what 15 arguments cost through ctypes)
_DTYPES = {torch.float32: FT_F32, torch.bfloat16: FT_BF16}
_OUT = {**_DTYPES, torch.float8_e4m3fn: FT_FP8E4M3}
_device = getattr(torch._C, "_cuda_getDevice", None)  # torch.cuda.current_device, once CUDA is initialised


class RMSNorm:
    """weight: a contiguous bf16 or float32 [hidden] tensor, or None for ones.  The memory that it has now is kept, and read by
    the calls: values written in place count, ``weight.data = other`` does not reach the norm."""

    def __init__(self, hidden: int, weight: torch.Tensor | None = None, eps: float = 1e-6, group: int = 0):
        if weight is not None:
            if weight.shape != (hidden,) or weight.dtype not in _DTYPES or not weight.is_contiguous() or not weight.is_cuda:
                raise ValueError("weight is a contiguous bf16 or float32 [hidden] tensor in a GPU's memory")
            weight = weight.detach()  # (the same memory, whatever becomes of the caller's tensor)
        self.hidden, self.weight, self.eps, self.group = hidden, weight, float(eps), group
        self.num_scales = -(-hidden // group) if group else 1
        self.index = None if weight is None else weight.get_device()
        self.c = ft_norm(None if weight is None else weight.data_ptr(), FT_F32 if weight is None else _DTYPES[weight.dtype],
                         hidden, self.eps, group)
        self.address = ctypes.addressof(self.c)

    def apply(self, x: torch.Tensor, out: torch.Tensor, delta: torch.Tensor | None = None,
              total: torch.Tensor | None = None, scales: torch.Tensor | None = None,
              stream: torch.cuda.Stream | None = None):
        # (called several times a layer: each tensor's attributes are asked for once)
        index, shape, xt, ot = x.get_device(), x.shape, _DTYPES.get(x.dtype), _OUT.get(out.dtype)
        if index < 0 or (index != self.index and self.index is not None):
            raise ValueError("x is in the weight's GPU's memory")
        if len(shape) != 2 or shape[1] != self.hidden or xt is None:
            raise ValueError(f"x is a bf16 or float32 [rows, {self.hidden}] tensor")
        if ot is None or out.shape != shape or out.get_device() != index:
            raise ValueError("out is a bf16, float32 or float8_e4m3fn tensor of x's shape and device")
        (xs, x1), (os, o1) = x.stride(), out.stride()
        ds = ts = dp = tp = sp = dt = 0
        d1 = t1 = 1
        if delta is not None:
            dt = _DTYPES.get(delta.dtype)
            if dt is None or delta.shape != shape or delta.get_device() != index:
                raise ValueError("delta is a bf16 or float32 tensor of x's shape and device")
            dp, (ds, d1) = delta.data_ptr(), delta.stride()
        if total is not None:
            if delta is None:
                raise ValueError("total goes with delta")
            if total.dtype != x.dtype or total.shape != shape or total.get_device() != index:
                raise ValueError("total is a tensor of x's type, shape and device")
            tp, (ts, t1) = total.data_ptr(), total.stride()
        if (x1 != 1 or o1 != 1 or d1 != 1 or t1 != 1) and x.numel():
            raise ValueError("rows are contiguous")
        if ot == FT_FP8E4M3:
            if (scales is None or scales.dtype != torch.float32 or scales.shape != (shape[0], self.num_scales) or
                    not scales.is_contiguous() or scales.get_device() != index):
                raise ValueError("scales go with a float8 out; scales is a contiguous float32 [rows, num_scales] tensor of x's device")
            sp = scales.data_ptr()
        elif scales is not None:
            raise ValueError("scales go with a float8 out, and only with it")
        # (a Stream object of the current stream takes 2 us to make)
        s = stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(index)
        args = _pack(shape[0], x.data_ptr(), xs, dp, ds, tp, ts, out.data_ptr(), os, sp, xt, dt, ot)
        if _device() == index:
            st = _add_norm(self.address, args, s)
        else:
            with torch.cuda.device(index):
                st = _add_norm(self.address, args, s)
        if st:
            _check(st, "ft_add_norm")
        if stream is not None:
            for t in (x, out, delta, total, scales, self.weight):
                if t is not None:
                    t.record_stream(stream)
