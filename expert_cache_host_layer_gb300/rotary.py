"""Rotary positions as torch calls.

    rotary = Rotary(head_dim, base=1e6)                       # once, for the model
    rotary.rotate(positions, x, out)                          # queries or keys at given positions
    pages.append(batch, k, v, rotary=rotary, q=q, q_out=q)    # a batch's keys into the cache, and its queries

Pair i of a head's first ``rot_dim`` values turns by position * frequency_i
(``frequencies``); pairs are (i, i + rot_dim / 2), or (2i, 2i + 1) if
``interleaved``.  The angles are exact at any position (include/ft.h, ft_rotary,
says how), so a long context costs no accuracy.  A negative position turns
back: rotating keys by the difference moves them to another place.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from . import _check, ft_rotary, library

_rotate = library().ft_rotate
_pack = struct.Struct("@PPqqPqqiii0q").pack  # ft_rotate_args
_device = getattr(torch._C, "_cuda_getDevice", None)  # torch.cuda.current_device, once CUDA is initialised


def frequencies(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0, original_length: int = 0,
                beta_fast: float = 32.0, beta_slow: float = 1.0) -> list:
    """Radians that a position turns each of the rot_dim / 2 pairs by: base ** (-2 i / rot_dim), and for contexts
    ``factor`` times the original_length that a model was first trained on

    * "linear": every frequency divided by factor (positions interpolated);
    * "yarn": pairs that turn beta_fast times or more over original_length as they are, those that turn beta_slow times or
      less divided by factor, in between a mix that is linear in the pair's index."""
    if not base > 0.0:
        raise ValueError("base is positive")
    freq = [base ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)]
    if scaling == "none":
        return freq
    if not factor >= 1.0:
        raise ValueError("factor is at least 1")
    if scaling == "linear":
        return [f / factor for f in freq]
    if scaling != "yarn":
        raise ValueError(f"scaling is none, linear or yarn, not {scaling}")
    if original_length < 1 or not base > 1.0 or not beta_fast > beta_slow > 0.0:
        raise ValueError("yarn needs original_length, a base above 1 and beta_fast above beta_slow")

    def index(turns):  # of the pair that turns so often over original_length
        return rot_dim * math.log(original_length / (2.0 * math.pi * turns)) / (2.0 * math.log(base))

    first = max(0, math.floor(index(beta_fast)))
    last = min(rot_dim - 1, math.ceil(index(beta_slow)))
    out = []
    for i, f in enumerate(freq):
        slow = min(1.0, max(0.0, (i - first) / max(last - first, 0.001)))
        out.append(f * (1.0 - slow) + f / factor * slow)
    return out


class Rotary:
    """scaling, factor, ...: of ``frequencies``, which may be given as a list instead.  ``scale`` multiplies the rotated
    values; by default 1, and 0.1 ln(factor) + 1 for "yarn"."""

    def __init__(self, rot_dim: int, base: float = 10000.0, interleaved: bool = False, scaling: str = "none",
                 factor: float = 1.0, original_length: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0,
                 scale: float | None = None, frequencies: list | None = None, device="cuda:0"):
        if rot_dim < 16 or rot_dim % 16:
            raise ValueError("rot_dim is a multiple of 16")
        if frequencies is None:
            frequencies = _frequencies(rot_dim, base, scaling, factor, original_length, beta_fast, beta_slow)
        if len(frequencies) != rot_dim // 2 or not all(math.isfinite(f) for f in frequencies):
            raise ValueError("frequencies are rot_dim / 2 finite numbers")
        if scale is None:
            scale = 0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0
        self.rot_dim, self.interleaved, self.scale = rot_dim, bool(interleaved), float(scale)
        self.frequencies = [float(f) for f in frequencies]
        turns = [int(math.ldexp(f / (2.0 * math.pi) % 1.0, 64)) % (1 << 64) for f in self.frequencies]
        self.turns = torch.tensor([t - (1 << 64) if t >> 63 else t for t in turns], dtype=torch.int64, device=device)
        if not self.turns.is_cuda:
            raise ValueError("the rotary is in a GPU's memory")
        self.index = self.turns.get_device()
        self.c = ft_rotary(self.turns.data_ptr(), rot_dim, int(self.interleaved), self.scale)
        self.address = ctypes.addressof(self.c)

    def rotate(self, positions: torch.Tensor, x: torch.Tensor, out: torch.Tensor, stream: torch.cuda.Stream | None = None):
        """out = x rotated; bf16 [tokens, heads, head_dim] (views of a projection's output are fine; out may be x),
        positions int32 [tokens].  Work is enqueued on ``stream`` (default: torch's current stream of the device)."""
        index = self.index
        if x.dtype != torch.bfloat16 or x.dim() != 3 or x.get_device() != index:
            raise ValueError("x is a bf16 [tokens, heads, head_dim] tensor of the rotary's device")
        if out.dtype != torch.bfloat16 or out.shape != x.shape or out.get_device() != index:
            raise ValueError("out is a bf16 tensor of x's shape and device")
        T, heads, dim = x.shape
        if (positions.dtype != torch.int32 or positions.shape != (T,) or positions.get_device() != index or
                not positions.is_contiguous()):
            raise ValueError("positions is a contiguous int32 [tokens] tensor of the rotary's device")
        xt, xh, x1 = x.stride()
        ot, oh, o1 = out.stride()
        if (x1 != 1 or o1 != 1) and x.numel():
            raise ValueError("rows are contiguous")
        s = stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(index)
        args = _pack(positions.data_ptr(), x.data_ptr(), xt, xh, out.data_ptr(), ot, oh, T, heads, dim)
        if _device() == index:
            st = _rotate(self.address, args, s)
        else:
            with torch.cuda.device(index):
                st = _rotate(self.address, args, s)
        if st:
            _check(st, "ft_rotate")
        if stream is not None:
            for t in (positions, x, out, self.turns):
                t.record_stream(stream)


_frequencies = frequencies
