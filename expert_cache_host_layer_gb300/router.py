"""How tokens choose their experts, as torch calls.

    router = Router(256, 8, score="sigmoid", bias=bias, groups=8, top_groups=4, group_top=2, scale=2.5)
    cache.set_router(router)              # an ExpertCache's routing by this rule
    router.route(logits, topk_idx, topk_w)   # or the choice alone, for experts elsewhere

Scores are the softmax or the sigmoid of the logits; the choice falls on the
largest scores plus ``bias``, in the best groups of experts if there are groups;
the gates are the picks' scores without the bias, renormalised over the picks or
not, times ``scale`` (include/ft.h, ft_router, has all of it).
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import FT_BF16, FT_F32, FT_SCORE_SIGMOID, FT_SCORE_SOFTMAX, _check, ft_router, library

_route = library().ft_route
_pack = struct.Struct("@PqPPiiii0q").pack  # ft_route_args
_SCORES = {"softmax": FT_SCORE_SOFTMAX, "sigmoid": FT_SCORE_SIGMOID}
_DTYPES = {torch.float32: FT_F32, torch.bfloat16: FT_BF16}
_device = getattr(torch._C, "_cuda_getDevice", None)  # torch.cuda.current_device, once CUDA is initialised


class Router:
    """bias: a contiguous float32 [experts] tensor, or [layers, experts] for a cache whose layers have their own.  The memory
    that it has now is kept, and read by the calls: values written in place between them count, ``bias.data = other`` does
    not reach the rule."""

    def __init__(self, num_experts: int, top_k: int, score: str = "softmax", bias: torch.Tensor | None = None, groups: int = 1,
                 top_groups: int = 1, group_top: int = 1, renormalise: bool = True, scale: float = 1.0):
        if score not in _SCORES:
            raise ValueError(f"score is softmax or sigmoid, not {score}")
        if bias is not None:
            if (bias.dtype != torch.float32 or bias.dim() not in (1, 2) or bias.shape[-1] != num_experts or
                    not bias.is_contiguous() or not bias.is_cuda):
                raise ValueError("bias is a contiguous float32 [experts] or [layers, experts] tensor in a GPU's memory")
            bias = bias.detach()  # (the same memory, whatever becomes of the caller's tensor)
        self.num_experts, self.top_k, self.bias = num_experts, top_k, bias
        self.index = None if bias is None else bias.get_device()
        self.c = ft_router(_SCORES[score], groups, top_groups, group_top, int(bool(renormalise)), float(scale),
                           None if bias is None else bias.data_ptr(),
                           num_experts if bias is not None and bias.dim() == 2 else 0)
        self.address = ctypes.addressof(self.c)

    def route(self, logits: torch.Tensor, topk_idx: torch.Tensor, topk_w: torch.Tensor,
              stream: torch.cuda.Stream | None = None):
        """logits: float32 or bf16 [tokens, experts] (rows may lie apart); topk_idx int32 and topk_w float32 [tokens, top_k]
        receive experts in selection order and gates.  Work is enqueued on ``stream`` (default: torch's current stream of the
        logits' device); tensors of a call with ``stream`` are recorded on it."""
        index = logits.get_device()
        if index < 0 or (self.index is not None and index != self.index):
            raise ValueError("the logits are in the bias's GPU's memory")
        if self.bias is not None and self.bias.dim() != 1:
            raise ValueError("a bias for each layer is for a cache's routing")
        dt = _DTYPES.get(logits.dtype)
        if dt is None or logits.dim() != 2 or logits.shape[1] != self.num_experts:
            raise ValueError(f"logits is a float32 or bf16 [tokens, {self.num_experts}] tensor")
        T = logits.shape[0]
        shape = (T, self.top_k)
        for t, want in ((topk_idx, torch.int32), (topk_w, torch.float32)):
            if t.dtype != want or t.shape != shape or not t.is_contiguous() or t.get_device() != index:
                raise ValueError("topk_idx and topk_w are contiguous int32 and float32 [tokens, top_k] tensors of the logits' device")
        stride, one = logits.stride()
        if one != 1 and self.num_experts > 1 and T:
            raise ValueError("rows are contiguous")
        s = stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(index)
        args = _pack(logits.data_ptr(), stride, topk_idx.data_ptr(), topk_w.data_ptr(), dt, T, self.num_experts, self.top_k)
        if _device() == index:
            st = _route(self.address, args, s)
        else:
            with torch.cuda.device(index):
                st = _route(self.address, args, s)
        if st:
            _check(st, "ft_route")
        if stream is not None:
            for t in (logits, topk_idx, topk_w, self.bias):
                if t is not None:
                    t.record_stream(stream)
