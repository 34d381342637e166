"""One layer's paged key/value cache as torch tensors, and the calls on it.

    pages = KVPages(k, v, k_scale, v_scale)          # once, for the layer's life
    batch = KVBatch(q_start, kv_len, block_table, num_tokens, max_q_len)   # once a step, for every layer
    pages.append(batch, k_new, v_new)                # store the new tokens
    pages.append(batch, k_new, v_new, rotary=rotary, q=q, q_out=q)   # or: with rotary positions (rotary.py)
    pages.attend(batch, q, out)                      # softmax(q k^T / sqrt(D)) v over their sequences
    pages.read(batch, kv_start, k_out, v_out)        # whole sequences back in bf16

The caller owns every tensor.  ``KVPages.empty`` allocates a layer's pages.
Work is enqueued on ``stream`` (default: torch's current stream of the cache's
device).  ``attend`` needs a workspace that no other call uses at the same time:
calls outside of a capture share one per stream, which grows to the largest;
calls captured by ``torch.cuda.graph`` share one that belongs to the graph, so
that it may be replayed on any stream, in any order, beside anything but itself.
Tensors of a call with ``stream`` are recorded on it, so that dropping them right
after is fine; waiting for what wrote them, and before what reads its results, is
the caller's.
Whoever captures by other means makes one (``new_workspace``), keeps it as long
as the graph, and passes it to each captured ``attend``.  Make one call before
capturing: the first of a kind loads its kernels.

Device-side errors are reported by ``check`` (see ft_kv_status in include/ft.h,
which also gives the layout and the sequences' description).
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import (FT_KV_BF16, FT_KV_FP8E4M3, FT_KV_WORKSPACE_ZERO, _check, ft_kv_attend_workspace, ft_kv_batch,
               ft_kv_pages, ft_kv_status, library)
from .rotary import Rotary

# The calls are made once per layer and step, so they go to the library
# directly: at a decode step's sizes the binding's own functions, a device guard
# and a stream object would cost as much as the GPU's work.
_lib = library()
_append, _attend, _read = _lib.ft_kv_append, _lib.ft_kv_attend, _lib.ft_kv_read
_append_rotary = _lib.ft_kv_append_rotary
_BF16 = torch.bfloat16
_NO_QUERIES = (0, 0, 0, 0, 0, 0)
_append_args = struct.Struct("@PqqPqqPqqPqqi0q").pack  # ft_append_args
_workspaces: dict = {}  # (device index, stream) -> uint8 tensor
_outgrown: list = []    # the smaller ones before them: three of a stream at most (sizes go by head_dim and the kernels)
_captured: dict = {}    # (device index, stream) -> (number, uint8 tensor) of the last capture that the stream was part of

# what torch.cuda.current_device and is_current_stream_capturing ask, once CUDA is initialised
_device, _capturing = (getattr(torch._C, n, None) for n in ("_cuda_getDevice", "_cuda_isCurrentStreamCapturing"))


def _need(ok, text, *args):
    if not ok:
        raise ValueError(text % args if args else text)


class KVBatch:
    """One step's sequences: int32 device tensors q_start [S + 1], kv_len [S]
    and block_table [S, pages], and the host's num_tokens and max_q_len.  Later
    values are written into the tensors; ``kv_len.data = other`` is not one."""

    def __init__(self, q_start: torch.Tensor, kv_len: torch.Tensor, block_table: torch.Tensor, num_tokens: int,
                 max_q_len: int):
        S = kv_len.shape[0]
        _need(q_start.dtype == kv_len.dtype == block_table.dtype == torch.int32,
              "q_start, kv_len and block_table are int32 tensors")
        _need(q_start.shape == (S + 1,) and kv_len.dim() == 1 and block_table.dim() == 2 and block_table.shape[0] == S,
              "shapes: q_start [S + 1], kv_len [S], block_table [S, pages]")
        _need(q_start.is_contiguous() and kv_len.is_contiguous(), "q_start and kv_len are contiguous")
        _need((block_table.stride(1) == 1 or block_table.shape[1] <= 1) and
              (S <= 1 or block_table.stride(0) >= block_table.shape[1]), "block_table's rows are contiguous")
        _need(q_start.device == kv_len.device == block_table.device, "one device")
        self.q_start, self.kv_len, self.block_table = q_start, kv_len, block_table  # keeps them alive
        self.num_seqs, self.num_tokens, self.max_q_len = S, int(num_tokens), int(max_q_len)
        self.device = kv_len.device
        self.index = kv_len.get_device()
        stride = block_table.stride(0) if S > 1 else block_table.shape[1]
        self.c = ft_kv_batch(q_start.data_ptr(), kv_len.data_ptr(), block_table.data_ptr(), stride, S, self.num_tokens,
                             self.max_q_len)
        self.address = ctypes.addressof(self.c)


class KVPages:
    """One layer's cache: k, v [pages, kv_heads, page_tokens, head_dim], bf16 or
    float8_e4m3fn; for the latter k_scale, v_scale [pages, kv_heads,
    page_tokens] uint8, the exponent bytes of the scales.  The memory that the
    tensors have now is the cache (``k.data = other`` does not reach it)."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor | None = None,
                 v_scale: torch.Tensor | None = None):
        _need(k.dim() == 4 and k.shape == v.shape and k.dtype == v.dtype and k.is_contiguous() and v.is_contiguous(),
              "k and v are contiguous [pages, kv_heads, page_tokens, head_dim] tensors of one type")
        _need(k.dtype in (torch.bfloat16, torch.float8_e4m3fn), "the cache is bf16 or float8_e4m3fn, not %s", k.dtype)
        fp8 = k.dtype == torch.float8_e4m3fn
        _need(fp8 == (k_scale is not None) == (v_scale is not None), "scales go with a float8 cache, and only with it")
        if fp8:
            for t in (k_scale, v_scale):
                _need(t.dtype == torch.uint8 and t.shape == k.shape[:3] and t.is_contiguous() and t.device == k.device,
                      "scales are contiguous uint8 [pages, kv_heads, page_tokens]")
        _need(k.is_cuda and v.device == k.device, "the pages are in one GPU's memory")
        # (the same memory, whatever becomes of the caller's tensors)
        self.k, self.v, self.k_scale, self.v_scale = (None if t is None else t.detach() for t in (k, v, k_scale, v_scale))
        self.device = k.device
        self.num_pages, self.num_kv_heads, self.page_tokens, self.head_dim = k.shape
        self.scale = self.head_dim ** -0.5  # of the scores, unless a call gives its own
        self.c = ft_kv_pages(k.data_ptr(), v.data_ptr(), k_scale.data_ptr() if fp8 else None,
                             v_scale.data_ptr() if fp8 else None, self.num_pages, self.num_kv_heads, self.head_dim,
                             self.page_tokens, FT_KV_FP8E4M3 if fp8 else FT_KV_BF16)
        self.address = ctypes.addressof(self.c)
        self.index = k.get_device()
        self._needs: dict = {}  # (q_heads, max_q_len) -> workspace bytes

    @classmethod
    def empty(cls, num_pages, num_kv_heads, page_tokens, head_dim, kv_dtype=FT_KV_BF16, device="cuda:0"):
        """A layer's pages, contents undefined (a page is written before it is read)."""
        shape = (num_pages, num_kv_heads, page_tokens, head_dim)
        dt = torch.float8_e4m3fn if kv_dtype == FT_KV_FP8E4M3 else torch.bfloat16
        kv = [torch.empty(shape, dtype=dt, device=device) for _ in range(2)]
        sc = [torch.empty(shape[:3], dtype=torch.uint8, device=device) for _ in range(2)] if dt != torch.bfloat16 else []
        return cls(*kv, *sc)

    # ---- the calls ---------------------------------------------------------
    def append(self, batch: KVBatch, k: torch.Tensor, v: torch.Tensor, stream: torch.cuda.Stream | None = None,
               rotary: Rotary | None = None, q: torch.Tensor | None = None, q_out: torch.Tensor | None = None):
        """Store the batch's new keys and values, bf16 [num_tokens, kv_heads, head_dim] (strided views are fine).
        With ``rotary`` the keys are stored rotated to their positions, and the queries q, bf16 [num_tokens, q_heads,
        head_dim], rotated into q_out (which may be q)."""
        heads = self.num_kv_heads
        rows = (*self._rows(batch, k, heads, "k"), *self._rows(batch, v, heads, "v"))
        if rotary is None:
            if q is not None or q_out is not None:
                raise ValueError("q and q_out go with rotary")
            self._call(_append, self.address, batch.address, *rows, self._stream(stream))
        else:
            if (q is None) != (q_out is None) or rotary.index != self.index:
                raise ValueError("q goes with q_out, and the rotary is on the cache's device")
            heads, queries = 0, _NO_QUERIES
            if q is not None:
                heads = q.shape[1] if q.dim() == 3 else 0
                queries = (*self._rows(batch, q, heads, "q"), *self._rows(batch, q_out, heads, "q_out"))
            self._call(_append_rotary, self.address, batch.address, rotary.address, _append_args(*rows, *queries, heads),
                       self._stream(stream))
        if stream is not None:
            self._record(stream, batch, k, v, q, q_out, None if rotary is None else rotary.turns)

    def attend(self, batch: KVBatch, q: torch.Tensor, out: torch.Tensor, lse: torch.Tensor | None = None,
               scale: float | None = None, causal: bool = True, window: int = 0,
               stream: torch.cuda.Stream | None = None, workspace: torch.Tensor | None = None):
        """Attention of the batch's new tokens; q, out: bf16 [num_tokens, q_heads,
        head_dim], lse: f32 [num_tokens, q_heads].  scale defaults to
        1 / sqrt(head_dim); window > 0 keeps that many last tokens, the row's own
        included.  workspace: the caller's own (see ``new_workspace``)."""
        heads = q.shape[1] if q.dim() == 3 else 0
        rows = (*self._rows(batch, q, heads, "q"), *self._rows(batch, out, heads, "out"))
        if lse is not None:
            _need(lse.dtype == torch.float32 and lse.shape == (batch.num_tokens, heads) and lse.is_contiguous() and
                  lse.get_device() == self.index, "lse is a contiguous float32 [num_tokens, q_heads] tensor")
        s = self._stream(stream)
        if workspace is None:
            ws = _workspaces.get((self.index, s))
            need = self._needs.get((heads, batch.max_q_len)) or self._need_bytes(batch, heads)
            if ws is None or ws.numel() < need or stream is not None or _device() != self.index or _capturing():
                ws = self._workspace(s, need, stream)
        else:
            ws = workspace
            _need(ws.dtype == torch.uint8 and ws.is_contiguous() and ws.get_device() == self.index,
                  "workspace is a contiguous uint8 tensor of the cache's device")
        self._call(_attend, self.address, batch.address, heads, *rows,
                   lse.data_ptr() if lse is not None else None, self.scale if scale is None else scale, causal,
                   window, ws.data_ptr(), ws.numel(), s)
        if stream is not None:
            self._record(stream, batch, q, out, lse, workspace)

    def new_workspace(self, batch: KVBatch, q_heads: int, stream: torch.cuda.Stream | None = None) -> torch.Tensor:
        """A workspace for ``attend`` of batches with this one's max_q_len, made on the stream."""
        with torch.cuda.device(self.device), torch.cuda.stream(stream):
            return torch.zeros(self._need_bytes(batch, q_heads), dtype=torch.uint8, device=self.device)

    def read(self, batch: KVBatch, kv_start: torch.Tensor, k_out: torch.Tensor, v_out: torch.Tensor,
             stream: torch.cuda.Stream | None = None):
        """Whole sequences back in bf16: token p of sequence s is row kv_start[s] + p of k_out and v_out,
        contiguous [rows, kv_heads, head_dim]."""
        _need(kv_start.dtype == torch.int32 and kv_start.shape == (batch.num_seqs + 1,) and kv_start.is_contiguous() and
              kv_start.get_device() == self.index, "kv_start is a contiguous int32 [S + 1] tensor of the cache's device")
        shape = (k_out.shape[0], self.num_kv_heads, self.head_dim)
        for t in (k_out, v_out):
            _need(t.dtype == torch.bfloat16 and t.shape == shape and t.is_contiguous() and t.get_device() == self.index,
                  "k_out and v_out are contiguous bf16 [rows, kv_heads, head_dim] tensors of the cache's device")
        _need(batch.index == self.index, "the batch and the cache are on one device")
        self._call(_read, self.address, batch.address, kv_start.data_ptr(), shape[0], k_out.data_ptr(),
                   v_out.data_ptr(), self._stream(stream))
        if stream is not None:
            self._record(stream, batch, kv_start, k_out, v_out)

    def check(self, stream: torch.cuda.Stream | None = None):
        """Wait for the stream and raise FtError if a call met device data out of range or a timeout."""
        with torch.cuda.device(self.device):
            ft_kv_status(self._stream(stream))

    # ---- helpers -------------------------------------------------------------
    def _rows(self, batch, t, heads, name):
        """Address and strides of a [num_tokens, heads, head_dim] tensor."""
        if (t.dtype != _BF16 or t.shape != (batch.num_tokens, heads, self.head_dim) or
                t.get_device() != self.index or batch.index != self.index):
            raise ValueError(f"{name} is a bf16 [num_tokens, heads, {self.head_dim}] tensor of the cache's device")
        s0, s1, s2 = t.stride()
        if s2 != 1 and t.numel():
            raise ValueError(f"{name}'s rows are contiguous")
        return t.data_ptr(), s0, s1

    def _call(self, fn, *args):
        if _device() == self.index:
            st = fn(*args)
        else:
            with torch.cuda.device(self.device):
                st = fn(*args)
        if st:
            _check(st, fn.__name__)

    def _stream(self, stream):
        # (a Stream object of the current stream takes 2 us to make)
        return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(self.index)

    def _record(self, stream, batch, *tensors):
        """Their memory is not given to others before the stream's work so far is done."""
        for t in (self.k, self.v, self.k_scale, self.v_scale, batch.q_start, batch.kv_len, batch.block_table, *tensors):
            if t is not None:
                t.record_stream(stream)

    def _need_bytes(self, batch, heads):
        key = (heads, batch.max_q_len)
        if key not in self._needs:
            with torch.cuda.device(self.device):
                self._needs[key] = max(256, ft_kv_attend_workspace(self.c, batch.c, heads))
        return self._needs[key]

    def _workspace(self, s, nbytes, stream):
        """The one of stream s, or of the capture that it is part of."""
        capture = _lib.ft_stream_capture(s)
        key = (self.index, s)
        if capture:
            of, ws = _captured.get(key, (0, None))
            if of == capture and ws.numel() >= nbytes:
                return ws
        else:
            ws = _workspaces.get(key)
            if ws is not None:
                if ws.numel() >= nbytes:
                    return ws
                _outgrown.append(ws)
        with torch.cuda.device(self.device), torch.cuda.stream(stream):  # reused in this stream's order
            ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
            ws[:FT_KV_WORKSPACE_ZERO].zero_()
        # (a capture's lies in its graph's memory, which outlives the tensor: it is let go with the stream's next capture)
        if capture:
            _captured[key] = (capture, ws)
        else:
            _workspaces[key] = ws
        return ws
