"""Paged cache: the compressed keys and values of a serving batch in pages of one buffer.

Argument marshalling for the ``kv1b_paged_*`` calls of ``include/kv1b.h``.  Lengths, page tables and
positions are device tensors that the kernels read, so a decode step (append, attend) can be captured
in a CUDA graph once and replayed while they change in place.
"""
from __future__ import annotations

import ctypes

import torch

from . import HEAD_DIM, Kv1bError, _check, _dtype_code, lib

BLOCK_TOKENS = 32
BLOCK_BYTES = 3200
ROPE_MAX_AXES = 3


class PagedDesc(ctypes.Structure):
    """Mirror of ``kv1b_paged_t``."""
    _fields_ = [("pages", ctypes.c_void_p), ("signs", ctypes.c_void_p), ("d_status", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32), ("page_tokens", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class RopeDesc(ctypes.Structure):
    """Mirror of ``kv1b_rope_t``."""
    _fields_ = [("cos_sin", ctypes.c_void_p), ("num_positions", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("axes", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("sections", ctypes.c_int32 * ROPE_MAX_AXES),
                ("reserved", ctypes.c_int32)]


def _int32(t: torch.Tensor, dims: int, device, name: str):
    if t.dtype != torch.int32 or t.dim() != dims or t.device != device or (t.shape[-1] > 1 and t.stride(-1) != 1):
        raise ValueError(f"{name} must be an int32 tensor of {dims} dimension(s) on {device}, unit stride in the last")


class Rope:
    """A rotary table: cos_sin fp32 [positions, rot_dim] (cos of the rot_dim / 2 pairs, then sin), the pairs
    of each axis (``sections``; one axis by default) and whether a pair's channels are neighbours."""

    def __init__(self, cos_sin: torch.Tensor, sections=None, interleaved: bool = False):
        if cos_sin.dtype != torch.float32 or cos_sin.dim() != 2 or not cos_sin.is_contiguous() or not cos_sin.is_cuda:
            raise ValueError("cos_sin must be a contiguous fp32 CUDA tensor [positions, rot_dim]")
        rot = cos_sin.shape[1]
        sections = [rot // 2] if sections is None else [int(s) for s in sections]
        if rot % 8 or not 8 <= rot <= HEAD_DIM:
            raise ValueError("rot_dim must be a multiple of 8 between 8 and 128")
        if not 1 <= len(sections) <= ROPE_MAX_AXES or min(sections) < 0 or sum(sections) != rot // 2:
            raise ValueError("sections: one to three pair counts that add up to rot_dim / 2")
        self.cos_sin, self.axes = cos_sin, len(sections)
        self.desc = RopeDesc(cos_sin.data_ptr(), cos_sin.shape[0], rot, len(sections), int(interleaved),
                             (ctypes.c_int32 * ROPE_MAX_AXES)(*sections), 0)
        self._ref = ctypes.addressof(self.desc)


class PagedCache:
    """Pages of compressed keys and values: ``pages`` uint8 [num_pages, num_kv_heads, page_tokens / 32, 3200]
    (layout in include/kv1b.h).  Which page belongs to which sequence is the caller's page table."""

    def __init__(self, num_pages: int, num_kv_heads: int, page_tokens: int = 128, seed: int = 0, device="cuda",
                 stream=None, rounds: int = 1):
        nbytes = lib().kv1b_paged_bytes(num_pages, num_kv_heads, HEAD_DIM, page_tokens)
        if nbytes == 0:
            raise Kv1bError(-1, "kv1b_paged_bytes")
        device = torch.device(device)
        s = stream if stream is not None else torch.cuda.current_stream(device)
        with torch.cuda.device(s.device), torch.cuda.stream(s):
            pages = torch.empty((num_pages, num_kv_heads, page_tokens // BLOCK_TOKENS, BLOCK_BYTES), dtype=torch.uint8,
                                device=device)
            signs = torch.empty((3, HEAD_DIM), dtype=torch.float32, device=device)
            status = torch.empty((1,), dtype=torch.int32, device=device)
            _check(lib().kv1b_paged_signs(signs.data_ptr(), seed, rounds, status.data_ptr(), s.cuda_stream),
                   "kv1b_paged_signs")
        self._attach(pages, signs, status)

    @classmethod
    def wrap(cls, pages: torch.Tensor, signs: torch.Tensor, status: torch.Tensor | None = None) -> "PagedCache":
        """A cache over buffers the caller holds: pages as above, signs fp32 [3, 128] (+-1, zeros in the
        rounds past the last), status int32 [1] (a new zero one by default)."""
        if pages.dtype != torch.uint8 or pages.dim() != 4 or pages.shape[3] != BLOCK_BYTES or not pages.is_contiguous():
            raise ValueError("pages must be a contiguous uint8 tensor [num_pages, num_kv_heads, page_tokens / 32, 3200]")
        if signs.dtype != torch.float32 or tuple(signs.shape) != (3, HEAD_DIM) or not signs.is_contiguous() \
                or signs.device != pages.device:
            raise ValueError("signs must be a contiguous fp32 tensor [3, 128] on the pages' device")
        if not pages.is_cuda:
            raise ValueError("pages must be a CUDA tensor")
        if status is None:
            status = torch.zeros((1,), dtype=torch.int32, device=pages.device)
        elif status.dtype != torch.int32 or status.numel() != 1 or status.device != pages.device:
            raise ValueError("status must be an int32 tensor of one element on the pages' device")
        if lib().kv1b_paged_bytes(pages.shape[0], pages.shape[1], HEAD_DIM, pages.shape[2] * BLOCK_TOKENS) == 0:
            raise Kv1bError(-1, "kv1b_paged_bytes")
        self = cls.__new__(cls)
        self._attach(pages, signs, status)
        return self

    def _attach(self, pages, signs, status):
        self.pages, self.signs, self.status_word = pages, signs, status
        self.num_pages, self.num_kv_heads = pages.shape[0], pages.shape[1]
        self.page_tokens = pages.shape[2] * BLOCK_TOKENS
        self.device = pages.device
        self.desc = PagedDesc(pages.data_ptr(), signs.data_ptr(), status.data_ptr(), self.num_pages, self.num_kv_heads,
                              self.page_tokens, 0)
        self._ref = ctypes.addressof(self.desc)
        self._ws_bytes = {}

    def _launch_stream(self, stream):
        s = stream if stream is not None else torch.cuda.current_stream(self.device)
        if s.device != self.device:
            raise ValueError(f"the stream is on {s.device}, the cache on {self.device}")
        return s

    def _on_device(self, t: torch.Tensor, name: str):
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, the cache on {self.device}")

    def append(self, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor, start: torch.Tensor, cu_new: torch.Tensor,
               rope: Rope | None = None, positions: torch.Tensor | None = None, q: torch.Tensor | None = None,
               q_out: torch.Tensor | None = None, stream=None) -> torch.Tensor | None:
        """Encode new tokens into the pages, keys turned by ``rope`` at ``positions`` on the way.

        k, v: [tokens, num_kv_heads, 128] rows of all sequences behind one another (any token and head
        strides that are multiples of 4); cu_new int32 [seqs + 1] says which rows are whose, start int32
        [seqs] how many tokens each sequence holds (not advanced here), page_table int32 [seqs, pages].
        positions: int32 [tokens], or [axes, tokens].  q [tokens, q heads, 128]: turned alike into q_out
        (a new contiguous tensor by default; q itself allowed), which is returned."""
        dev = self.device
        if k.dim() != 3 or k.shape != v.shape or k.dtype != v.dtype or k.shape[1:] != (self.num_kv_heads, HEAD_DIM) \
                or k.stride(2) != 1 or v.stride(2) != 1:
            raise ValueError("k and v must be [tokens, num_kv_heads, 128] of one type with unit channel stride")
        self._on_device(k, "k")
        self._on_device(v, "v")
        T = k.shape[0]
        _int32(page_table, 2, dev, "page_table")
        _int32(start, 1, dev, "start")
        _int32(cu_new, 1, dev, "cu_new")
        B = page_table.shape[0]
        if start.shape[0] != B or cu_new.shape[0] != B + 1:
            raise ValueError("page_table [seqs, pages], start [seqs] and cu_new [seqs + 1] disagree")
        ps, pos = 0, None
        if rope is not None:
            if positions is None:
                raise ValueError("rope needs positions")
            _int32(positions, positions.dim(), dev, "positions")
            if positions.shape != ((rope.axes, T) if positions.dim() == 2 else (T,)) or (positions.dim() == 1 and rope.axes > 1):
                raise ValueError("positions must be [tokens] or [axes, tokens]")
            self._on_device(rope.cos_sin, "cos_sin")
            ps, pos = (positions.stride(0) if rope.axes > 1 else 0), positions.data_ptr()
        elif positions is not None:
            raise ValueError("positions need rope")
        s = self._launch_stream(stream)
        qp = qo = None
        hq = qs0 = qs1 = os0 = os1 = 0
        if q is not None:
            if q.dim() != 3 or q.shape[0] != T or q.shape[2] != HEAD_DIM or q.dtype != k.dtype or q.stride(2) != 1:
                raise ValueError("q must be [tokens, q heads, 128] of k's type with unit channel stride")
            self._on_device(q, "q")
            if q_out is None:
                with torch.cuda.stream(s):
                    q_out = torch.empty(q.shape, dtype=q.dtype, device=dev)
            elif q_out.shape != q.shape or q_out.dtype != q.dtype or q_out.stride(2) != 1 or q_out.device != dev:
                raise ValueError("q_out must have q's shape, type and device, unit channel stride")
            hq, qp, qo = q.shape[1], q.data_ptr(), q_out.data_ptr()
            qs0, qs1, os0, os1 = q.stride(0), q.stride(1), q_out.stride(0), q_out.stride(1)
        elif q_out is not None:
            raise ValueError("q_out needs q")
        if T == 0:
            return q_out
        with torch.cuda.device(dev):
            _check(lib().kv1b_paged_append(self._ref, k.data_ptr(), v.data_ptr(), _dtype_code(k), T, k.stride(0), k.stride(1),
                                           v.stride(0), v.stride(1), B, cu_new.data_ptr(), start.data_ptr(),
                                           page_table.data_ptr(), page_table.stride(0), page_table.shape[1],
                                           rope._ref if rope is not None else None, pos, ps, qp, qo, hq, qs0, qs1, os0, os1,
                                           s.cuda_stream), "kv1b_paged_append")
        return q_out

    def _attend_args(self, q, page_table, lengths, out, s):
        if q.dim() != 3 or q.shape[2] != HEAD_DIM or not q.is_contiguous():
            raise ValueError("q must be a contiguous tensor [seqs, q heads, 128]")
        self._on_device(q, "q")
        _int32(page_table, 2, self.device, "page_table")
        _int32(lengths, 1, self.device, "lengths")
        if page_table.shape[0] != q.shape[0] or lengths.shape[0] != q.shape[0]:
            raise ValueError("q, page_table and lengths disagree on the number of sequences")
        if out is None:
            with torch.cuda.stream(s):
                out = torch.empty(q.shape, dtype=q.dtype, device=self.device)
        elif out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous() or out.device != self.device:
            raise ValueError("out must be a contiguous tensor of q's shape and type")
        return out

    def _workspace(self, key, s):
        """A workspace of this call's own, from the stream's memory (a capture's from its graph's)."""
        n = self._ws_bytes.get(key)
        if n is None:
            with torch.cuda.device(self.device):
                n = lib().kv1b_paged_attend_workspace_bytes(self._ref, key[1]) if key[0] == 0 else \
                    lib().kv1b_paged_shared_workspace_bytes(self._ref, *key)
            if n == 0:
                raise Kv1bError(-1, "kv1b_paged_attend_workspace_bytes")
            self._ws_bytes[key] = n
        with torch.cuda.stream(s):
            return torch.empty(n, dtype=torch.uint8, device=self.device)

    def attend(self, q: torch.Tensor, scale: float, page_table: torch.Tensor, lengths: torch.Tensor, window: int = 0,
               sinks: int = 0, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """Decode attention of q [seqs, q heads, 128] (bf16 / fp16) over each sequence's first lengths[b]
        tokens (int32, on the device); with window > 0 over the last `window` and the first `sinks` of them.
        Returns q's shape and type."""
        s = self._launch_stream(stream)
        out = self._attend_args(q, page_table, lengths, out, s)
        if q.shape[0] == 0:
            return out
        ws = self._workspace((0, q.shape[1]), s)
        with torch.cuda.device(self.device):
            _check(lib().kv1b_paged_attend(self._ref, q.data_ptr(), _dtype_code(q), q.shape[1], scale, q.shape[0],
                                           page_table.data_ptr(), page_table.stride(0), page_table.shape[1],
                                           lengths.data_ptr(), window, sinks, out.data_ptr(), ws.data_ptr(), ws.numel(),
                                           s.cuda_stream), "kv1b_paged_attend")
        return out

    def attend_shared(self, q: torch.Tensor, scale: float, prefix_pages: torch.Tensor, prefix_length: torch.Tensor,
                      page_table: torch.Tensor, lengths: torch.Tensor, out: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
        """Decode attention for sequences that all begin with the prefix_length[0] tokens (int32 [1], on the
        device) of prefix_pages (int32 [pages]) and go on with lengths[b] tokens of their own."""
        s = self._launch_stream(stream)
        out = self._attend_args(q, page_table, lengths, out, s)
        _int32(prefix_pages, 1, self.device, "prefix_pages")
        _int32(prefix_length, 1, self.device, "prefix_length")
        if prefix_length.shape[0] != 1 or prefix_pages.shape[0] < 1:
            raise ValueError("prefix_length must hold one number and prefix_pages one page at least")
        if q.shape[0] == 0:
            return out
        ws = self._workspace((q.shape[0], q.shape[1], prefix_pages.shape[0]), s)
        with torch.cuda.device(self.device):
            _check(lib().kv1b_paged_attend_shared(self._ref, q.data_ptr(), _dtype_code(q), q.shape[1], scale, q.shape[0],
                                                  prefix_pages.data_ptr(), prefix_pages.shape[0], prefix_length.data_ptr(),
                                                  page_table.data_ptr(), page_table.stride(0), page_table.shape[1],
                                                  lengths.data_ptr(), out.data_ptr(), ws.data_ptr(), ws.numel(),
                                                  s.cuda_stream), "kv1b_paged_attend_shared")
        return out

    def status(self, stream=None) -> int:
        """The KV1B_STATUS_* bits since the cache was made (waits for the stream)."""
        s = self._launch_stream(stream)
        with torch.cuda.stream(s):
            return int(self.status_word.item())
