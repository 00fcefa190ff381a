"""Paged cache: the compressed keys and values of a serving batch in pages of one buffer.

Argument marshalling for the ``kv1b_paged_*`` calls of ``include/kv1b.h``.  Lengths, page tables and
positions are device tensors that the kernels read, so a decode step (append, attend) can be captured
in a CUDA graph once and replayed while they change in place.
"""
from __future__ import annotations

import ctypes

import torch

from . import DTYPE_BF16, DTYPE_F16, DTYPE_F32, HEAD_DIM, Kv1bError, _check, lib

# the current stream's handle without a Stream object around it (microseconds a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)

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


_DTYPE_CODES = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16}


def _int32(t: torch.Tensor, dims: int, index: int, name: str):
    if t.dtype is not torch.int32 or t.dim() != dims or t.get_device() != index or (t.stride(-1) != 1 and t.shape[-1] > 1):
        raise ValueError(f"{name} must be an int32 tensor of {dims} dimension(s) on cuda:{index}, unit stride in the last")


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
        self.cos_sin, self.axes, self.index = cos_sin, len(sections), cos_sin.get_device()
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
        self._index = pages.get_device()
        self._lib = lib()
        self.desc = PagedDesc(pages.data_ptr(), signs.data_ptr(), status.data_ptr(), self.num_pages, self.num_kv_heads,
                              self.page_tokens, 0)
        self._ref = ctypes.addressof(self.desc)
        self._ws_bytes = {}

    def _on(self, stream):
        """Context of a call's allocations and launches: the cache's device, and `stream` if one is given."""
        if stream is None:
            return torch.cuda.device(self._index)
        if stream.device != self.device:
            raise ValueError(f"the stream is on {stream.device}, the cache on {self.device}")
        return torch.cuda.stream(stream)  # its device too

    def _away(self, stream) -> bool:
        return stream is not None or torch.cuda.current_device() != self._index

    def _on_device(self, t: torch.Tensor, name: str):
        if t.get_device() != self._index:
            raise ValueError(f"{name} is on {t.device}, the cache on {self.device}")

    def append(self, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor, start: torch.Tensor, cu_new: torch.Tensor,
               rope: Rope | None = None, positions: torch.Tensor | None = None, q: torch.Tensor | None = None,
               q_out: torch.Tensor | None = None, stream=None) -> torch.Tensor | None:
        """Encode new tokens into the pages, keys turned by ``rope`` at ``positions`` on the way.

        k, v: [tokens, num_kv_heads, 128] rows of all sequences behind one another (any token and head
        strides that are multiples of 4); cu_new int32 [seqs + 1] says which rows are whose, start int32
        [seqs] how many tokens each sequence holds (not advanced here), page_table int32 [seqs, pages].
        positions: int32 [tokens], or [axes, tokens] (positions.expand(axes, tokens) where all axes agree).
        q [tokens, q heads, 128]: turned alike into q_out (a new contiguous tensor by default; q itself
        allowed, otherwise clear of q, k and v), which is returned."""
        if self._away(stream):
            with self._on(stream):
                return self.append(k, v, page_table, start, cu_new, rope, positions, q, q_out)
        index = self._index
        T, H, D = shape = k.shape
        dtype = _DTYPE_CODES.get(k.dtype)
        (kt, kh, kc), (vt, vh, vc) = k.stride(), v.stride()
        if H != self.num_kv_heads or D != HEAD_DIM or v.shape != shape or k.dtype is not v.dtype or kc != 1 or vc != 1 \
                or dtype is None:
            raise ValueError("k and v must be [tokens, num_kv_heads, 128] of one floating type with unit channel stride")
        self._on_device(k, "k")
        self._on_device(v, "v")
        _int32(page_table, 2, index, "page_table")
        _int32(start, 1, index, "start")
        _int32(cu_new, 1, index, "cu_new")
        B, pages = page_table.shape
        if start.shape[0] != B or cu_new.shape[0] != B + 1:
            raise ValueError("page_table [seqs, pages], start [seqs] and cu_new [seqs + 1] disagree")
        ps, pos, ro = 0, None, None
        if rope is not None:
            if positions is None:
                raise ValueError("rope needs positions")
            dims = positions.dim()
            _int32(positions, dims, index, "positions")
            if positions.shape != ((rope.axes, T) if dims == 2 else (T,)) or (dims == 1 and rope.axes > 1):
                raise ValueError("positions must be [tokens] or [axes, tokens]")
            if rope.index != index:
                raise ValueError(f"cos_sin is on cuda:{rope.index}, the cache on {self.device}")
            ps, pos, ro = (positions.stride(0) if rope.axes > 1 else 0), positions.data_ptr(), rope._ref
        elif positions is not None:
            raise ValueError("positions need rope")
        qp = qo = None
        hq = qs0 = qs1 = os0 = os1 = 0
        if q is not None:
            tq, hq, dq = q.shape
            qs0, qs1, qc = q.stride()
            if tq != T or dq != HEAD_DIM or q.dtype is not k.dtype or qc != 1:
                raise ValueError("q must be [tokens, q heads, 128] of k's type with unit channel stride")
            self._on_device(q, "q")
            if q_out is None:
                q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
            elif q_out.shape != q.shape or q_out.dtype is not q.dtype or q_out.stride(2) != 1 or q_out.get_device() != index:
                raise ValueError("q_out must have q's shape, type and device, unit channel stride")
            qp, qo = q.data_ptr(), q_out.data_ptr()
            os0, os1, _ = q_out.stride()
        elif q_out is not None:
            raise ValueError("q_out needs q")
        if T == 0:
            return q_out
        code = self._lib.kv1b_paged_append(self._ref, k.data_ptr(), v.data_ptr(), dtype, T, kt, kh, vt, vh, B,
                                           cu_new.data_ptr(), start.data_ptr(), page_table.data_ptr(), page_table.stride(0),
                                           pages, ro, pos, ps, qp, qo, hq, qs0, qs1, os0, os1, _raw_stream(index))
        if code:
            _check(code, "kv1b_paged_append")
        return q_out

    def _attend_args(self, q, page_table, lengths, out):
        B, Hq, D = shape = q.shape
        dtype = _DTYPE_CODES.get(q.dtype)
        if D != HEAD_DIM or not q.is_contiguous() or dtype is None:
            raise ValueError("q must be a contiguous floating tensor [seqs, q heads, 128]")
        self._on_device(q, "q")
        _int32(page_table, 2, self._index, "page_table")
        _int32(lengths, 1, self._index, "lengths")
        rows, pages = page_table.shape
        if rows != B or lengths.shape[0] != B:
            raise ValueError("q, page_table and lengths disagree on the number of sequences")
        if out is None:
            out = torch.empty_like(q)
        elif out.shape != shape or out.dtype is not q.dtype or not out.is_contiguous() or out.get_device() != self._index:
            raise ValueError("out must be a contiguous tensor of q's shape and type")
        return out, B, Hq, dtype, pages

    def _workspace(self, key):
        """A workspace of this call's own, from the stream's memory (a capture's from its graph's)."""
        n = self._ws_bytes.get(key)
        if n is None:
            n = self._lib.kv1b_paged_attend_workspace_bytes(self._ref, key[1]) if key[0] == 0 else \
                self._lib.kv1b_paged_shared_workspace_bytes(self._ref, *key)
            if n == 0:
                raise Kv1bError(-1, "kv1b_paged_attend_workspace_bytes")
            self._ws_bytes[key] = n
        return torch.empty(n, dtype=torch.uint8, device=self.device), n

    def attend(self, q: torch.Tensor, scale: float, page_table: torch.Tensor, lengths: torch.Tensor, window: int = 0,
               sinks: int = 0, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """Decode attention of q [seqs, q heads, 128] (bf16 / fp16) over each sequence's first lengths[b]
        tokens (int32, on the device); with window > 0 over the last `window` and the first `sinks` of them.
        Returns q's shape and type (in ``out`` if given, q itself allowed)."""
        if self._away(stream):
            with self._on(stream):
                return self.attend(q, scale, page_table, lengths, window, sinks, out)
        out, B, Hq, dtype, pages = self._attend_args(q, page_table, lengths, out)
        if B == 0:
            return out
        ws, n = self._workspace((0, Hq))
        code = self._lib.kv1b_paged_attend(self._ref, q.data_ptr(), dtype, Hq, scale, B, page_table.data_ptr(),
                                           page_table.stride(0), pages, lengths.data_ptr(), window, sinks, out.data_ptr(),
                                           ws.data_ptr(), n, _raw_stream(self._index))
        if code:
            _check(code, "kv1b_paged_attend")
        return out

    def attend_shared(self, q: torch.Tensor, scale: float, prefix_pages: torch.Tensor, prefix_length: torch.Tensor,
                      page_table: torch.Tensor, lengths: torch.Tensor, out: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
        """Decode attention for sequences that all begin with the prefix_length[0] tokens (int32 [1], on the
        device) of prefix_pages (int32 [pages]) and go on with lengths[b] tokens of their own."""
        if self._away(stream):
            with self._on(stream):
                return self.attend_shared(q, scale, prefix_pages, prefix_length, page_table, lengths, out)
        out, B, Hq, dtype, pages = self._attend_args(q, page_table, lengths, out)
        _int32(prefix_pages, 1, self._index, "prefix_pages")
        _int32(prefix_length, 1, self._index, "prefix_length")
        npre = prefix_pages.shape[0]
        if prefix_length.shape[0] != 1 or npre < 1:
            raise ValueError("prefix_length must hold one number and prefix_pages one page at least")
        if B == 0:
            return out
        ws, n = self._workspace((B, Hq, npre))
        code = self._lib.kv1b_paged_attend_shared(self._ref, q.data_ptr(), dtype, Hq, scale, B, prefix_pages.data_ptr(), npre,
                                                  prefix_length.data_ptr(), page_table.data_ptr(), page_table.stride(0), pages,
                                                  lengths.data_ptr(), out.data_ptr(), ws.data_ptr(), n,
                                                  _raw_stream(self._index))
        if code:
            _check(code, "kv1b_paged_attend_shared")
        return out

    def status(self, stream=None) -> int:
        """The KV1B_STATUS_* bits since the cache was made (waits for the stream)."""
        with self._on(stream):
            return int(self.status_word.item())
