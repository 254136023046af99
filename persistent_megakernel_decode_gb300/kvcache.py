"""8-bit paged KV cache: attention over it, storing, loading, copying pages, and the accounting of pages.

Binding of the ``mk_cache_*`` and ``mk_pages_*`` calls of ``include/mk.h``, which has the definitions (layout, scales,
masks, what a failed check does); this module checks arguments and marshals them.  Every call is asynchronous on
``stream`` (default: the current torch stream of the cache's device), where its tensors have to be ready, and may be
captured into a CUDA graph, except ``Kv8Cache.check``, which synchronises.  Tensors may be dropped after the call.
Threads may share a ``Kv8Cache`` (not a ``PagePool``).
"""
from __future__ import annotations

import ctypes as C
import threading
from array import array
from typing import List, Optional, Sequence, Tuple

import numpy as np
import torch

from . import runtime as rt

rt.need_torch()
_CODES = (torch.float8_e4m3fn, torch.uint8)
_I32, _BF16 = torch.int32, torch.bfloat16


class Kv8Cache:
    """e4m3 K codes [L, N, Hkv, P, D], V codes [L, N, Hkv, D, P] and their fp32 scales [L, N, Hkv] (contiguous CUDA
    tensors, codes as float8_e4m3fn or uint8); P 32 or 64, D 64 or 128.  The tensors stay the caller's: nothing is
    copied.  ``table`` arguments are int32 [B, width]: sequence b's token j lies in page table[b, j // P]."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor):
        if not k.is_cuda:
            raise ValueError("the cache must be CUDA tensors")
        if k.dim() != 5 or k.dtype not in _CODES:
            raise ValueError(f"k must be e4m3 codes [L, N, Hkv, P, D], got {k.dtype} {tuple(k.shape)}")
        L, N, H, P, D = k.shape
        self.index = k.get_device()
        rt.check_tensor("v", v, self.index, k.dtype, (L, N, H, D, P))
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            rt.check_tensor(name, t, self.index, torch.float32, (L, N, H))
        if not all(t.is_contiguous() for t in (k, v, k_scale, v_scale)):
            raise ValueError("the cache's tensors must be contiguous")
        if P not in (32, 64) or D not in (64, 128):
            raise ValueError(f"pages of {P} tokens with head_dim {D}: 32 or 64 tokens, 64 or 128 dims are supported")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.layers, self.pages, self.kv_heads, self.page_tokens, self.head_dim = L, N, H, P, D
        self.device = k.device
        self.status = torch.zeros(4, dtype=torch.int32, device=k.device)
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(self.index).synchronize()  # the status words are zero for calls on any stream
        self.num_sms = 0  # SMs that attend plans for; 0: all of the device
        self._desc = rt.CacheDesc(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                                  self.status.data_ptr(), L, N, H, P, D)
        self._ref = C.byref(self._desc)  # never changed after this
        self._lib = rt.load()
        self._kept = None  # the default stream's workspace
        self._lock = threading.Lock()  # of _kept, from its choice to the last launch that uses it
        self._sizes = {}  # workspace bytes by (batch, table width, q heads, tokens, most tokens of a sequence, num_sms)

    @classmethod
    def empty(cls, layers: int, pages: int, kv_heads: int, head_dim: int, page_tokens: int = 64, device="cuda"):
        """A cache of zeroed pages."""
        dev = torch.device(device)
        codes = lambda *s: torch.zeros((layers, pages, kv_heads) + s, dtype=torch.uint8, device=dev)  # noqa: E731
        scale = lambda: torch.zeros((layers, pages, kv_heads), dtype=torch.float32, device=dev)  # noqa: E731
        return cls(codes(page_tokens, head_dim).view(torch.float8_e4m3fn),
                   codes(head_dim, page_tokens).view(torch.float8_e4m3fn), scale(), scale())

    def _ints(self, b, name, t):
        """An int32 [b] device array, contiguous: its address."""
        if t.dtype is not _I32 or t.get_device() != self.index or t.shape != (b,) or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 [{b}] tensor on cuda:{self.index}, got {t.dtype} "
                             f"{tuple(t.shape)} on {t.device}")
        return t.data_ptr()

    def _table(self, table, b):
        """Address and width of an int32 [b, width] device array, contiguous."""
        shape = table.shape
        if (table.dtype is not _I32 or table.get_device() != self.index or len(shape) != 2 or shape[0] != b
                or not table.is_contiguous()):
            raise ValueError(f"table must be a contiguous int32 [{b}, width] tensor on cuda:{self.index}, got "
                             f"{table.dtype} {tuple(table.shape)} on {table.device}")
        return table.data_ptr(), shape[1]

    def _beside(self, stream, call, *args):
        for t in (self.k, self.v, self.k_scale, self.v_scale, self.status):
            t.record_stream(stream)
        return rt.beside(self.index, stream, call, *args)

    # ---- moving tokens ----
    def _move(self, call, k, v, table, start, count, row0, max_count, stream, writes):
        if stream is not None and not rt.is_current(self.index, stream):
            return self._beside(stream, self._move, call, k, v, table, start, count, row0, max_count, None, writes)
        shape = k.shape
        if len(shape) != 5 or shape[0] != self.layers or shape[3] != self.kv_heads or shape[4] != self.head_dim:
            raise ValueError(f"k has shape {tuple(shape)}, expected ({self.layers}, B, T, {self.kv_heads}, {self.head_dim})")
        ks, vs, kp, vp = k.stride(), v.stride(), k.data_ptr(), v.data_ptr()
        if (k.dtype is not _BF16 or v.dtype is not _BF16 or k.get_device() != self.index or v.get_device() != self.index
                or v.shape != shape):
            for name, t in (("k", k), ("v", v)):
                rt.check_tensor(name, t, self.index, _BF16, shape)
        if (ks[4] != 1 or vs[4] != 1 or (kp | vp) % 16
                or (ks[0] | ks[1] | ks[2] | ks[3] | vs[0] | vs[1] | vs[2] | vs[3]) % 8):
            raise ValueError("k and v: head_dim must be contiguous, the base 16-byte aligned, strides multiples of 8 elements")
        if writes and any(s[i] == 0 and shape[i] > 1 for s in (ks, vs) for i in ((0, 2, 3) if row0 is not None else (0, 1, 2, 3))):
            raise ValueError("rows that overlap cannot be written")
        b, rows = shape[1], shape[2]
        at, width = self._table(table, b)
        first, n = self._ints(b, "start", start), self._ints(b, "count", count)
        offset = 0 if row0 is None else self._ints(b, "row0", row0)
        if b == 0 or rows == 0:
            return
        r = rt.CacheRows(kp, vp, *ks[:4], *vs[:4], rows, offset)
        rt.launch(self.index, None, call, self._ref, C.byref(r), at, width, first, n, b,
                  rows if max_count is None else rt.c_int(max_count))

    def store(self, k, v, table, start, count, row0=None, max_count: Optional[int] = None, stream=None):
        """Quantise new tokens into the cache, all layers: row ``row0[b] + i`` (default 0 + i) of sequence b in ``k`` and
        ``v`` (bf16 [L, B, T, Hkv, D], any strides with D contiguous; packed ragged tokens [L, total, Hkv, D] are
        ``x[:, None].expand(L, B, total, Hkv, D)`` with ``row0``) becomes cache position ``start[b] + i``, i <
        ``count[b]``.  ``max_count`` (default T) bounds the counts.  Pages written must belong to one sequence only."""
        self._move(self._lib.mk_cache_store, k, v, table, start, count, row0, max_count, stream, False)

    def load(self, k, v, table, start, count, row0=None, max_count: Optional[int] = None, stream=None):
        """The inverse of :meth:`store`: cache positions ``start[b] + i`` into rows ``row0[b] + i``; other rows stay.
        (Packed rows as in :meth:`store`: the sequences' rows must not overlap.)"""
        self._move(self._lib.mk_cache_load, k, v, table, start, count, row0, max_count, stream, True)

    # ---- attention ----
    def attend(self, q, table, lens, layer: int = 0, q_start=None, max_tokens: Optional[int] = None,
               scale: Optional[float] = None, window: int = 0, out=None, lse=None, workspace=None,
               stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
        """Attention of new tokens over ``layer`` of the cache (their K/V stored before): ``lens[b]`` tokens are cached,
        the last T of them are the queries.  ``q`` is bf16 [B, T, Hq, D], or with ``q_start`` (int32 [B + 1]) packed
        [total, Hq, D], sequence b's queries being rows q_start[b] .. q_start[b + 1] - 1 (``max_tokens``: the most of
        one sequence, a hint for the height of the tiles and so for the workspace; default: all rows).  ``window`` > 0:
        a query sees that many last tokens, itself among them.  Returns (out bf16 like q, lse fp32 without the last
        axis); a query that sees nothing gets 0 and -inf.  ``workspace``: uint8 tensor of at least
        :meth:`attend_workspace` bytes, used by one call at a time; by default calls on the default stream share one
        that the cache keeps, others allocate their own."""
        if stream is not None and not rt.is_current(self.index, stream):
            return self._beside(stream, self.attend, q, table, lens, layer, q_start, max_tokens, scale, window, out, lse,
                                workspace)
        D, packed, shape = self.head_dim, q_start is not None, q.shape
        if (q.dtype is not torch.bfloat16 or q.get_device() != self.index or len(shape) != (3 if packed else 4)
                or shape[-1] != D):
            raise ValueError(f"q must be bf16 {'[total, Hq' if packed else '[B, T, Hq'}, {D}] on cuda:{self.index}, got "
                             f"{q.dtype} {tuple(shape)} on {q.device}")
        hq = shape[-2]
        if packed:
            b = q_start.numel() - 1
            queries = self._ints(max(b, 0) + 1, "q_start", q_start)
            total, most = shape[0], shape[0] if max_tokens is None else rt.c_int(max_tokens)
        else:
            b, most, queries = shape[0], shape[1], 0
            total = b * most
            if max_tokens is not None and max_tokens != most:
                raise ValueError("max_tokens is q's second axis without q_start")
        at, width = self._table(table, b)
        held = self._ints(b, "lens", lens)
        if out is None:
            out = torch.empty(shape, dtype=_BF16, device=self.device)
        else:
            rt.check_tensor("out", out, self.index, _BF16, shape)
            if any(n > 1 and x == 0 for n, x in zip(shape, out.stride())):
                raise ValueError("rows that overlap cannot be written")
        if lse is None:
            lse = torch.empty(shape[:-1], dtype=torch.float32, device=self.device)
        else:
            rt.check_tensor("lse", lse, self.index, torch.float32, shape[:-1])
            if not lse.is_contiguous():
                raise ValueError("lse must be contiguous")
        qs, os, qp, op = q.stride(), out.stride(), q.data_ptr(), out.data_ptr()
        # rows are tokens: one a sequence apart, or the sequences one after the other
        qt, ot = (qs[0], os[0]) if packed or most == 1 else (qs[1], os[1])
        if total and (qs[-1] != 1 or os[-1] != 1 or (qp | op) % 16 or (qs[-2] | qt | os[-2] | ot) % 8
                      or (not packed and b > 1 and (qs[0] != qt * most or os[0] != ot * most))):
            raise ValueError("q and out: head_dim must be contiguous, the base 16-byte aligned, strides multiples of 8 "
                             "elements, and sequences evenly spaced rows")
        a = rt.AttendDesc(qp, op, lse.data_ptr(), qt, qs[-2], ot, os[-2], at, held, queries, b, width, hq, total,
                          most, rt.c_int(window), D ** -0.5 if scale is None else scale, self.num_sms)
        own = workspace is None
        if own:
            size = self._sizes.get((b, width, hq, total, most, self.num_sms)) or self._workspace(a)
        else:
            rt.check_tensor("workspace", workspace, self.index, torch.uint8)
            if not workspace.is_contiguous():
                raise ValueError("workspace must be contiguous")
            size = workspace.numel()
        if own and torch._C._cuda_getCurrentRawStream(self.index) == 0:
            # Calls on the default stream share a workspace.  One call is two launches, which another thread's must not
            # come between; the stream orders the calls, and cannot be captured.
            with self._lock:
                if self._kept is None or self._kept.numel() < size:
                    self._kept = torch.empty(size, dtype=torch.uint8, device=self.device)
                rt.launch(self.index, None, self._lib.mk_cache_attend, self._ref, rt.c_int(layer), C.byref(a),
                          self._kept.data_ptr(), size)
        else:
            if own:
                workspace = torch.empty(size, dtype=torch.uint8, device=self.device)
            rt.launch(self.index, None, self._lib.mk_cache_attend, self._ref, rt.c_int(layer), C.byref(a),
                      workspace.data_ptr(), size)
        return out, lse

    def _workspace(self, a) -> int:
        n = C.c_uint64()
        with torch.cuda.device(self.index):
            rt._check(self._lib.mk_cache_attend_workspace(self._ref, C.byref(a), C.byref(n)))
        if len(self._sizes) >= 1024:
            self._sizes.clear()
        self._sizes[a.batch, a.table_width, a.q_heads, a.tokens, a.max_tokens, a.num_sms] = n.value
        return n.value

    def attend_workspace(self, batch: int, q_heads: int, max_tokens: int = 1, table_width: int = 1 << 20) -> int:
        """Bytes of workspace :meth:`attend` needs for up to ``batch`` sequences of up to ``max_tokens`` queries (and
        ``table_width`` pages; packed queries: with that ``max_tokens`` as its hint)."""
        a = rt.AttendDesc()
        a.batch, a.q_heads, a.tokens, a.max_tokens = map(rt.c_int, (batch, q_heads, batch * max_tokens, max_tokens))
        a.table_width, a.num_sms = rt.c_int(table_width), self.num_sms
        return self._workspace(a)

    # ---- pages ----
    def copy_pages(self, src: Sequence[int], dst: Sequence[int], table=None, stream=None):
        """Copy pages ``src[i]`` -> ``dst[i]`` in all layers (codes and scales); no dst may repeat or be a src.  With
        ``table`` (a contiguous int32 tensor) its entries that name a src are renamed to the dst."""
        if stream is not None and not rt.is_current(self.index, stream):
            return self._beside(stream, self.copy_pages, src, dst, table)
        s, d = array("i", src), array("i", dst)
        if len(s) != len(d):
            raise ValueError("src and dst must be lists of the same length")
        if table is not None:
            rt.check_tensor("table", table, self.index, torch.int32)
            if not table.is_contiguous():
                raise ValueError("table must be contiguous")
        rt.launch(self.index, None, self._lib.mk_cache_copy, self._ref, s.buffer_info()[0], d.buffer_info()[0], len(s),
                  table.data_ptr() if table is not None else None, table.numel() if table is not None else 0)

    def check(self, stream=None):
        """Wait for ``stream`` and raise ``MkError`` if a device-side check has failed since the last call."""
        rt.launch(self.index, stream, self._lib.mk_cache_status, self._ref, 1, None)


class PagePool:
    """Which pages of a cache are in use, with reference counts (host only; not thread-safe).  Sequences are lists of
    page numbers in token order."""

    def __init__(self, num_pages: int):
        self.num_pages = num_pages
        self._lib = rt.load()
        self.h = C.c_void_p()
        rt._check(self._lib.mk_pages_create(num_pages, C.byref(self.h)))

    def alloc(self, n: int) -> List[int]:
        """Take ``n`` free pages, the lowest-numbered first; ``MkError`` (and none taken) if there are fewer."""
        ids = np.zeros(max(n, 1), np.int32)
        rt._check(self._lib.mk_pages_alloc(self.h, n, ids.ctypes.data))
        return ids[:n].tolist()

    def share(self, pages: Sequence[int]):
        """One more reference to each page."""
        a = np.ascontiguousarray(pages, dtype=np.int32)
        rt._check(self._lib.mk_pages_share(self.h, a.ctypes.data, len(a)))

    def release(self, pages: Sequence[int]):
        """Drop one reference to each page; one that nobody holds is free."""
        a = np.ascontiguousarray(pages, dtype=np.int32)
        rt._check(self._lib.mk_pages_release(self.h, a.ctypes.data, len(a)))

    def fork(self, pages: Sequence[int], length: int, page_tokens: int) -> Tuple[List[int], List[int], List[int]]:
        """A child of a sequence of ``length`` tokens: its full pages are shared, a last page that is not full gets a page
        of its own.  Returns (child's pages, src, dst): copy src -> dst with ``Kv8Cache.copy_pages``."""
        used = -(-length // page_tokens)
        if length < 0 or used > len(pages):
            raise ValueError(f"{len(pages)} pages do not hold {length} tokens")
        full = length // page_tokens
        fresh = self.alloc(used - full)
        try:
            self.share(pages[:full])
        except rt.MkError:
            self.release(fresh)
            raise
        return list(pages[:full]) + fresh, list(pages[full:used]), fresh

    def compact(self) -> Tuple[List[int], List[int]]:
        """Renumber the pages in use to 0 .. used - 1; returns the moves (src, dst): pass them, with the page tables, to
        ``Kv8Cache.copy_pages``."""
        s, d, n = np.zeros(self.num_pages, np.int32), np.zeros(self.num_pages, np.int32), C.c_int()
        rt._check(self._lib.mk_pages_compact(self.h, s.ctypes.data, d.ctypes.data, C.byref(n)))
        return s[:n.value].tolist(), d[:n.value].tolist()

    def refs(self) -> np.ndarray:
        """Reference counts, int32 [num_pages]."""
        out = np.zeros(self.num_pages, np.int32)
        rt._check(self._lib.mk_pages_info(self.h, out.ctypes.data, None))
        return out

    @property
    def free_pages(self) -> int:
        n = C.c_int()
        rt._check(self._lib.mk_pages_info(self.h, None, C.byref(n)))
        return n.value

    def free(self):
        if self.h and self.h.value:
            self._lib.mk_pages_free(self.h)
            self.h = C.c_void_p()

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass
