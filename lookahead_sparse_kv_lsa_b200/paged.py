"""A paged cache of grouped query heads, bounded by eviction: the handle over
lsa_paged_append, lsa_paged_attn and lsa_paged_evict (include/lsa.h).

PyTorch only allocates memory here, and the handle only checks and marshals: every step is
one call of the library.
"""
from __future__ import annotations

import ctypes as C
from typing import Optional

import torch

from . import _lib
from ._lib import BLOCK, LsaPagedCacheC, LsaPagedTablesC

_DTYPES = {torch.bfloat16: _lib.DTYPE_BF16, torch.float16: _lib.DTYPE_F16}


def _check(t, dtype, name: str, shape, device) -> Optional[int]:
    """The tensor's address; ValueError unless it is a contiguous tensor of this type, shape and
    device."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.device == device and t.is_contiguous()):
        return t.data_ptr()
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.device != device:
        raise ValueError("%s is on %s, the cache on %s" % (name, t.device, device))
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    raise ValueError("%s must be contiguous" % name)


class LsaPagedTables:
    """The page tables of a batch (lsa_paged_tables): block_table i32 [B][E], block_pos i32
    [B][E] or None (entry j is block j: not for tables with blocks left out, as lsa_gather's),
    score f32 [B][E] or None, n_entries and tail_len i32 [B], free_list i32 [B][F] and free_cnt
    i32 [B], or None (no pages to take or give back)."""

    def __init__(self, block_table, n_entries, tail_len, block_pos=None, score=None,
                 free_list=None, free_cnt=None):
        if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2 or not block_table.is_cuda:
            raise ValueError("block_table must be a CUDA tensor [B][entries]")
        B, E = block_table.shape
        dev, i32 = block_table.device, torch.int32
        if (free_list is None) != (free_cnt is None):
            raise ValueError("free_list and free_cnt come together")
        self.block_table, self.block_pos, self.score = block_table, block_pos, score
        self.n_entries, self.tail_len = n_entries, tail_len
        self.free_list, self.free_cnt = free_list, free_cnt
        self.B, self.bt_stride = B, E
        self.free_stride = 0 if free_list is None else free_list.shape[-1]
        self.device = dev
        for name in ("n_entries", "tail_len"):
            if getattr(self, name) is None:
                raise ValueError("%s is missing" % name)
        self.c = LsaPagedTablesC(
            _check(block_table, i32, "block_table", (B, E), dev),
            _check(block_pos, i32, "block_pos", (B, E), dev),
            _check(score, torch.float32, "score", (B, E), dev),
            _check(n_entries, i32, "n_entries", (B,), dev),
            _check(tail_len, i32, "tail_len", (B,), dev),
            _check(free_list, i32, "free_list", (B, self.free_stride), dev),
            _check(free_cnt, i32, "free_cnt", (B,), dev))
        self.ref = C.byref(self.c)
        self.layout = (B, E, self.free_stride, dev)

    @classmethod
    def allocate(cls, B: int, entries: int, pages_per_seq: int, device, score: bool = True,
                 first_page: int = 0):
        """Empty tables: sequence b owns the pages first_page + b * pages_per_seq ..., all of
        them on its free stack."""
        i32 = dict(dtype=torch.int32, device=device)
        own = first_page + torch.arange(B * pages_per_seq, **i32).view(B, pages_per_seq)
        return cls(torch.zeros((B, entries), **i32), torch.zeros(B, **i32), torch.zeros(B, **i32),
                   torch.zeros((B, entries), **i32),
                   torch.zeros((B, entries), device=device) if score else None,
                   own.flip(1).contiguous(), torch.full((B,), pages_per_seq, **i32))


class LsaPagedCache:
    """A pool, its tables and the attention's options (lsa_paged_cache); owns the workspace and
    the error word. Holds references to the tensors it is given, whose addresses it passes on.

    pool    bf16 or fp16 [pages][2][Hkv][64][d]
    tables  LsaPagedTables
    H       query heads (a multiple of Hkv); scale: 1/sqrt(d) by default
    cap     > 0: scores become cap * tanh(score / cap); window > 0: sliding window in tokens
    slopes  f32 [H]: bias -slopes[h] * distance; prefix_len, doc_start: i32 [B]
    decay   factor of the pages' scores per attended token
    """

    def __init__(self, pool, tables: LsaPagedTables, H: int, scale: Optional[float] = None,
                 cap: float = 0.0, window: int = 0, decay: float = 1.0, slopes=None,
                 prefix_len=None, doc_start=None):
        if not isinstance(pool, torch.Tensor) or pool.dtype not in _DTYPES:
            raise ValueError("pool must be a bf16 or fp16 tensor")
        if pool.dim() != 5 or pool.shape[1] != 2 or pool.shape[3] != BLOCK:
            raise ValueError("pool must have shape [pages][2][Hkv][%d][d]" % BLOCK)
        if tables.device != pool.device:
            raise ValueError("the tables are on %s, the pool on %s" % (tables.device, pool.device))
        dev = pool.device
        B, Hkv, d = tables.B, pool.shape[2], pool.shape[4]
        self.pool, self.tables, self.device = pool, tables, dev
        self.slopes, self.prefix_len, self.doc_start = slopes, prefix_len, doc_start
        self.B, self.H, self.Hkv, self.d, self.dtype = B, int(H), Hkv, d, pool.dtype
        self.err = torch.zeros(1, dtype=torch.int32, device=dev)
        s = LsaPagedCacheC()
        s.B, s.H, s.Hkv, s.d, s.dtype = B, int(H), Hkv, d, _DTYPES[pool.dtype]
        s.bt_stride, s.free_stride, s.window = tables.bt_stride, tables.free_stride, int(window)
        s.scale = float(d ** -0.5 if scale is None else scale)
        s.cap, s.decay = float(cap), float(decay)
        s.pool = _check(pool, pool.dtype, "pool", pool.shape, dev)
        s.n_pages = pool.shape[0]
        s.t = tables.c
        s.slopes = _check(slopes, torch.float32, "slopes", (int(H),), dev)
        s.prefix_len = _check(prefix_len, torch.int32, "prefix_len", (B,), dev)
        s.doc_start = _check(doc_start, torch.int32, "doc_start", (B,), dev)
        s.err = self.err.data_ptr()
        self._lib = _lib.lib()
        _lib.check("lsa_paged_check", self._lib.lsa_paged_check(s))
        n_sm = torch.cuda.get_device_properties(dev).multi_processor_count
        size = self._lib.lsa_paged_attn_workspace_size(B, int(H), Hkv, d, tables.bt_stride,
                                                       int(tables.score is not None), n_sm)
        self.ws = torch.empty(size, dtype=torch.uint8, device=dev)
        s.ws, s.ws_bytes = self.ws.data_ptr(), size
        self.state = s
        self._ref = C.byref(s)
        self._calls = {f: getattr(self._lib, f)
                       for f in ("lsa_paged_attn", "lsa_paged_append", "lsa_paged_evict")}
        self._q_shape = torch.Size((B, int(H), d))

    def _call(self, name: str, stream, *args) -> None:
        """One library call on `stream` (default: the current stream of the cache's device),
        with that device current."""
        f, index = self._calls[name], self.device.index
        if stream is None:
            stream = torch._C._cuda_getCurrentRawStream(index)
        elif isinstance(stream, torch.cuda.Stream):
            if stream.device != self.device:
                raise ValueError("the stream is on %s, the cache on %s" % (stream.device, self.device))
            stream = stream.cuda_stream
        if torch._C._cuda_getDevice() == index:
            st = f(self._ref, *args, stream)
        else:
            with torch.cuda.device(self.device):
                st = f(self._ref, *args, stream)
        if st:
            _lib.check(name, st)

    def _dst(self, dst: Optional[LsaPagedTables]):
        if dst is None:
            return None
        if dst.layout != self.tables.layout:
            raise ValueError("dst must have the shapes and the device of the cache's tables")
        return dst.ref

    def attend(self, q, out, stream=None) -> None:
        """One new token of every sequence over the cache (lsa_paged_attn). q, out: [B][H][d];
        adds the pages' weights to the tables' scores."""
        self._call("lsa_paged_attn", stream, _check(q, self.dtype, "q", self._q_shape, self.device),
                   _check(out, self.dtype, "out", self._q_shape, self.device))

    def append(self, k, v, tok_off=None, dst: Optional[LsaPagedTables] = None, stream=None) -> None:
        """New tokens behind every sequence's last (lsa_paged_append). k, v: [tokens][Hkv][d];
        tok_off: i32 [B+1], or None for one token per sequence."""
        n = k.shape[0] if isinstance(k, torch.Tensor) and k.dim() == 3 else self.B
        shape = (n, self.Hkv, self.d)
        off = None
        if tok_off is not None:
            off = _check(tok_off, torch.int32, "tok_off", (self.B + 1,), self.device)
        self._call("lsa_paged_append", stream, _check(k, self.dtype, "k", shape, self.device),
                   _check(v, self.dtype, "v", shape, self.device), n, off, self._dst(dst))

    def evict(self, budget: int, n_sink: int = 1, n_recent: int = 1,
              dst: Optional[LsaPagedTables] = None, stream=None) -> None:
        """Trim every sequence to `budget` entries by score (lsa_paged_evict)."""
        self._call("lsa_paged_evict", stream, int(budget), int(n_sink), int(n_recent), self._dst(dst))

    def read_err(self) -> int:
        return int(self.err.item())
