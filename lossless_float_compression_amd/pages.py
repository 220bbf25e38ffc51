"""Who holds which page of a paged K/V cache: rows of a page table that go on from other rows, pages given out
and taken back, pages brought together at the front, and the copies that this asks for, in all layers' caches at once.

A `PagePool` keeps one count for each page, the number of table rows that hold it; the caches of a model's layers
(`PagedKVCache`) have the same pages, so one pool and one table serve them all.  One step of a beam search:

    beams = beam_select(logits, scores, n_beams)                 # parents and tokens of the next beams
    pool.fork(table, held, beams.parents)                        # each row goes on from its parent's pages
    layers.copy_pages(pool.extend(batch, held))                  # room for a token; shared pages that it is written to are copied
    cache.append(k, v, batch); cache.attend(q, batch)            # in each layer

Nothing waits for the GPU, so a step can be captured in a HIP graph.
"""
from __future__ import annotations

import ctypes as C
from typing import Optional, Sequence, Tuple

import torch
import torch.autograd.forward_ad as _forward

from . import paged as _paged
from . import zx as _zx
from .paged import PagedBatch, PagedKVCache, _device_of, _int32, _meet

MOST_PAGES = 1 << 23
MOST_SEQS = 2048                         # of one `extend`, and beams of a group


class zx_page_pool(C.Structure):
    _fields_ = [("n_pages", C.c_uint32), ("page_tokens", C.c_uint32), ("refs", C.c_void_p)]


class zx_page_rows(C.Structure):
    _fields_ = [("page_table", C.c_void_p), ("held", C.c_void_p), ("n_seqs", C.c_uint32), ("table_width", C.c_uint32)]


class zx_page_copies(C.Structure):
    _fields_ = [("pairs", C.c_void_p), ("count", C.c_void_p), ("cap", C.c_uint32), ("reserved_", C.c_uint32)]


def _bind(L) -> None:
    P, U32, I, SZ = C.c_void_p, C.c_uint32, C.c_int, C.c_size_t
    O, R, K = C.POINTER(zx_page_pool), C.POINTER(zx_page_rows), C.POINTER(zx_page_copies)
    L.zx_pages_fork.argtypes = [O, R, U32, P, P, P]
    L.zx_pages_trim.argtypes = [O, R, P, P, P]
    L.zx_pages_extend_workspace_bytes.argtypes = [O, U32]
    L.zx_pages_extend_workspace_bytes.restype = SZ
    L.zx_pages_extend.argtypes = [O, R, P, U32, U32, P, K, P, SZ, P, P]
    L.zx_pages_compact_workspace_bytes.argtypes = [O]
    L.zx_pages_compact_workspace_bytes.restype = SZ
    L.zx_pages_compact.argtypes = [O, R, P, K, P, SZ, P, P]
    L.zx_paged_copy.argtypes = [C.POINTER(_paged.zx_paged_cache), U32, K, P, P]
    for f in ("zx_pages_fork", "zx_pages_trim", "zx_pages_extend", "zx_pages_compact", "zx_paged_copy"):
        getattr(L, f).restype = I


_bound = None


def _lib():
    global _bound
    if _bound is None:
        L = _zx.lib()
        _bind(L)
        _bound = L
    return _bound


# the cheap accessors, where this torch build has them
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _away(index: int, stream) -> bool:
    """Whether a call has to change the current device or stream first (a raw stream handle will not do: memory is
    allocated on the stream that uses it)."""
    if stream is None:
        return _device() != index
    if not isinstance(stream, torch.Stream):
        raise ValueError("stream must be a torch stream (torch.cuda.ExternalStream makes one of a raw handle)")
    return _device() != index or _zx._side_stream(stream) is not None


def _elsewhere(device: torch.device, stream, tensors, call):
    """`call(stream)` with the device current, or on a side stream after what the current one holds; the tensors' memory is
    not handed out again before the side stream is done with them."""
    if torch.cuda.current_device() != device.index:
        with torch.cuda.device(device):
            return call(stream)
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the call's tensors on {device}")
    stream.wait_stream(torch.cuda.current_stream())
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    with torch.cuda.stream(stream):
        return call(None)


def _span(t: torch.Tensor) -> Tuple[int, int]:
    """First and last byte, and one more, that a tensor reaches."""
    p = t.data_ptr()
    if t.numel() == 0:
        return p, p
    return p, p + (sum((n - 1) * st for n, st in zip(t.shape, t.stride())) + 1) * t.element_size()


def _meets(a: torch.Tensor, b: torch.Tensor) -> bool:
    (p, q), (r, s) = _span(a), _span(b)
    return p < s and r < q


def _words(t: torch.Tensor) -> Tuple[int, int]:
    """`_span` of a contiguous int32 tensor."""
    p = t.data_ptr()
    return p, p + 4 * t.numel()


def _all_apart(spans: list) -> None:
    """Refuse stretches of memory that meet."""
    spans.sort()
    end = 0
    for p, q in spans:
        if p < end and p < q:
            raise ValueError("the tensors that are read and written must not share memory")
        if q > end:
            end = q


class PageCopies:
    """A list of copies to be made, on the device: `count` (int32 [1]) says how many of the rows of `pairs` (int32 [cap, 3]: source
    page, destination page, tokens from the page's start) are meant.  Allocated here, or given."""

    def __init__(self, cap: int, pairs: Optional[torch.Tensor] = None, count: Optional[torch.Tensor] = None, device="cuda"):
        if cap < 0 or cap > MOST_PAGES:
            raise ValueError(f"cap must be 0..{MOST_PAGES}")
        given = pairs if pairs is not None else count
        device = _device_of(device) if given is None else given.device
        if pairs is None:
            pairs = torch.full((cap, 3), -1, dtype=torch.int32, device=device)
        if count is None:
            count = torch.zeros(1, dtype=torch.int32, device=device)
        _int32(pairs, "pairs")
        _int32(count, "count")
        if pairs.shape != (cap, 3) or count.shape != (1,) or pairs.device != count.device or _meets(pairs, count):
            raise ValueError(f"pairs must be [{cap}, 3] and count [1], on one device and apart")
        self.cap, self.pairs, self.count, self.device = int(cap), pairs, count, pairs.device
        self._spans = (_words(pairs), _words(count))
        self._c = zx_page_copies(pairs.data_ptr(), count.data_ptr(), self.cap, 0)
        self._ref = C.byref(self._c)


class PagePool:
    """Which of `n_pages` pages (up to 2^23) of page_tokens tokens are held, and by how many table rows: `refs`, int32
    [n_pages], allocated (all free) or given.  A page with a count of 0 or less is free; raise a page's count to
    keep it beside the rows (a cached prompt's, say).

    The methods take a page table (device int32 [rows, width]) and `held` (device int32 [rows]): row s holds the pages of its first
    ceil(held[s] / page_tokens) entries; those behind are neither looked at nor changed, except that `extend` fills them.  Everything
    is read on the device when the work runs.  err: device int32 word, set to 4 where lengths, parents or page ids were out of range
    or a count fell below zero (such rows are left out, or groups), to 6 where too few pages were free.  stream: a torch
    stream to run on after the work already enqueued on the current one.  Calls on one pool must not overlap in time."""

    def __init__(self, n_pages: int, page_tokens: int, refs: Optional[torch.Tensor] = None, device="cuda"):
        if not 0 < n_pages <= MOST_PAGES:
            raise ValueError(f"n_pages must be 1..{MOST_PAGES}")
        if not (16 <= page_tokens <= 4096 and page_tokens & (page_tokens - 1) == 0):
            raise ValueError("page_tokens must be a power of two from 16 to 4096")
        if refs is None:
            refs = torch.zeros(n_pages, dtype=torch.int32, device=_device_of(device))
        if _int32(refs, "refs").shape != (n_pages,):
            raise ValueError(f"refs must be [{n_pages}]")
        self.n_pages, self.page_tokens, self.refs, self.device = int(n_pages), int(page_tokens), refs, refs.device
        self._index = refs.get_device()
        self._c = zx_page_pool(self.n_pages, self.page_tokens, refs.data_ptr())
        self._ref = C.byref(self._c)
        self._bytes = torch.empty(0, dtype=torch.uint8, device=self.device)     # what workspaces are allocated like
        self._own = _words(refs)
        self._needs = {}                         # workspace sizes, by the number of rows

    # ---- argument checks
    def _rows(self, table: torch.Tensor, held: torch.Tensor, err: Optional[torch.Tensor], *apart) -> Tuple[zx_page_rows, Optional[int]]:
        """The rows, and err's address; `apart`: spans of what else is read or written."""
        _int32(table, "table", self._index)
        try:
            n, width = table.shape
        except ValueError:
            n, width = -1, 0
        return self._rows_at(table.data_ptr(), n, width, held, err, apart)

    def _rows_at(self, t: int, n: int, width: int, held: torch.Tensor, err: Optional[torch.Tensor], apart) -> Tuple[zx_page_rows, Optional[int]]:
        """The same for a table at an address."""
        if _int32(held, "held", self._index).shape != (n,):
            raise ValueError("table must be [rows, width] and held [rows]")
        h, e = held.data_ptr(), None
        spans = [(t, t + 4 * n * width), (h, h + 4 * n), self._own, *apart]
        if err is not None:
            spans.append(_words(_int32(err, "err", self._index)))
            e = err.data_ptr()
        _all_apart(spans)
        return zx_page_rows(t, h, n, width), e

    def _list(self, copies: Optional[PageCopies], least: int) -> PageCopies:
        if copies is None:
            return PageCopies(least, device=self.device)
        if copies.device != self.device or copies.cap < least:
            raise ValueError(f"copies must be on {self.device} with room for {least}")
        return copies

    # ---- operators
    def fork(self, table: torch.Tensor, held: torch.Tensor, parents: torch.Tensor, err: Optional[torch.Tensor] = None, stream=None) -> None:
        """Rows go on from other rows.  parents: device int32 [groups, beams] (up to 2048 beams) for rows groups * beams:
        row r of a group takes what row parents[r] of the group held before the call, -1: nothing.  No page is copied:
        rows share them, and pages that no row holds any more are free.  A group with a parent or a length out of range stays as it is."""
        if _away(self._index, stream):
            return _elsewhere(self.device, stream, (table, held, parents, err, self.refs), lambda s: self.fork(table, held, parents, err, s))
        _int32(parents, "parents", self._index)
        rows, e = self._rows(table, held, err, _words(parents))
        if parents.dim() != 2 or parents.numel() != rows.n_seqs or not 0 < parents.shape[1] <= MOST_SEQS:
            raise ValueError(f"parents must be [groups, beams] for the table's {rows.n_seqs} rows, of up to {MOST_SEQS} beams")
        st = (_bound or _lib()).zx_pages_fork(self._ref, C.byref(rows), parents.shape[1], parents.data_ptr(), e, _stream_of(self._index))
        if st != 0:
            raise _zx.ZxError("zx_pages_fork", st)

    def trim(self, table: torch.Tensor, held: torch.Tensor, keep: Optional[torch.Tensor] = None, err: Optional[torch.Tensor] = None,
             stream=None) -> None:
        """Rows keep their first keep[s] tokens (device int32 [rows]; None: none, the rows are freed) and give back the pages behind
        them.  A row that has no more than that stays as it is."""
        if _away(self._index, stream):
            return _elsewhere(self.device, stream, (table, held, keep, err, self.refs), lambda s: self.trim(table, held, keep, err, s))
        if keep is not None and _int32(keep, "keep", self._index).shape != held.shape:
            raise ValueError("keep must be [rows]")
        rows, e = self._rows(table, held, err, *(() if keep is None else (_words(keep),)))
        st = (_bound or _lib()).zx_pages_trim(self._ref, C.byref(rows), None if keep is None else keep.data_ptr(), e, _stream_of(self._index))
        if st != 0:
            raise _zx.ZxError("zx_pages_trim", st)

    def extend(self, batch: PagedBatch, held: torch.Tensor, copies: Optional[PageCopies] = None, err: Optional[torch.Tensor] = None,
               stream=None) -> PageCopies:
        """Room for a batch's new tokens: row s of batch.page_table gets pages for q_start[s + 1] - q_start[s] tokens more than held[s], and
        held[s] and batch.kv_len[s] become what it then has.  New pages are the lowest free ones, in order of row and place.
        A row that goes on in a page with tokens that other rows hold too gets one of its own there, and a copy of its tokens is
        entered in `copies` (allocated when None), which is returned: carry it out (`PagedLayers.copy_pages`) before appending.  Where all that hold
        the page go on in it, the first of them keeps it.

        Where fewer pages are free than the call needs nothing is given out, held stays, all kv_len are 0 (append and attend
        then skip the tokens) and `err` is 6.  The same, with 4, for a single row that is out of range or passes the
        batch's max_q or max_kv.  Up to 2048 rows."""
        if _away(self._index, stream):
            return _elsewhere(self.device, stream, (batch.q_start, batch.kv_len, batch.page_table, held, err, self.refs,
                                                    *(() if copies is None else (copies.pairs, copies.count))),
                              lambda s: self.extend(batch, held, copies, err, s))
        if batch._index != self._index:
            raise ValueError(f"the batch is on {batch.device}, the pool on {self.device}")
        if batch.n_seqs > MOST_SEQS:
            raise ValueError(f"a batch of up to {MOST_SEQS} sequences")
        copies = self._list(copies, batch.n_seqs)
        c = batch._c
        n, q, kv = c.n_seqs, c.q_start, c.kv_len
        rows, e = self._rows_at(c.page_table or 0, n, c.table_width, held, err, (*copies._spans, (q, q + 4 * n + 4), (kv or 0, (kv or 0) + 4 * n)))
        need = self._needs.get(n)
        if need is None:
            need = self._needs[n] = _lib().zx_pages_extend_workspace_bytes(self._ref, n)
        ws = self._bytes.new_empty(need)         # (held until the launches are enqueued: the call lets other threads run)
        st = (_bound or _lib()).zx_pages_extend(self._ref, C.byref(rows), q, c.max_q, c.max_kv, kv, copies._ref, ws.data_ptr(), need, e,
                                                _stream_of(self._index))
        if st != 0:
            raise _zx.ZxError("zx_pages_extend", st)
        return copies

    def compact(self, table: Optional[torch.Tensor] = None, held: Optional[torch.Tensor] = None, copies: Optional[PageCopies] = None,
                remap: Optional[torch.Tensor] = None, err: Optional[torch.Tensor] = None, stream=None) -> Tuple[PageCopies, torch.Tensor]:
        """Bring the pages in use together: with L of them, those at L and behind move, in order, into the free ones ahead, and the table
        follows.  Returns the copies to be made (room for n_pages // 2, allocated when None; carry them out before anything else) and
        remap, int32 [n_pages]: where each page is now, -1 for a free one (other tables follow by it).  Afterwards the pages
        from L on are free, and `cache.k[:L]` is all there is."""
        if _away(self._index, stream):
            return _elsewhere(self.device, stream, (table, held, remap, err, self.refs, *(() if copies is None else (copies.pairs, copies.count))),
                              lambda s: self.compact(table, held, copies, remap, err, s))
        if (table is None) != (held is None):
            raise ValueError("give both table and held, or neither")
        copies = self._list(copies, self.n_pages // 2)
        if remap is None:
            remap = torch.empty(self.n_pages, dtype=torch.int32, device=self.device)
        elif _int32(remap, "remap", self._index).shape != (self.n_pages,):
            raise ValueError(f"remap must be [{self.n_pages}]")
        spans = (*copies._spans, _words(remap))
        if table is None:
            rows, e = zx_page_rows(None, None, 0, 0), None
            if err is not None:
                e = _int32(err, "err", self._index).data_ptr()
                spans += (_words(err),)
            _all_apart([self._own, *spans])
        else:
            rows, e = self._rows(table, held, err, *spans)
        need = self._needs.get(None)
        if need is None:
            need = self._needs[None] = _lib().zx_pages_compact_workspace_bytes(self._ref)
        ws = self._bytes.new_empty(need)         # (held as in extend)
        st = (_bound or _lib()).zx_pages_compact(self._ref, C.byref(rows), remap.data_ptr(), copies._ref, ws.data_ptr(), need, e, _stream_of(self._index))
        if st != 0:
            raise _zx.ZxError("zx_pages_compact", st)
        return copies, remap


class PagedLayers:
    """The caches of a model's layers, of one shape and type: what `copy_pages` acts on in one launch (or one for every 40)."""

    def __init__(self, caches: Sequence[PagedKVCache]):
        caches = list(caches)
        if not caches:
            raise ValueError("no caches")
        f = caches[0]
        for c in caches:
            if c._key != f._key or c.n_pages != f.n_pages or c.device != f.device:
                raise ValueError("the caches must have one shape, type and device")
        self.caches, self.device, self._index = caches, f.device, f._index
        pages = sorted(((*_span(t), t) for c in caches for t in (c.k, c.v)), key=lambda x: x[0])
        steps = lambda t: sorted(((st, n) for st, n in zip(t.stride()[:3], t.shape[:3]) if n > 1), reverse=True)   # noqa: E731
        for i, (p, q, t) in enumerate(pages):    # against those that begin before this one ends
            for r, _, u in pages[i + 1:]:
                if r >= q:
                    break
                if _meet(steps(t), steps(u), (r - p) // t.element_size(), f.head_dim):
                    raise ValueError("the caches must have pages of their own")
        bounds = sorted((_span(c.bounds) for c in caches if c.bounds is not None))
        if any(a[1] > b[0] for a, b in zip(bounds, bounds[1:])):
            raise ValueError("the caches must have bounds of their own")
        self._c = (_paged.zx_paged_cache * len(caches))(*[c._c for c in caches])
        self._tensors = tuple(t for c in caches for t in (c.k, c.v, c.bounds) if t is not None)
        self._gradients = any(t.requires_grad for t in self._tensors)

    def copy_pages(self, copies: PageCopies, err: Optional[torch.Tensor] = None, stream=None) -> None:
        """Carry `copies` out in every cache: the first tokens of a source page's keys and values, bit for bit, over those of the destination
        page, and the bounds of the blocks that they reach into.  A page that is written must be in no other pair.  Pairs with page ids
        or counts of tokens out of range are left out, with 4 in `err` (device int32 word).  stream: as `PagePool`."""
        _copy(self, self._c, len(self.caches), copies, err, stream)


def _copy(of, structs, n: int, copies: PageCopies, err: Optional[torch.Tensor], stream) -> None:
    """The copies in the caches of `of` (a PagedLayers or one PagedKVCache), n structs."""
    if _away(of._index, stream):
        return _elsewhere(of.device, stream, (copies.pairs, copies.count, err, *of._tensors), lambda s: _copy(of, structs, n, copies, err, s))
    if copies.device != of.device:
        raise ValueError(f"the copies are on {copies.device}, the caches on {of.device}")
    if of._gradients or _forward._current_level >= 0:
        for t in of._tensors:
            _paged._no_gradient(t, "a tensor of the caches")
    e = None if err is None else _int32(err, "err", of._index).data_ptr()
    st = (_bound or _lib()).zx_paged_copy(structs, n, copies._ref, e, _stream_of(of._index))
    if st != 0:
        raise _zx.ZxError("zx_paged_copy", st)
