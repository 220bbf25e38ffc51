"""Paged K/V cache: append with the position rotation on the way, attention over the pages,
and attention over the blocks that a cheap score selects.

This is the uncompressed side of a K/V cache: a model's new keys and values go into
pages token by token, attention reads the pages, and full pages can be compressed into
a `KVSlotPool` (`PagedKVCache.stow`) and brought back (`restore`).  With 8 heads, pages of
512 tokens and 128 channels, each head's part of a page is one 65536-element block.

One step of a model, per layer:

    cache.append(k, v, batch, q=q, rotary=rotary, q_out=q)   # keys into pages, queries turned in place
    out = cache.attend(q, batch)                             # or, over selected blocks only:
    out = cache.attend(q, batch, blocks=cache.select(q, batch, top_k=32))

Nothing waits for the GPU, so a step can be captured in a HIP graph; lengths and page
tables are read on the device and may be rewritten between replays.
"""
from __future__ import annotations

import ctypes as C
import math
from typing import Optional, Tuple, Union

import torch
import torch.autograd.forward_ad as _forward

from . import zx as _zx

_ANY = 0x7FFFFFFF
_MOST_NEEDS = 256                        # workspace sizes that a batch remembers


class zx_paged_cache(C.Structure):
    _fields_ = [
        ("dtype", C.c_int32), ("n_pages", C.c_uint32), ("kv_heads", C.c_uint32), ("head_dim", C.c_uint32),
        ("page_tokens", C.c_uint32), ("block_tokens", C.c_uint32), ("k", C.c_void_p), ("v", C.c_void_p),
        ("k_page_stride", C.c_uint64), ("k_head_stride", C.c_uint64), ("k_token_stride", C.c_uint64),
        ("v_page_stride", C.c_uint64), ("v_head_stride", C.c_uint64), ("v_token_stride", C.c_uint64),
        ("k_scale", C.c_void_p), ("v_scale", C.c_void_p), ("bounds", C.c_void_p),
    ]


class zx_paged_batch(C.Structure):
    _fields_ = [
        ("n_seqs", C.c_uint32), ("table_width", C.c_uint32), ("max_q", C.c_uint32), ("max_kv", C.c_uint32),
        ("q_start", C.c_void_p), ("kv_len", C.c_void_p), ("page_table", C.c_void_p),
    ]


class zx_rows(C.Structure):
    _fields_ = [("p", C.c_void_p), ("token_stride", C.c_uint64), ("head_stride", C.c_uint64)]


class zx_rotary(C.Structure):
    _fields_ = [("inv_freq", C.c_void_p), ("dims", C.c_uint32), ("interleaved", C.c_int32), ("magnitude", C.c_float),
                ("reserved_", C.c_uint32)]


def _bind(L) -> None:
    P, U32, I, SZ = C.c_void_p, C.c_uint32, C.c_int, C.c_size_t
    K, B, R = C.POINTER(zx_paged_cache), C.POINTER(zx_paged_batch), C.POINTER(zx_rows)
    L.zx_paged_append.argtypes = [K, B, U32, R, R, C.POINTER(zx_rotary), P, R, U32, R, P, P]
    L.zx_paged_attend_workspace_bytes.argtypes = [K, B, U32, U32, U32, U32]
    L.zx_paged_attend_workspace_bytes.restype = SZ
    L.zx_paged_attend.argtypes = [K, B, U32, R, U32, R, P, C.c_float, I, U32, P, U32, P, SZ, P, P]
    L.zx_paged_select_workspace_bytes.argtypes = [K, B, U32]
    L.zx_paged_select_workspace_bytes.restype = SZ
    L.zx_paged_select.argtypes = [K, B, U32, R, U32, U32, U32, U32, P, P, SZ, P, P]
    for f in ("zx_paged_append", "zx_paged_attend", "zx_paged_select"):
        getattr(L, f).restype = I


_bound = None


def _lib():
    global _bound
    if _bound is None:
        L = _zx.lib()
        _bind(L)
        _bound = L
    return _bound


def _device_of(device) -> torch.device:
    d = torch.device(device)
    if d.type == "cuda" and d.index is None:
        d = torch.device("cuda", torch.cuda.current_device())
    return d


def _int32(t, name: str, index: Optional[int] = None) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.int32 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous device int32 tensor")
    if index is not None and t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the cache on cuda:{index}")
    return t


def _no_gradient(t: torch.Tensor, name: str) -> None:
    """Refuse a tensor that autograd, of either mode, would want the result to follow from."""
    if (t.requires_grad and torch.is_grad_enabled()) or (
            _forward._current_level >= 0 and _forward.unpack_dual(t).tangent is not None):
        raise ValueError(f"{name} requires a gradient, which these operators do not have: detach it or use torch.no_grad() "
                         "(a tangent is carried there too)")


def _apart(sizes, strides, width: int) -> bool:
    """Whether rows of `width` elements at these strides are apart from each other: each stride
    steps over all that the smaller ones reach."""
    for st, n in sorted((st, n) for n, st in zip(sizes, strides) if n > 1):
        if st < width:
            return False
        width = st * (n - 1) + width
    return True


def _meet(a, b, offset: int, width: int) -> bool:
    """Whether rows of `width` elements at the strides of `a` and, `offset` elements on, of `b` may share memory.  `a` and
    `b` are lists of (stride, n) that are apart in themselves, the largest stride first.  Layouts that step alike from the
    outside in are followed to the rows; where they part, what is left of each counts as one stretch."""
    reach = lambda x: sum(st * (n - 1) for st, n in x) + width   # noqa: E731
    if offset >= reach(a) or -offset >= reach(b):
        return False
    if not a or not b or a[0] != b[0]:
        return True
    st, n = a[0]
    a, b = a[1:], b[1:]
    least = -((offset + reach(b) - 1) // st)                  # steps of b less those of a for which the rest may meet
    most = (reach(a) - 1 - offset) // st
    return any(_meet(a, b, offset + m * st, width) for m in range(max(least, 1 - n), min(most, n - 1) + 1))


class Rotary:
    """Rotary positions: in the first `dims` channels of a head (a multiple of 16), pair j
    is turned by position * inv_freq[j] and scaled by `magnitude`.  Pairs are channels
    (j, j + dims / 2), or (2 j, 2 j + 1) with `interleaved`.

    inv_freq[j] = base^(-2 j / dims), stretched for long contexts by `scaling`:
      "linear"  divided by `factor`
      "ntk"     a larger base, base * factor^(dims / (dims - 2)): the slowest pair is divided by
                `factor`, the fastest left alone
      "bands"   by wavelength against the trained length `original`: pairs that turn more than
                `high` times in it are left alone, those that turn less than `low` times are
                divided by `factor`, a straight blend between
      "yarn"    the same two ends with a blend that is straight over the pairs' indices
                (defaults high = 32, low = 1), and magnitude 0.1 ln(factor) + 1
    or given as a float64 tensor [dims / 2].  Frequencies and angles are kept in 64 bits, so
    positions in the millions turn by the right angle."""

    def __init__(self, dims: int, base: float = 10000.0, interleaved: bool = False, scaling: Optional[str] = None,
                 factor: float = 1.0, original: int = 8192, low: float = 1.0, high: Optional[float] = None,
                 magnitude: Optional[float] = None, inv_freq: Optional[torch.Tensor] = None, device="cuda"):
        if dims <= 0 or dims % 16 or dims > 256:
            raise ValueError("dims must be a multiple of 16, at most 256")
        if inv_freq is None:
            inv_freq = self.frequencies(dims, base, scaling, factor, original, low, high).to(_device_of(device))
        elif scaling is not None:
            raise ValueError("give either inv_freq or a scaling")
        if inv_freq.dtype != torch.float64 or inv_freq.shape != (dims // 2,) or not inv_freq.is_contiguous():
            raise ValueError("inv_freq must be a contiguous float64 tensor [dims / 2]")
        if magnitude is None:
            magnitude = 0.1 * math.log(factor) + 1.0 if scaling == "yarn" and factor > 1.0 else 1.0
        self.dims, self.interleaved, self.magnitude, self.inv_freq = int(dims), bool(interleaved), float(magnitude), inv_freq
        self._c = zx_rotary(inv_freq.data_ptr(), self.dims, int(self.interleaved), self.magnitude, 0)
        self._ref = C.byref(self._c)

    @staticmethod
    def frequencies(dims: int, base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0,
                    original: int = 8192, low: float = 1.0, high: Optional[float] = None) -> torch.Tensor:
        """The float64 angle per position of each pair (on the host)."""
        if not (base > 0 and factor > 0 and original > 0):
            raise ValueError("base, factor and original must be positive")
        j = torch.arange(0, dims, 2, dtype=torch.float64)
        if scaling == "ntk":
            if dims < 4:
                raise ValueError("ntk needs dims above 2")
            base = base * factor ** (dims / (dims - 2))
        f = base ** (-j / dims)
        if scaling in (None, "ntk"):
            return f
        if scaling == "linear":
            return f / factor
        if scaling == "bands":
            high = 4.0 if high is None else high
            if not high > low:
                raise ValueError("high must be above low")
            keep = ((original * f / (2 * math.pi) - low) / (high - low)).clamp(0.0, 1.0)
        elif scaling == "yarn":
            high = 32.0 if high is None else high
            if not high > low > 0:
                raise ValueError("high must be above low, and low positive")
            at = lambda turns: dims * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))   # noqa: E731
            a, b = max(math.floor(at(high)), 0), min(math.ceil(at(low)), dims - 1)
            keep = 1.0 - ((j / 2 - a) / max(b - a, 1e-3)).clamp(0.0, 1.0)
        else:
            raise ValueError(f"unknown scaling {scaling!r}")
        return (1.0 - keep) * f / factor + keep * f


class PagedBatch:
    """Which tokens a call is about: sequence s has the packed rows q_start[s] .. q_start[s + 1]
    - 1 as its new tokens and kv_len[s] tokens in all, the new ones included; token t is in page
    page_table[s, t // page_tokens].  Device int32 tensors [n + 1], [n] and [n, width]; they
    may be rewritten in place between calls.

    max_q and max_kv say on the host how long a sequence may get (new tokens, all tokens);
    launches are shaped by them, and a sequence that passes one is left out and reported in
    `err`.  Without them any length that fits the call and the table is taken."""

    def __init__(self, q_start: torch.Tensor, kv_len: torch.Tensor, page_table: torch.Tensor,
                 max_q: Optional[int] = None, max_kv: Optional[int] = None):
        for t, name in ((q_start, "q_start"), (kv_len, "kv_len"), (page_table, "page_table")):
            _int32(t, name)
            if t.device != q_start.device:
                raise ValueError("q_start, kv_len and page_table must be on one device")
        n = kv_len.numel()
        if q_start.shape != (n + 1,) or kv_len.shape != (n,) or page_table.dim() != 2 or page_table.shape[0] != n:
            raise ValueError("q_start must be [n + 1], kv_len [n] and page_table [n, width]")
        if (max_q is not None and max_q < 0) or (max_kv is not None and max_kv < 0):
            raise ValueError("max_q and max_kv must not be negative")
        self.q_start, self.kv_len, self.page_table = q_start, kv_len, page_table
        self.n_seqs = n
        self.device = q_start.device
        self._index = q_start.get_device()
        self._needs = {}                 # workspace sizes, by the sizes that decide them
        self._c = zx_paged_batch(n, page_table.shape[1], _ANY if max_q is None else min(int(max_q), _ANY),
                                 _ANY if max_kv is None else min(int(max_kv), _ANY), q_start.data_ptr(),
                                 kv_len.data_ptr(), page_table.data_ptr())
        self._ref = C.byref(self._c)

    def _ask(self, key, f, *args) -> int:
        """The workspace size `f(*args)`, remembered under `key` (all are let go when there are many)."""
        if len(self._needs) >= _MOST_NEEDS:
            self._needs.clear()
        need = self._needs[key] = f(*args)
        return need


class PagedKVCache:
    """`n_pages` pages of page_tokens tokens (a power of two, 16..4096) of kv_heads heads of
    head_dim (64, 128 or 256) channels, BF16 or FP8 E4M3.

    k, v           the pages, [n_pages, kv_heads, page_tokens, head_dim]; allocated (zeroed) here, or
                   given, apart from each other: any strides that are multiples of 16 bytes, channels contiguous
                   (so [n_pages, page_tokens, kv_heads, head_dim] pages are given as `.transpose(1, 2)`)
    k_scale, v_scale  FP8: a stored value x stands for x * scale[head] (a positive number, or a
                   device float32 tensor [kv_heads])
    block_tokens   keep bounds, the smallest and largest key per channel, of every so many
                   tokens (a power of two, 16..256, at most page_tokens): what `select` needs
    bounds         BF16 [n_pages, kv_heads, page_tokens / block_tokens, 2, head_dim], allocated or given
    """

    def __init__(self, n_pages: int, kv_heads: int, head_dim: int = 128, page_tokens: int = 512, dtype: int = _zx.BF16,
                 block_tokens: Optional[int] = None, k: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None,
                 bounds: Optional[torch.Tensor] = None, k_scale: Union[None, float, torch.Tensor] = None,
                 v_scale: Union[None, float, torch.Tensor] = None, device="cuda"):
        if dtype not in (_zx.BF16, _zx.FP8_E4M3FN):
            raise ValueError("dtype must be BF16 or FP8_E4M3FN")
        if n_pages <= 0 or kv_heads <= 0:
            raise ValueError("n_pages and kv_heads must be positive")
        if head_dim not in (64, 128, 256):
            raise ValueError("head_dim must be 64, 128 or 256")
        pow2 = lambda x, a, b: a <= x <= b and x & (x - 1) == 0   # noqa: E731
        if not pow2(page_tokens, 16, 4096):
            raise ValueError("page_tokens must be a power of two from 16 to 4096")
        if block_tokens is not None and not pow2(block_tokens, 16, min(256, page_tokens)):
            raise ValueError("block_tokens must be a power of two from 16 to 256, at most page_tokens")
        if (k is None) != (v is None):
            raise ValueError("give both k and v, or neither")
        if bounds is not None and block_tokens is None:
            raise ValueError("bounds need block_tokens")
        self.dtype, self.n_pages, self.kv_heads = int(dtype), int(n_pages), int(kv_heads)
        self.head_dim, self.page_tokens = int(head_dim), int(page_tokens)
        self.block_tokens = None if block_tokens is None else int(block_tokens)
        self.torch_dtype = torch.bfloat16 if dtype == _zx.BF16 else torch.float8_e4m3fn
        self.device = k.device if k is not None else _device_of(device)
        shape = (self.n_pages, self.kv_heads, self.page_tokens, self.head_dim)
        if k is None:
            bits = torch.int16 if dtype == _zx.BF16 else torch.uint8
            k = torch.zeros(shape, dtype=bits, device=self.device).view(self.torch_dtype)
            v = torch.zeros(shape, dtype=bits, device=self.device).view(self.torch_dtype)
        per16 = 8 if dtype == _zx.BF16 else 16
        for t, name in ((k, "k"), (v, "v")):
            if t.shape != shape or t.dtype != self.torch_dtype or not t.is_cuda or t.device != self.device:
                raise ValueError(f"{name} must be a {self.torch_dtype} device tensor {list(shape)}")
            if t.stride(3) != 1 or any(t.stride(i) % per16 for i in range(3)) or t.data_ptr() % 16:
                raise ValueError(f"{name}: channels must be contiguous and the other strides multiples of 16 bytes")
            if t.stride(2) < self.head_dim or not _apart(t.shape[:3], t.stride()[:3], self.head_dim):
                raise ValueError(f"{name}: rows must not overlap")
        steps = lambda t: sorted(((st, n) for st, n in zip(t.stride()[:3], shape[:3]) if n > 1), reverse=True)   # noqa: E731
        if _meet(steps(k), steps(v), (v.data_ptr() - k.data_ptr()) // k.element_size(), self.head_dim):
            raise ValueError("k and v must be pages of their own")
        self.k, self.v = k, v
        self.k_scale, self.v_scale = (self._scale(s, n) for s, n in ((k_scale, "k_scale"), (v_scale, "v_scale")))
        if self.block_tokens is not None:
            bshape = (self.n_pages, self.kv_heads, self.page_tokens // self.block_tokens, 2, self.head_dim)
            if bounds is None:
                bounds = torch.zeros(bshape, dtype=torch.bfloat16, device=self.device)
            if (bounds.shape != bshape or bounds.dtype != torch.bfloat16 or bounds.device != self.device
                    or not bounds.is_contiguous() or bounds.data_ptr() % 16):
                raise ValueError(f"bounds must be a contiguous bfloat16 device tensor {list(bshape)}")
        self.bounds = bounds
        ptr = lambda t: None if t is None else t.data_ptr()   # noqa: E731
        self._index = self.device.index
        self._key = (self.dtype, self.kv_heads, self.head_dim, self.page_tokens, self.block_tokens)
        self._c = zx_paged_cache(self.dtype, self.n_pages, self.kv_heads, self.head_dim, self.page_tokens,
                                 self.block_tokens or 0, k.data_ptr(), v.data_ptr(), k.stride(0), k.stride(1), k.stride(2),
                                 v.stride(0), v.stride(1), v.stride(2), ptr(self.k_scale), ptr(self.v_scale),
                                 ptr(bounds))
        self._ref = C.byref(self._c)
        self._bytes = torch.empty(0, dtype=torch.uint8, device=self.device)     # what workspaces are allocated like
        self._gradients = any(t is not None and t.requires_grad for t in (k, v, bounds, self.k_scale, self.v_scale))
        self._tensors = tuple(t for t in (self.k, self.v, self.k_scale, self.v_scale, self.bounds) if t is not None)

    def _scale(self, s, name: str) -> Optional[torch.Tensor]:
        if s is None:
            return None
        if self.dtype == _zx.BF16:
            raise ValueError(f"{name}: a BF16 cache has no scales")
        if not torch.is_tensor(s):
            if not (s > 0 and math.isfinite(s)):
                raise ValueError(f"{name} must be positive")
            s = torch.full((self.kv_heads,), float(s), dtype=torch.float32, device=self.device)
        if s.dtype != torch.float32 or s.shape != (self.kv_heads,) or s.device != self.device or not s.is_contiguous():
            raise ValueError(f"{name} must be a contiguous float32 device tensor [kv_heads]")
        return s

    def nbytes(self) -> int:
        """Device bytes of the pages and their bounds."""
        return sum(t.numel() * t.element_size() for t in (self.k, self.v, self.bounds) if t is not None)

    # ---- argument checks
    def _rows(self, t: torch.Tensor, name: str, heads: Optional[int], n: Optional[int], written: bool = False) -> zx_rows:
        sh = t.shape
        if t.dtype is not torch.bfloat16 or len(sh) != 3 or sh[2] != self.head_dim or (n is not None and sh[0] != n) or (
                heads is not None and sh[1] != heads):
            raise ValueError(f"{name} must be a bfloat16 tensor [{'tokens' if n is None else n}, "
                             f"{'heads' if heads is None else heads}, {self.head_dim}], got {t.dtype} {list(sh)}")
        if t.get_device() != self._index:
            raise ValueError(f"{name} is on {t.device}, the cache on {self.device}")
        if t.requires_grad:
            _no_gradient(t, name)
        s0, s1, s2 = t.stride()
        p = t.data_ptr()
        if s2 != 1 or s1 != sh[2] or s0 != s1 * sh[1]:           # (contiguous rows meet all that is asked for below)
            if sh[0] == 1:
                s0 = 0
            if sh[1] == 1:
                s1 = 0
            if s2 != 1 or s0 % 8 or s1 % 8:
                raise ValueError(f"{name}: channels must be contiguous and the other strides multiples of 16 bytes")
            if written and not _apart(sh[:2], (s0, s1), self.head_dim):
                raise ValueError(f"{name}: rows that are written must not overlap")
        if p % 16:
            raise ValueError(f"{name} must start at a multiple of 16 bytes")
        return zx_rows(p, s0, s1)

    def _common(self, batch: PagedBatch, err: Optional[torch.Tensor]):
        if batch._index != self._index:
            raise ValueError(f"the batch is on {batch.device}, the cache on {self.device}")
        if err is not None:
            return _int32(err, "err", self._index).data_ptr()
        return None

    def _followed(self, *given: Optional[torch.Tensor]) -> None:
        """Refuse what autograd follows."""
        for t in (*given, *self._tensors):
            if t is not None:
                _no_gradient(t, "an argument or a tensor of the cache")

    def _group(self, q: torch.Tensor) -> Tuple[int, int]:
        sh = q.shape
        if len(sh) != 3 or sh[1] == 0 or sh[1] % self.kv_heads:
            raise ValueError(f"q must be [tokens, heads, {self.head_dim}] with a multiple of {self.kv_heads} heads")
        return sh[0], sh[1]

    def _away(self, stream) -> bool:
        """Whether a call has to change the current device or stream first.  Workspaces and outputs are allocated on the
        stream that uses them, so a raw handle will not do: memory that the current stream let go would be shared with it."""
        if stream is not None and not isinstance(stream, torch.Stream):
            raise ValueError("stream must be a torch stream (torch.cuda.ExternalStream makes one of a raw handle)")
        return torch.cuda.current_device() != self._index or (stream is not None and _zx._side_stream(stream) is not None)

    def _elsewhere(self, stream, batch, tensors, call):
        """`call(stream)` with the cache's device current, or on a side stream after what the
        current one holds.  The tensors' memory is not handed out again before the side
        stream is done with them."""
        if torch.cuda.current_device() != self._index:
            with torch.cuda.device(self.device):
                return call(stream)
        if stream.device != self.device:
            raise ValueError(f"the stream is on {stream.device}, the cache on {self.device}")
        stream.wait_stream(torch.cuda.current_stream())
        for t in (*tensors, batch.q_start, batch.kv_len, batch.page_table, *self._tensors):
            if t is not None:
                t.record_stream(stream)
        with torch.cuda.stream(stream):
            return call(None)

    # ---- operators
    def append(self, k: torch.Tensor, v: torch.Tensor, batch: PagedBatch, q: Optional[torch.Tensor] = None,
               rotary: Optional[Rotary] = None, positions: Optional[torch.Tensor] = None,
               q_out: Optional[torch.Tensor] = None, err: Optional[torch.Tensor] = None, stream=None) -> Optional[torch.Tensor]:
        """Put the new tokens' keys and values (bf16 [tokens, kv_heads, head_dim]) at their
        places, keys rotated by `rotary`, rounded to the cache's type (FP8: divided by the
        head's scale, saturating), and widen the bounds of the blocks they fall into.  With
        `q` (bf16 [tokens, heads, head_dim]) the queries are rotated too, into q_out (allocated
        when None; q itself is fine, another overlap is not), which is returned.

        positions: device int32 [tokens] to rotate by, instead of the tokens' places.  Pages
        that are written must belong to one sequence only.  A token written at a place that
        held one widens its block's bounds further (they still hold, but are not the tightest),
        except at a block's first place, where they start anew.  Tokens whose place would be
        negative (kv_len below the number of new tokens), rows behind the last sequence and
        sequences that are out of range are skipped, their rows of q_out left as they are.

        err: device int32 word, 4 where lengths or page ids were out of range.  `stream`: a
        torch stream (no raw handle) to run on after the work already enqueued on the current one."""
        if self._away(stream):
            return self._elsewhere(stream, batch, (k, v, q, q_out, positions, err, None if rotary is None else rotary.inv_freq),
                                   lambda s: self.append(k, v, batch, q, rotary, positions, q_out, err, s))
        if self._gradients or _forward._current_level >= 0:
            self._followed(k, v, q, q_out, None if rotary is None else rotary.inv_freq)
        e = self._common(batch, err)
        n = k.shape[0]
        ck, cv = self._rows(k, "k", self.kv_heads, None), self._rows(v, "v", self.kv_heads, n)
        cq = co = None
        heads = 0
        if q is not None:
            heads = q.shape[1] if q.dim() == 3 else 0
            if heads == 0:
                raise ValueError("q must be [tokens, heads, head_dim]")
            cq = C.byref(self._rows(q, "q", None, n))
            if q_out is None:
                q_out = torch.empty((n, heads, self.head_dim), dtype=torch.bfloat16, device=self.device)
            co = C.byref(self._rows(q_out, "q_out", heads, n, True))
        elif q_out is not None:
            raise ValueError("q_out without q")
        cr = None
        if rotary is not None:
            if rotary.dims > self.head_dim or rotary.inv_freq.device != self.device:
                raise ValueError("rotary turns more channels than a head has, or is on another device")
            if rotary.inv_freq.requires_grad:
                _no_gradient(rotary.inv_freq, "inv_freq")
            cr = rotary._ref
        cp = None
        if positions is not None:
            if rotary is None or _int32(positions, "positions", self._index).shape != (n,):
                raise ValueError("positions must be [tokens], and need a rotary")
            cp = positions.data_ptr()
        st = _lib().zx_paged_append(self._ref, batch._ref, n, C.byref(ck), C.byref(cv), cr, cp, cq, heads, co, e,
                                    _zx._raw_stream(self.device))
        if st != 0:
            raise _zx.ZxError("zx_paged_append", st)
        return q_out

    def attend(self, q: torch.Tensor, batch: PagedBatch, scale: Optional[float] = None, causal: bool = True,
               window: int = 0, blocks: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
               lse: Optional[torch.Tensor] = None, err: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """softmax(scale q.k) v of the new tokens' queries (bf16 [tokens, heads, head_dim], heads a
        multiple of kv_heads; neighbouring heads share a K/V head) over their sequence's tokens:
        up to their own place (causal) or all, and with `window` only those less than `window`
        places before it (table entries of pages behind every window may hold anything).  scale defaults to
        head_dim^-1/2.  A row that sees no token is zero.  `out` may be q itself, and must not overlap it otherwise.

        blocks: int32 [tokens, kv_heads, n] (from `select`, or any list): only these blocks of
        block_tokens tokens, counted from the sequence's start, are read; a list ends at its first
        negative entry, a block entered twice counts twice.  Causal only, no window.
        lse: float32 [tokens, heads], filled with ln of the sum of exp(scaled scores).

        Rows behind the last sequence, and of sequences that are out of range, keep what they
        hold.  The same inputs give the same bits.  err, stream: as `append`."""
        if self._away(stream):
            return self._elsewhere(stream, batch, (q, out, lse, err, blocks),
                                   lambda s: self.attend(q, batch, scale, causal, window, blocks, out, lse, err, s))
        if self._gradients or _forward._current_level >= 0:
            self._followed(q, out, lse)
        e = self._common(batch, err)
        n, heads = self._group(q)
        cq = self._rows(q, "q", None, None)
        if out is None:
            out = torch.empty((n, heads, self.head_dim), dtype=torch.bfloat16, device=self.device)
        co = self._rows(out, "out", heads, n, True)
        if scale is None:
            scale = self.head_dim ** -0.5
        elif not (0.0 < scale <= 1e30):
            raise ValueError("scale must be positive")
        if not 0 <= window <= 0x3FFFFFFF:
            raise ValueError("window must be 0 (none) or a number of tokens")
        pl = pb = None
        if lse is not None:
            if lse.dtype is not torch.float32 or lse.shape != (n, heads) or lse.get_device() != self._index or not lse.is_contiguous():
                raise ValueError("lse must be a contiguous float32 device tensor [tokens, heads]")
            if lse.requires_grad:
                _no_gradient(lse, "lse")
            pl = lse.data_ptr()
        nb = 0
        if blocks is not None:
            if self.block_tokens is None or not causal or window:
                raise ValueError("blocks need a cache with block_tokens, causal attention and no window")
            _int32(blocks, "blocks", self._index)
            if blocks.dim() != 3 or blocks.shape[0] != n or blocks.shape[1] != self.kv_heads or not 0 < blocks.shape[2] <= 65536:
                raise ValueError(f"blocks must be [tokens, {self.kv_heads}, n]")
            nb = blocks.shape[2]
            pb = blocks.data_ptr()
        if n == 0:
            return out
        L = _lib()
        key = (self._key, n, heads, window, nb)
        need = batch._needs.get(key)
        if need is None:
            need = batch._ask(key, L.zx_paged_attend_workspace_bytes, self._ref, batch._ref, n, heads, window, nb)
        ws = self._bytes.new_empty(need) if need else None
        st = L.zx_paged_attend(self._ref, batch._ref, n, C.byref(cq), heads, C.byref(co), pl, scale, causal, window, pb, nb,
                               ws.data_ptr() if need else None, need, e, _zx._raw_stream(self.device))
        if st != 0:
            raise _zx.ZxError("zx_paged_attend", st)
        return out

    def select(self, q: torch.Tensor, batch: PagedBatch, top_k: int, keep_first: int = 1, keep_last: int = 1,
               blocks: Optional[torch.Tensor] = None, err: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """The blocks that each new token should read, for each K/V head: int32 [tokens, kv_heads,
        top_k], ascending, -1 behind the last.  The first keep_first blocks and the newest
        keep_last are always among them; the others are those with the largest upper bound of
        the group's summed scores, from the bounds that `append` keeps (ties: the earlier block).
        q holds rotated queries, as for `attend`.  Rows behind the last sequence are left as they
        are (-1 when allocated here).  err, stream: as `append`."""
        if self._away(stream):
            return self._elsewhere(stream, batch, (q, blocks, err),
                                   lambda s: self.select(q, batch, top_k, keep_first, keep_last, blocks, err, s))
        if self._gradients or _forward._current_level >= 0:
            self._followed(q)
        e = self._common(batch, err)
        n, heads = self._group(q)
        cq = self._rows(q, "q", None, None)
        if self.block_tokens is None:
            raise ValueError("select needs a cache with block_tokens")
        if not 0 < top_k <= 1024 or keep_first < 0 or keep_last < 0 or keep_first + keep_last > top_k:
            raise ValueError("top_k must be 1..1024 and at least keep_first + keep_last")
        if blocks is None:
            blocks = torch.full((n, self.kv_heads, top_k), -1, dtype=torch.int32, device=self.device)
        _int32(blocks, "blocks", self._index)
        if blocks.shape != (n, self.kv_heads, top_k):
            raise ValueError(f"blocks must be [{n}, {self.kv_heads}, {top_k}]")
        if n == 0:
            return blocks
        L = _lib()
        need = batch._needs.get((self._key, n))
        if need is None:
            need = batch._ask((self._key, n), L.zx_paged_select_workspace_bytes, self._ref, batch._ref, n)
        ws = self._bytes.new_empty(need) if need else None
        st = L.zx_paged_select(self._ref, batch._ref, n, C.byref(cq), heads, top_k, keep_first, keep_last, blocks.data_ptr(),
                               ws.data_ptr() if need else None, need, e, _zx._raw_stream(self.device))
        if st != 0:
            raise _zx.ZxError("zx_paged_select", st)
        return blocks

    # ---- pages in a slot pool
    def blocks_per_page(self) -> int:
        """65536-element codec blocks of the keys (and of the values) of one page."""
        n = self.kv_heads * self.page_tokens * self.head_dim
        if n % _zx.BLOCK_ELEMS:
            raise ValueError("a page of keys is not a whole number of 65536-element blocks")
        return n // _zx.BLOCK_ELEMS

    def _page_ids(self, pages: torch.Tensor, pool, slots: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
        """(which ids are pages, the ids with any page for the others, the slots with none for the others)"""
        if pool.dtype != self.dtype:
            raise TypeError("the pool has another dtype than the cache")
        if pool.signmant.device != self.device:
            raise ValueError(f"the pool is on {pool.signmant.device}, the cache on {self.device}")
        if not torch.is_tensor(pages) or pages.dtype not in (torch.int32, torch.int64) or pages.dim() != 1 or pages.device != self.device:
            raise ValueError("pages must be a device integer tensor [n]")
        _int32(slots, "slots", self._index)
        bpp = self.blocks_per_page()
        if slots.shape != (2, pages.numel(), bpp):
            raise ValueError(f"slots must be [2, {pages.numel()}, {bpp}]: keys, then values")
        ids = pages.long()
        ok = (ids >= 0) & (ids < self.n_pages)
        return ok, ids.clamp(0, self.n_pages - 1), torch.where(ok[:, None], slots, -1)

    def _pages_of(self, ids: torch.Tensor) -> torch.Tensor:
        raw = torch.int16 if self.dtype == _zx.BF16 else torch.uint8
        return torch.stack((self.k.view(raw)[ids], self.v.view(raw)[ids]))

    def stow(self, pages: torch.Tensor, pool, slots: torch.Tensor,
             err: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
        """Compress whole pages into `pool` (a KVSlotPool of the cache's dtype): the keys of page
        pages[i] into slots[0, i], its values into slots[1, i] (device int32 [2, n, blocks_per_page()],
        distinct).  Returns (status, bounds): status [2, n, blocks_per_page()] is 0, or 6 for a block
        that did not fit its slot (keep that page), or 1 where the page or the slot is none; bounds are the pages' rows of `self.bounds`,
        for `restore` (None without bounds).  The pages themselves are left as they are.  Runs on the current stream of the
        cache's device."""
        if torch.cuda.current_device() != self._index:
            with torch.cuda.device(self.device):
                return self.stow(pages, pool, slots, err)
        _, ids, slots = self._page_ids(pages, pool, slots)
        if slots.numel() == 0:
            return torch.empty_like(slots), None if self.bounds is None else self.bounds[ids]
        status = pool.append(self._pages_of(ids).reshape(-1), slots.reshape(-1), err=err)
        return status.view(slots.shape), None if self.bounds is None else self.bounds[ids]

    def restore(self, pages: torch.Tensor, pool, slots: torch.Tensor, bounds: Optional[torch.Tensor] = None,
                err: Optional[torch.Tensor] = None) -> None:
        """Bring stowed pages back, bit for bit, into pages pages[i] (any free ones, distinct), and
        their bounds with them.  A block whose slot is empty keeps what the page holds; ids that are
        no page are left out, with 4 in `err`.  Stream: as `stow`."""
        if torch.cuda.current_device() != self._index:
            with torch.cuda.device(self.device):
                return self.restore(pages, pool, slots, bounds, err)
        ok, ids, slots = self._page_ids(pages, pool, slots)
        if (bounds is None) != (self.bounds is None):
            raise ValueError("give the bounds that stow returned")
        if bounds is not None and (bounds.shape != (ids.numel(), *self.bounds.shape[1:]) or bounds.dtype != torch.bfloat16
                                   or bounds.device != self.device):
            raise ValueError("bounds are not those of these pages")
        if slots.numel() == 0:
            return
        held = self._pages_of(ids)
        pool.decode(slots.reshape(-1), out=held.view(-1, _zx.BLOCK_ELEMS).view(self.torch_dtype), err=err)
        # an id that is no page stands for one that is; where none is, the page put in its place keeps what it has
        same = torch.where(ok, torch.arange(ids.numel(), device=self.device), ok.int().argmax())
        ids, held = ids[same], held[:, same]
        if bounds is not None:
            bounds = torch.where(ok.any(), bounds[same], self.bounds[ids])
        raw = held.dtype
        self.k.view(raw).index_copy_(0, ids, held[0])
        self.v.view(raw).index_copy_(0, ids, held[1])
        if bounds is not None:
            self.bounds.index_copy_(0, ids, bounds)
